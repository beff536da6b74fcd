"""Rotary positions, attention weights of cached rows and the choice of the rows that stay, in 64 bits or whole numbers on
the CPU (test infrastructure), and the tolerances."""
from __future__ import annotations

import math
from decimal import Decimal, localcontext

import numpy as np

from tests.kv_ref import BF16, F32


# ------------------------------------------------------------------------------------------ rotary positions

def frequencies(rot, theta, scaling="none", factor=1.0, original_len=0, low=None, high=None):
    """radians per position of every pair, one at a time from the formulas"""
    low = 1.0 if low is None else low
    high = (32.0 if scaling == "ramp" else 4.0) if high is None else high
    f = []
    for j in range(rot // 2):
        x = theta ** (-2.0 * j / rot)
        if scaling == "linear":
            x /= factor
        elif scaling == "bands":
            wave = 2 * math.pi / x
            if wave >= original_len / low:
                x /= factor
            elif wave > original_len / high:
                s = (original_len / wave - low) / (high - low)
                x = (1 - s) * x / factor + s * x
        elif scaling == "ramp":
            def pair(turns):
                return rot * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(theta))
            a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
            r = min(1.0, max(0.0, (j - a) / max(b - a, 0.001)))
            x = x / factor * r + x * (1 - r)
        f.append(x)
    return np.array(f)


PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def exact_turns(rot, theta, factor=1):
    """turns per position of every pair, f_j / (2 pi factor), to 80 digits"""
    with localcontext() as c:
        c.prec = 80
        return [Decimal(theta) ** (Decimal(-2 * j) / rot) / (2 * PI * factor) for j in range(rot // 2)]


def turns_off(f, theta, position=1):
    """How many turns a position's angle may be off by the table: half of its last bit, and f [turns per position] in double
    precision: an exponent rounded by 2^-53 (ln theta times as much of f, the exponent being below 1), a power (2 halves of a
    step), 2 pi, a division by it and one by the scaling's factor."""
    return abs(position) * (2.0 ** -65 + (math.log(theta) + 5) * 2.0 ** -53 * float(f))


def turned(x, turns, gain, layout, transpose=False):
    """x [T, H, dk] in 64 bits, turned by the given turns [T, rot/2]; and how far a computation may be off"""
    pairs = turns.shape[1]
    ang = 2 * math.pi * (turns - np.round(turns)) * (-1 if transpose else 1)
    c, s = gain * np.cos(ang)[:, None], gain * np.sin(ang)[:, None]
    i = np.arange(pairs)
    a, b = (i, i + pairs) if layout == "halves" else (2 * i, 2 * i + 1)
    y, tol = x.copy(), np.zeros(x.shape)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    # A cosine or sine is off by the angle's rounding to 24 bits (up to pi 2^-24) and its last 2^-32 turn (0.03 of that), 2 units
    # of the function (4 halves of a step) and the product with the gain; a product and a sum round once each.
    off = (math.pi + 0.1 + 4 + 1 + 2) * F32 * gain * (np.abs(x[..., a]) + np.abs(x[..., b]))
    for k in (a, b):
        tol[..., k] = BF16 * np.abs(y[..., k]) + (1 + BF16) * off + 1e-37
    return y, tol


# ------------------------------------------------------------------------------------------ weights

def weights(q, k_rows, lse, sm_scale):
    """sum over a key head's query heads of exp(q . k sm_scale - lse) [Hkv, n], and how far it may be off.
    q [Hq, dk], k_rows [n, Hkv, dk], lse [Hq] (fp32 numbers)."""
    Hq, dk = q.shape
    n, Hkv, _ = k_rows.shape
    g = Hq // Hkv
    w, tol = np.zeros((Hkv, n)), np.zeros((Hkv, n))
    for h in range(Hq):
        if np.isneginf(lse[h]):
            continue
        k = k_rows[:, h // g]
        one = np.exp((k @ q[h]) * sm_scale - lse[h])
        d = (np.abs(k) @ np.abs(q[h])) * abs(sm_scale)
        # the exponent: dk products summed in fp32, then its own roundings; the exponential (2 units); the heads' sum
        ds = (dk + 4) * F32 * d + 4 * F32 * np.maximum(1.0, np.abs((k @ q[h]) * sm_scale - lse[h]))
        w[h // g] += one
        tol[h // g] += one * (np.expm1(ds) + (8 + g) * F32)
    return w, tol + 1e-37


# ------------------------------------------------------------------------------------------ the rows that stay

def evict(mass, born, total, k, sinks, recent):
    """positions that stay, as moves [(from, to)]: k of len(mass) rows by a plain sort"""
    n = len(mass)
    k = min(k, n)

    def rank(i):
        safe = born[i] < sinks or born[i] >= total - recent
        x = float(mass[i])
        return (0 if safe else 1, 0 if math.isnan(x) else 1, 0.0 if math.isnan(x) else -x, i)
    stay = set(sorted(range(n), key=rank)[:k])
    tails = [i for i in range(k, n) if i in stay]
    holes = [i for i in range(k) if i not in stay]
    assert len(tails) == len(holes)
    return list(zip(tails, holes))


# The forms that up_kv_evict's rule takes on a GPU of 152 SMs, by lists (requests and heads) and the tables' width: warps of a CTA,
# CTAs of a list, whether short lists go first by themselves, and whether the longest list's keys stay in shared memory.
FORMS = {                        # requests, heads, positions of the longest: warps, CTAs, apart, held
    "one_alone": ((1, 1, 4000), (16, 1, False, True)),
    "a_hundred_alone": ((50, 2, 20_000), (16, 1, False, True)),
    "many_alone": ((100, 2, 3000), (8, 1, False, True)),
    "pairs": ((30, 2, 16_000), (16, 2, False, True)),
    "pairs_of_32": ((30, 2, 40_000), (32, 2, False, True)),
    "pairs_of_many": ((160, 1, 20_000), (16, 2, False, True)),
    "fours": ((15, 2, 20_000), (16, 4, False, True)),
    "fours_of_32": ((15, 2, 50_000), (32, 4, False, True)),
    "fours_of_many": ((160, 1, 50_000), (16, 4, True, True)),
    "eights": ((4, 2, 40_000), (16, 8, False, True)),
    "eights_of_32": ((4, 2, 100_000), (32, 8, False, True)),
    "eights_of_many": ((160, 1, 70_000), (16, 8, True, True)),
    "eights_of_32_again": ((10, 1, 270_000), (32, 8, False, False)),
    "eights_of_many_again": ((160, 1, 270_000), (16, 8, True, False)),
    "sixteens": ((1, 1, 300_000), (32, 16, False, True)),
    "sixteens_again": ((1, 1, 530_000), (32, 16, False, False)),
}


def form_lengths(name):
    """a long list, some of half and of 7,000 positions where the form has as many, the others short"""
    (R, _, n), _ = FORMS[name]
    return ([n, n // 2 + 1, min(n, 7000)] + [50] * R)[:R]
