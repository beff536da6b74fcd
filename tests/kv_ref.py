"""The paged cache and its decode attention in 64 bits on the CPU (test infrastructure), and the tolerances.

A cache here is numpy arrays [num_blocks, Hkv, B, dk]; e4m3 codes are uint8 with one scale byte per row.
"""
from __future__ import annotations

import numpy as np

BF16, F16, F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24     # half a step of a rounding, relative to the value


def bf16_value(bits):
    return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_bits(x):
    """nearest bf16 bit pattern (ties to even) of finite numbers that fp32 holds exactly"""
    b = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def _e4m3_table():
    v = np.empty(256)
    for c in range(256):
        s, e, m = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        v[c] = s * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    v[0x7F] = v[0xFF] = np.nan
    return v


E4M3 = _e4m3_table()


def e4m3_codes(x):
    """nearest e4m3 code of |x| <= 448 by search over the format's values, ties to the even code; NaN, inf -> 0x7f
    with x's sign or without"""
    x = np.asarray(x, dtype=np.float64)
    pos = E4M3[:0x7F]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(pos, a), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(pos[hi] == a, hi, c)
    c = c + np.where(np.signbit(x), 128, 0)
    return np.where(np.isfinite(x), c, 0x7F).astype(np.uint8)


def quantise(x):
    """codes and scale bytes of rows x [..., dk] (64-bit values of bf16 numbers)"""
    a = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    b = np.full(a.shape, 127, dtype=np.int64)
    it = np.nditer(a, flags=["multi_index"])
    for v in it:
        if v > 0:
            e = -126
            f = int(np.floor(np.log2(float(v)))) - 10
            e = max(e, f)
            while float(v) > 448.0 * 2.0 ** e:
                e += 1
            b[it.multi_index] = e + 127
    with np.errstate(invalid="ignore"):
        return e4m3_codes(x * 2.0 ** (127.0 - b)[..., None]), b.astype(np.uint8)


def dequantise(codes, b):
    return E4M3[codes] * 2.0 ** (b.astype(np.float64) - 127)[..., None]


def attend(q, k, v, sm_scale):
    """one query head over its keys [n, dk], values [n, dk]: output, natural log of the sum, and the two
    sums that the tolerances need (of p|v| per column, and the largest sum of |q k|)"""
    if len(k) == 0:
        return np.zeros(len(q)), -np.inf, np.zeros(len(q)), 0.0
    s = (k @ q) * sm_scale
    m = s.max()
    p = np.exp(s - m)
    lse = m + np.log(p.sum())
    p = p / p.sum()
    return p @ v, lse, p @ np.abs(v), float((np.abs(k) @ np.abs(q)).max() * abs(sm_scale))


def decode(q, k_rows, v_rows, sm_scale):
    """q [R, Hq, dk]; k_rows[r], v_rows[r] [n_r, Hkv, dk] the attended rows.  out, lse and their tolerances."""
    R, Hq, dk = q.shape
    out, lse = np.zeros((R, Hq, dk)), np.zeros((R, Hq))
    tol_o, tol_l = np.zeros((R, Hq, dk)), np.zeros((R, Hq))
    for r in range(R):
        g = Hq // k_rows[r].shape[1]
        for h in range(Hq):
            n = len(k_rows[r])
            o, l, a, d = attend(q[r, h], k_rows[r][:, h // g], v_rows[r][:, h // g], sm_scale)
            out[r, h], lse[r, h] = o, l
            # a logit: dk products summed in fp32, the scale and the base change; its error moves p by twice that
            # much relative to p.  A sum of n terms in fp32, the exponential (2 units) and the chunks' weights.
            ds = (dk + 4) * F32 * d + 4 * F32 * max(1.0, d)
            rel = 2 * ds + (n + 16) * F32
            # one rounding of the weights to f16 (or two bf16 parts, which is finer), one of the result to bf16
            tol_o[r, h] = BF16 * np.abs(o) + (1 + BF16) * (rel + F16) * a + 1e-37
            tol_l[r, h] = rel + 4 * F32 * (abs(l) if np.isfinite(l) else 0.0)
    return out, lse, tol_o, tol_l
