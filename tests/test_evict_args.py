"""What up_rope_plan, up_rope, up_kv_mass, up_kv_evict and up_kv_move refuse before anything is launched, the tables that
up_rope_plan makes, and the references of their GPU tests (no GPU needed)."""
import ctypes
import math
from decimal import Decimal

import numpy as np
import pytest
import torch

from tests import evict_ref
from tests.test_kvcache_args import A, BAD_CACHES, ODD, _cache, up  # noqa: F401
from tests.test_launch_host import lib  # noqa: F401


# ------------------------------------------------------------------------------------------ the plan

@pytest.mark.parametrize("scaling,factor,length", [("none", 1.0, 0), ("linear", 4.0, 0), ("bands", 8.0, 8192),
                                                   ("bands", 32.0, 100), ("ramp", 4.0, 32768), ("ramp", 40.0, 4096),
                                                   ("ramp", 2.0, 3)])
@pytest.mark.parametrize("rot,theta", [(128, 500000.0), (64, 10000000.0), (16, 10000.0), (256, 1.5)])
def test_the_plans_turns_are_the_formulas(up, rot, theta, scaling, factor, length):
    plan = up.up_rope_plan(rot, theta=theta, scaling=scaling, factor=factor, original_len=length)
    f = evict_ref.frequencies(rot, theta, scaling, factor, length)
    turns = np.array(list(plan.turns[:rot // 2]), dtype=np.float64) * 2.0 ** -64
    # a dozen roundings to 53 bits on either side (pow's argument grows its error by up to ln theta), and 2^-65 of the table's
    assert np.allclose(turns * 2 * math.pi, f, rtol=64 * 2.0 ** -53 * max(1.0, math.log(theta)), atol=2.0 ** -62)
    want = 1 + math.log(factor) / 10 if scaling == "ramp" else 1.0
    assert plan.gain == pytest.approx(want, rel=2.0 ** -23)
    assert (plan.rot, plan.layout) == (rot, 0) and not any(plan.turns[rot // 2:])


@pytest.mark.parametrize("rot,theta,factor", [(128, 500000.0, 1), (64, 10000000.0, 4), (16, 10000.0, 1), (256, 1.5, 8), (256, 1e300, 1)])
def test_the_plans_turns_to_their_last_bit(up, rot, theta, factor):
    plan = up.up_rope_plan(rot, theta=theta, scaling="linear" if factor > 1 else "none", factor=factor)
    for j, f in enumerate(evict_ref.exact_turns(rot, theta, factor)):
        assert abs(float(f - Decimal(plan.turns[j]) / (1 << 64))) <= evict_ref.turns_off(f, theta), j


def test_a_plans_own_turns_and_gain(up):
    a = up.up_rope_plan(64, scaling="bands", factor=8.0, original_len=8192)
    b = up.up_rope_plan(64, scaling="bands", factor=8.0, original_len=8192, low=1.0, high=4.0, gain=0.5)
    assert list(a.turns) == list(b.turns) and (a.gain, b.gain) == (1.0, 0.5)
    assert list(up.up_rope_plan(64, scaling="bands", factor=8.0, original_len=8192, high=8.0).turns) != list(a.turns)
    assert up.up_rope_plan(64, layout="pairs").layout == 1


def test_what_a_plan_refuses(up):
    for bad in (dict(theta=1.0), dict(theta=float("nan")), dict(theta=math.inf), dict(gain=-1.0), dict(gain=math.inf),
                dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("nan")),
                dict(scaling="bands", factor=8.0), dict(scaling="ramp", factor=8.0, original_len=-1.0),
                dict(scaling="bands", factor=8.0, original_len=100, low=4.0, high=4.0),
                dict(scaling="ramp", factor=8.0, original_len=100, low=0.0)):
        with pytest.raises(up.UpError) as e:
            up.up_rope_plan(64, **bad)
        assert e.value.code == up.UP_ERR_ARG, bad
    for rot in (0, -16, 8, 20, 272):
        with pytest.raises(up.UpError) as e:
            up.up_rope_plan(rot)
        assert e.value.code == up.UP_ERR_SHAPE, rot
    with pytest.raises(KeyError):
        up.up_rope_plan(64, layout="thirds")
    with pytest.raises(KeyError):
        up.up_rope_plan(64, scaling="dynamic")
    lib = up.load_library()
    plan = up.RopeTable()
    assert lib.up_rope_plan(64, 10000.0, 0, 0, 1.0, 0, 0, 0, 0, None) == up.UP_ERR_ARG
    assert lib.up_rope_plan(64, 10000.0, 2, 0, 1.0, 0, 0, 0, 0, ctypes.byref(plan)) == up.UP_ERR_ARG
    assert lib.up_rope_plan(64, 10000.0, 0, 4, 1.0, 0, 0, 0, 0, ctypes.byref(plan)) == up.UP_ERR_ARG


# ------------------------------------------------------------------------------------------ up_rope

def test_what_rope_refuses(up):
    lib, plan = up.load_library(), up.up_rope_plan(128)
    good = dict(plan=ctypes.byref(plan), q=A, q_stride=512, q_out=A, q_out_stride=512, Hq=4, k=A, k_stride=256, k_out=A,
                k_out_stride=256, Hkv=2, dk=128, positions=A, T=4, num=None, transpose=0, status=A, stream=None)

    def call(**kw):
        return lib.up_rope(*dict(good, **kw).values())
    for bad in (dict(plan=None), dict(status=None), dict(T=-1), dict(positions=None), dict(q=None), dict(q_out=None),
                dict(k=None), dict(k_out=None), dict(Hq=0), dict(Hkv=-1)):
        assert call(**bad) == up.UP_ERR_ARG, bad
    for bad in (dict(dk=96), dict(dk=64), dict(q=ODD), dict(q_out=ODD), dict(k=ODD), dict(k_out=ODD), dict(q_stride=513),
                dict(q_stride=504), dict(q_out_stride=504), dict(k_stride=248), dict(k_out_stride=260), dict(q_out_stride=520)):
        assert call(**bad) == up.UP_ERR_SHAPE, bad
    wrong = up.up_rope_plan(128)
    wrong.rot = 24
    assert call(plan=ctypes.byref(wrong)) == up.UP_ERR_SHAPE
    wrong.rot, wrong.layout = 128, 5
    assert call(plan=ctypes.byref(wrong)) == up.UP_ERR_ARG
    # nothing to do
    assert call(T=0, positions=None) == up.UP_OK
    assert call(q=None, q_out=None, k=None, k_out=None, positions=None) == up.UP_OK


# ------------------------------------------------------------------------------------------ the cache's calls

MASS = dict(q=A, q_stride=512, cache=None, table=A, seqused=A, lse=A, R=2, max_blocks=4, Hq=4, scale=0.1, counted=None,
            total=None, decay=1.0, mass=A, mass_out=A, born=A, status=A, stream=None)
EVICT = dict(mass=A, born=A, num_blocks=8, Hkv=2, B=16, table=A, seqused=4 * A, budget=2 * A, R=2, max_blocks=4, total=None,
             sinks=0, recent=0, moves=256 * A, max_moves=10, num_moves=A, new_len=3 * A, status=A, stream=None)
MOVE = dict(cache=None, table=A, R=2, max_blocks=4, moves=A, max_moves=10, num_moves=A, mass=None, born=None, status=A,
            stream=None)


@pytest.mark.parametrize("bad,code", BAD_CACHES, ids=lambda x: str(x))
def test_bad_caches_are_refused(up, bad, code):
    lib, want, c = up.load_library(), getattr(up, "UP_ERR_" + code), ctypes.byref(_cache(up, **bad))
    assert lib.up_kv_mass(*dict(MASS, cache=c).values()) == want
    assert lib.up_kv_move(*dict(MOVE, cache=c).values()) == want


def test_what_mass_refuses(up):
    lib, cache = up.load_library(), _cache(up)

    def call(**kw):
        return lib.up_kv_mass(*dict(dict(MASS, cache=ctypes.byref(cache)), **kw).values())
    for name in ("q", "cache", "table", "seqused", "lse", "mass", "mass_out", "born", "status"):
        assert call(**{name: None}) == up.UP_ERR_ARG, name
    for bad in (dict(R=0), dict(max_blocks=0), dict(Hq=0), dict(scale=math.nan), dict(scale=math.inf), dict(decay=-0.1),
                dict(decay=1.5), dict(decay=math.nan)):
        assert call(**bad) == up.UP_ERR_ARG, bad
    for bad in (dict(Hq=3), dict(q=ODD), dict(q_stride=511), dict(q_stride=504), dict(max_blocks=1 << 27)):
        assert call(**bad) == up.UP_ERR_SHAPE, bad


def test_what_evict_refuses(up):
    lib = up.load_library()

    def call(**kw):
        return lib.up_kv_evict(*dict(EVICT, **kw).values())
    for name in ("mass", "born", "table", "seqused", "budget", "moves", "num_moves", "new_len", "status"):
        assert call(**{name: None}) == up.UP_ERR_ARG, name
    for bad in (dict(R=0), dict(Hkv=0), dict(max_blocks=0), dict(B=0), dict(B=(1 << 20) + 1), dict(num_blocks=0),
                dict(num_blocks=1 << 31), dict(sinks=-1), dict(recent=-1), dict(max_moves=-1)):
        assert call(**bad) == up.UP_ERR_ARG, bad
    # an output that is, or runs into, what other CTAs still read (R = 2: 8 bytes of lengths, 16 of counts, 320 of moves)
    for bad in (dict(new_len=4 * A), dict(new_len=2 * A), dict(total=3 * A), dict(new_len=4 * A + 4), dict(new_len=4 * A - 4),
                dict(num_moves=2 * A - 12), dict(num_moves=4 * A + 4), dict(total=A + 12), dict(moves=4 * A - 312),
                dict(moves=2 * A), dict(total=256 * A + 316), dict(max_moves=1 << 62, budget=300 * A)):
        assert call(**bad) == up.UP_ERR_ARG, bad
    for bad in (dict(max_blocks=(1 << 26) + 1), dict(R=1 << 24), dict(moves=256 * A + 4)):
        assert call(**bad) == up.UP_ERR_SHAPE, bad


def test_what_move_refuses(up):
    lib, cache = up.load_library(), _cache(up)

    def call(**kw):
        return lib.up_kv_move(*dict(dict(MOVE, cache=ctypes.byref(cache)), **kw).values())
    for name in ("cache", "table", "moves", "num_moves", "status"):
        assert call(**{name: None}) == up.UP_ERR_ARG, name
    for bad in (dict(R=0), dict(max_blocks=0), dict(max_moves=-1)):
        assert call(**bad) == up.UP_ERR_ARG, bad
    for bad in (dict(max_blocks=(1 << 26) + 1), dict(R=1 << 24), dict(moves=256 * A + 4)):
        assert call(**bad) == up.UP_ERR_SHAPE, bad
    assert call(max_moves=0) == up.UP_OK and call(max_moves=0, moves=None) == up.UP_OK       # room for no move: none


def test_the_status_strings(up):
    for code in (11, 12):
        assert "unknown" not in up.up_status_string(code, True)


# ------------------------------------------------------------------------------------------ the references

def test_the_reference_turn_against_complex_numbers_and_its_transpose():
    rng = np.random.default_rng(1)
    x, turns = rng.standard_normal((7, 3, 64)), rng.uniform(-5, 5, (7, 16))
    for layout in ("halves", "pairs"):
        y, _ = evict_ref.turned(x, turns, 1.25, layout)
        a, b = (slice(0, 16), slice(16, 32)) if layout == "halves" else (slice(0, 32, 2), slice(1, 32, 2))
        z = (x[..., a] + 1j * x[..., b]) * 1.25 * np.exp(2j * math.pi * turns)[:, None]
        assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag) and np.array_equal(y[..., 32:], x[..., 32:])
        back, _ = evict_ref.turned(y, turns, 1 / 1.25, layout, transpose=True)
        assert np.allclose(back, x)
        # the gradient: of a sum with any weights, by differences
        w = rng.standard_normal(x.shape)
        grad, _ = evict_ref.turned(w, turns, 1.25, layout, transpose=True)
        e, at = 1e-6, (3, 1, 5)
        more, less = x.copy(), x.copy()
        more[at] += e
        less[at] -= e
        diff = [(evict_ref.turned(v, turns, 1.25, layout)[0] * w).sum() for v in (more, less)]
        assert np.isclose((diff[0] - diff[1]) / (2 * e), grad[at], atol=1e-7)


def test_the_reference_weights_add_up_to_the_heads():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((6, 64)), rng.standard_normal((50, 2, 64))
    s = torch.einsum("hd,nhd->hn", torch.from_numpy(q), torch.from_numpy(np.repeat(k, 3, 1))) * 0.125
    w, _ = evict_ref.weights(q, k, s.logsumexp(-1).numpy(), 0.125)
    assert np.allclose(w, s.softmax(-1).view(2, 3, 50).sum(1).numpy()) and np.allclose(w.sum(1), 3)


def test_the_reference_choice():
    mass = [5.0, 1.0, 1.0, 9.0, math.nan, 1.0, 7.0]
    born = [0, 1, 2, 3, 4, 5, 6]
    assert evict_ref.evict(mass, born, 7, 4, 0, 0) == [(4, 1), (6, 2)]           # 0, 3, 4 (NaN), 6
    assert evict_ref.evict(mass, born, 7, 5, 0, 0) == [(6, 2)]                   # and of the equal ones row 1
    assert evict_ref.evict(mass, born, 7, 3, 2, 2) == [(6, 2)]                   # rows 0, 1, 5, 6 protected, by mass, then position
    assert evict_ref.evict(mass, born, 7, 7, 0, 0) == [] and evict_ref.evict(mass, born, 7, 0, 3, 3) == []


# ------------------------------------------------------------------------------------------ launches

def _calls(m, up):
    """every kernel's form of the calls, on sizes that want them"""
    plan = up.RopeTable()
    assert m.up_rope_plan(64, 10000.0, 0, 0, 1.0, 0, 0, 0, 0, ctypes.byref(plan)) == 0
    for dk in (64, 128, 256):
        for layout in (0, 1):
            plan.layout = layout
            yield lambda dk=dk: m.up_rope(ctypes.byref(plan), A, 4 * dk, A, 4 * dk, 4, None, 0, None, 0, 0, dk, A, 100, None, 0, A, None)
        for e4m3 in (0, 1):
            for B in (16, 24):
                cache = up._KvCache(A, A, A, A, 8, 2 * B * dk, B * dk, dk, 2, B, dk, e4m3)
                for Hq in (4, 40):
                    yield lambda cache=cache, Hq=Hq, dk=dk: m.up_kv_mass(A, Hq * dk, ctypes.byref(cache), A, A, A, 2, 4, Hq, 0.1, None, None, 1.0,
                                                                         A, A, A, A, None)
            yield lambda cache=cache: m.up_kv_move(ctypes.byref(cache), A, 2, 4, A, 10, A, None, None, A, None)
    for R, max_blocks in ((1, 4), (1, 60000), (300, 4), (300, 2000), (60, 1500)):
        yield lambda R=R, max_blocks=max_blocks: m.up_kv_evict(A, A, 8, 2, 16, A, 4 * A, 2 * A, R, max_blocks, None, 0, 0, 256 * A, 10, A, 3 * A, A, None)


def test_every_call_launches_on_every_device_and_an_error_is_its_own(lib, up):
    for device in (40, 41):
        for call in _calls(lib, up):
            lib.fake_reset(device, 16)
            assert call() == 0 and lib.fake_launches() == 1
            lib.fake_fail(0, 1)
            assert call() == 4 and call() == 0


def test_a_list_goes_to_a_cluster_where_it_is_worth_one(lib, up):
    for R, max_blocks, cluster in ((1, 4, 1), (1, 60000, 16), (1, 16384, 8), (1, 300, 1), (300, 4, 1), (300, 2000, 2), (300, 60000, 8), (30, 1000, 2)):
        wide = (R, max_blocks) == (300, 60000)                   # short lists first, a CTA each
        lib.fake_reset(42, 16)
        assert lib.up_kv_evict(A, A, 8, 2, 16, A, 4 * A, 2 * A, R, max_blocks, None, 0, 0, 256 * A, 10, A, 3 * A, A, None) == 0
        assert [lib.fake_launch_cluster(i) for i in range(lib.fake_launches())] == [1] * wide + [cluster], (R, max_blocks)


@pytest.mark.parametrize("largest", [1, 2, 4, 8, 16])
def test_a_cluster_that_the_device_cannot_place_is_a_smaller_one(lib, up, largest):
    """(a partition of a GPU may have room for smaller clusters only)"""
    for R, max_blocks, cluster in ((1, 60000, 16), (1, 500, 8), (300, 2000, 2), (1, 4, 1), (300, 60000, 8)):
        for _ in range(2):
            lib.fake_reset(43 + largest, largest)
            assert lib.up_kv_evict(A, A, 8, 2, 16, A, 4 * A, 2 * A, R, max_blocks, None, 0, 0, 256 * A, 10, A, 3 * A, A, None) == 0
            n = lib.fake_launches()
            assert (n, lib.fake_launch_cluster(n - 1)) == (1 + ((R, max_blocks) == (300, 60000)), min(cluster, largest)), (R, max_blocks)


@pytest.mark.parametrize("name", evict_ref.FORMS)
def test_the_form_that_a_choice_takes(lib, up, name):
    """what the GPU tests of the forms take them for"""
    (R, Hkv, n), (warps, cluster, apart, held) = evict_ref.FORMS[name]
    max_blocks = -(-n // 16) + 2                                 # as _tables makes them
    lib.fake_reset(42, 16)
    assert lib.up_kv_evict(A, A, 8, Hkv, 16, A, 4 * A, 2 * A, R, max_blocks, None, 0, 0, 256 * A, 10, A, 3 * A, A, None) == 0
    launched = [(lib.fake_launch_name(i).decode(), lib.fake_launch_cluster(i)) for i in range(lib.fake_launches())]
    kind = f"evict_kernelILi{warps}ELi{1 if cluster == 1 else 16 if cluster == 16 else 8}E"
    assert len(launched) == 1 + apart and kind in launched[-1][0] and launched[-1][1] == cluster, launched
    assert not apart or ("evict_kernelILi8ELi1E" in launched[0][0] and launched[0][1] == 1)
    # a CTA's positions, in whole steps of its warps, and the keys that it holds
    ctas = min(cluster, -(-n // (16_384 if R * Hkv > 152 else 1024))) if n > (16_384 if R * Hkv > 152 else 6144) else 1
    assert (-(-n // (ctas * 128 * warps)) * 128 * warps <= 32_768) == held
