"""up_rope on the GPU against 64-bit rotations on the CPU: layouts, parts of the head, scalings, positions from negative to
far beyond 32 bits, strides, single tokens, in place, the gradient, counts on the device."""
import math
from decimal import localcontext

import numpy as np
import pytest
import torch

import long_context_prefill_varlen_gb300 as up
from long_context_prefill_varlen_gb300 import _build
from tests import evict_ref, kv_ref
from tests.test_gpu_debug_bounds import library
from tests.test_gpu_kvcache import _bits, _from_bits, _status

pytestmark = pytest.mark.gpu


def _turns(plan, positions):
    """turns [T, rot/2] within a turn, in whole numbers from the plan's table"""
    t = [[((int(p) * plan.turns[j]) % (1 << 64)) * 2.0 ** -64 for j in range(plan.rot // 2)] for p in positions]
    return np.array(t).reshape(len(positions), plan.rot // 2)


def _stream(rng, T, heads, dk):
    return _from_bits(kv_ref.bf16_bits((rng.standard_normal((T, heads, dk)) * 2.0 ** rng.integers(-4, 5, (T, heads, 1))).astype(np.float32)))


def _check(got, x, turns, plan, layout, transpose=False):
    y, tol = evict_ref.turned(kv_ref.bf16_value(_bits(x)), turns, plan.gain, layout, transpose)
    d = np.abs(kv_ref.bf16_value(_bits(got)) - y)
    assert (d <= tol).all(), float((d - tol).max())
    if x.shape[2] > plan.rot:
        assert np.array_equal(_bits(got)[..., plan.rot:], _bits(x)[..., plan.rot:])


def _call(plan, pos, q, k, **kw):
    st = _status()
    qo, ko = (None if x is None else torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in (q, k))
    up.up_rope(plan, pos, st, q=q, q_out=qo, k=k, k_out=ko, **kw)
    assert up.up_read_status(st) == 0
    return qo, ko


@pytest.mark.parametrize("T", [1, 2, 7, 300])
@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("Hq,Hkv,dk,rot", [(32, 8, 128, 128), (8, 8, 64, 64), (16, 2, 256, 64), (28, 4, 128, 16), (3, 1, 256, 256),
                                           (40, 8, 128, 96), (5, 5, 64, 16), (1, 1, 128, 112)])
def test_turning(Hq, Hkv, dk, rot, layout, T):
    rng = np.random.default_rng(T + rot)
    q, k = _stream(rng, T, Hq, dk), _stream(rng, T, Hkv, dk)
    pos = torch.from_numpy(rng.integers(0, 200_000, T)).cuda()
    plan = up.up_rope_plan(rot, theta=500000.0, layout=layout)
    turns = _turns(plan, pos.tolist())
    for transpose in (False, True):
        qo, ko = _call(plan, pos, q, k, transpose=transpose)
        _check(qo, q, turns, plan, layout, transpose)
        _check(ko, k, turns, plan, layout, transpose)


@pytest.mark.parametrize("scaling,factor,length", [("none", 1.0, 0), ("linear", 4.0, 0), ("bands", 8.0, 8192), ("ramp", 4.0, 32768),
                                                   ("ramp", 40.0, 4096)])
def test_scalings_against_the_formulas_in_radians(scaling, factor, length):
    """positions up to 10 million: 64-bit radians are still good to 2^-29 there"""
    rng = np.random.default_rng(1)
    T, dk, rot, theta = 200, 128, 128, 500000.0
    q = _stream(rng, T, 4, dk)
    pos = rng.integers(0, 10_000_000, T)
    pos[:4] = 0, 1, 9_999_999, 131_071
    plan = up.up_rope_plan(rot, theta=theta, scaling=scaling, factor=factor, original_len=length)
    f = evict_ref.frequencies(rot, theta, scaling, factor, length)
    qo, _ = _call(plan, torch.from_numpy(pos).cuda(), q, None)
    y, tol = evict_ref.turned(kv_ref.bf16_value(_bits(q)), pos[:, None] * f / (2 * math.pi), plan.gain, "halves")
    # 64-bit angles on either side: 10^7 radians times 2^-53, some twenty roundings and pow's growth by ln theta
    x = np.abs(kv_ref.bf16_value(_bits(q)))
    far = 40 * 13 * 1e7 * 2.0 ** -53 * plan.gain * (x + np.roll(x, 64, -1))
    assert (np.abs(kv_ref.bf16_value(_bits(qo)) - y) <= tol + far).all()
    assert np.array_equal(_bits(qo)[0], _bits(q)[0]) or plan.gain != 1.0           # position 0 turns nothing


def test_positions_of_any_size_and_sign():
    rng = np.random.default_rng(2)
    pos = [0, -1, 1, -5, (1 << 31) - 1, 1 << 31, -(1 << 31), (1 << 40) + 12345, -(1 << 40), (1 << 62) + 7, -(1 << 63), (1 << 63) - 1]
    q = _stream(rng, len(pos), 3, 128)
    for layout in ("halves", "pairs"):
        plan = up.up_rope_plan(128, theta=10000.0, layout=layout)
        qo, _ = _call(plan, torch.tensor(pos, device="cuda"), q, None)
        _check(qo, q, _turns(plan, pos), plan, layout)


@pytest.mark.parametrize("theta,factor", [(500000.0, 1), (10000.0, 1), (10000000.0, 8)])
def test_far_positions_against_angles_of_80_digits(theta, factor):
    """frequencies that are not the plan's own: off by what its table is, times the position"""
    pos = [100_000, 131_071, -10_000_019, (1 << 31) + 77, (1 << 33) + 5, -(1 << 37) + 1, (1 << 40) + 12345, -(1 << 44) - 3]
    rot = 128
    plan = up.up_rope_plan(rot, theta=theta, scaling="linear" if factor > 1 else "none", factor=factor)
    f = evict_ref.exact_turns(rot, theta, factor)
    with localcontext() as c:
        c.prec = 80
        turns = np.array([[float((p * x) % 1) for x in f] for p in pos])
    off = np.array([[evict_ref.turns_off(x, theta, p) for x in f] for p in pos])
    q = _stream(np.random.default_rng(9), len(pos), 3, 128)
    got, _ = _call(plan, torch.tensor(pos, device="cuda"), q, None)
    x = np.abs(kv_ref.bf16_value(_bits(q)))
    y, tol = evict_ref.turned(kv_ref.bf16_value(_bits(q)), turns, 1.0, "halves")
    far = 2 * math.pi * np.concatenate((off, off), 1)[:, None] * (x + np.roll(x, 64, -1))
    assert (np.abs(kv_ref.bf16_value(_bits(got)) - y) <= tol + (1 + kv_ref.BF16) * far).all()


def test_the_gradient_by_differences():
    """sum(w * rope(x)) differs by w . rope(e_i) along e_i, which transpose gives for all i at once (both exact but for their
    roundings to bf16)"""
    rng = np.random.default_rng(3)
    T, H, dk = 3, 2, 64
    w, pos = _stream(rng, T, H, dk), torch.tensor([5, 1234, 99_999], device="cuda")
    for layout in ("halves", "pairs"):
        plan = up.up_rope_plan(32, layout=layout, scaling="ramp", factor=4.0, original_len=4096)
        grad, _ = _call(plan, pos, w, None, transpose=True)
        grad, wv = kv_ref.bf16_value(_bits(grad)), kv_ref.bf16_value(_bits(w))
        for i in range(0, dk, 5):
            e = torch.zeros(T, H, dk, dtype=torch.bfloat16, device="cuda")
            e[:, :, i] = 1
            col, _ = _call(plan, pos, e, None)
            col = kv_ref.bf16_value(_bits(col))
            want = (wv * col).sum(-1)
            tol = 2 * kv_ref.BF16 * (np.abs(wv) * np.abs(col)).sum(-1) + 1e-5 * plan.gain * np.abs(wv).max(-1)
            assert (np.abs(grad[:, :, i] - want) <= tol).all()


def test_slices_of_a_fused_projection_each_side_alone_and_in_place():
    rng = np.random.default_rng(4)
    T, Hq, Hkv, dk = 65, 4, 2, 128
    qkv = _stream(rng, T, Hq + 2 * Hkv, dk)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    pos = torch.arange(T, device="cuda") * 3
    plan = up.up_rope_plan(64)
    qo, ko = _call(plan, pos, q, k)
    q1, k1 = _call(plan, pos, q.contiguous(), k.contiguous())
    assert torch.equal(qo, q1) and torch.equal(ko, k1)
    assert torch.equal(_call(plan, pos, q, None)[0], qo) and torch.equal(_call(plan, pos, None, k)[1], ko)
    st, same = _status(), qkv.clone()
    up.up_rope(plan, pos, st, q=same[:, :Hq], q_out=same[:, :Hq], k=same[:, Hq:Hq + Hkv], k_out=same[:, Hq:Hq + Hkv])
    assert up.up_read_status(st) == 0
    assert torch.equal(same[:, :Hq], qo) and torch.equal(same[:, Hq:Hq + Hkv], ko)
    assert torch.equal(same[:, Hq + Hkv:], qkv[:, Hq + Hkv:])
    # to rows of a wider buffer
    wide = torch.full((T, Hq + 3, dk), 5.0, dtype=torch.bfloat16, device="cuda")
    up.up_rope(plan, pos, st, q=q, q_out=wide[:, 1:1 + Hq])
    assert torch.equal(wide[:, 1:1 + Hq], qo) and (wide[:, 0] == 5.0).all() and (wide[:, 1 + Hq:] == 5.0).all()


def test_a_count_on_the_device():
    rng = np.random.default_rng(5)
    q, pos, plan = _stream(rng, 50, 4, 64), torch.arange(50, device="cuda"), up.up_rope_plan(64)
    whole, _ = _call(plan, pos, q, None)
    for n in (0, 1, 33, 50):
        got, _ = _call(plan, pos, q, None, num_tokens=torch.tensor([n], dtype=torch.int32, device="cuda"))
        assert torch.equal(got[:n], whole[:n]) and (got[n:] == 7.0).all()
    for n in (-1, 51):
        st, out = _status(), torch.full_like(q, 7.0)
        up.up_rope(plan, pos, st, q=q, q_out=out, num_tokens=torch.tensor([n], dtype=torch.int32, device="cuda"))
        assert up.up_read_status(st) == 6 and (out == 7.0).all()


def test_infinities_and_nan_stay_in_their_pairs():
    rng = np.random.default_rng(6)
    q, plan = _stream(rng, 4, 2, 128), up.up_rope_plan(128)
    clean, _ = _call(plan, torch.arange(4, device="cuda") + 9, q, None)
    q[0, 0, 3], q[1, 1, 70], q[2, 0, 127] = math.nan, math.inf, -math.inf
    got, _ = _call(plan, torch.arange(4, device="cuda") + 9, q, None)
    touched = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    for t, h, j in ((0, 0, 3), (1, 1, 70), (2, 0, 127)):
        touched[t, h, j], touched[t, h, (j + 64) % 128] = True, True
    assert torch.equal(got[~touched], clean[~touched]) and not torch.isfinite(got[touched]).any()


def test_no_tokens_a_stream_and_a_graph():
    rng = np.random.default_rng(7)
    plan = up.up_rope_plan(128, layout="pairs")
    empty = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    _call(plan, torch.empty(0, dtype=torch.int64, device="cuda"), empty, empty)
    q, pos = _stream(rng, 300, 4, 128), torch.arange(300, device="cuda")
    want, _ = _call(plan, pos, q, None)
    out, st, side = torch.zeros_like(q), _status(), torch.cuda.Stream()
    torch.cuda.synchronize()
    up.up_rope(plan, pos, st, q=q, q_out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        up.up_rope(plan, pos, st, q=q, q_out=out)
    new = _stream(rng, 300, 4, 128)
    want, _ = _call(plan, pos, new, None)
    q.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and up.up_read_status(st) == 0


def test_a_long_stream_is_that_of_its_pieces_and_the_bounds_checked_builds():
    rng = np.random.default_rng(8)
    T = 30_011
    x = torch.randn(T, 5, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    pos = torch.from_numpy(rng.integers(0, 1 << 20, T)).cuda()
    plan = up.up_rope_plan(96, layout="pairs")
    whole, _ = _call(plan, pos, x, None)
    for t in range(0, T, 4999):
        assert torch.equal(_call(plan, pos[t:t + 4999].contiguous(), x[t:t + 4999], None)[0], whole[t:t + 4999])
    with library(_build.build(debug_bounds=True)):
        assert torch.equal(_call(plan, pos, x, None)[0], whole)


def test_tensors_elsewhere_are_refused():
    plan, q = up.up_rope_plan(64), torch.zeros(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(AssertionError):
        up.up_rope(plan, torch.zeros(2, dtype=torch.int64), _status(), q=q, q_out=q)
    with pytest.raises(AssertionError):
        up.up_rope(plan, torch.zeros(2, dtype=torch.int32, device="cuda"), _status(), q=q, q_out=q)
    with pytest.raises(AssertionError):
        up.up_rope(plan, torch.zeros(2, dtype=torch.int64, device="cuda"), _status(), q=q)
    with pytest.raises(up.UpError):
        up.up_rope(up.up_rope_plan(128), torch.zeros(2, dtype=torch.int64, device="cuda"), _status(), q=q, q_out=q)


def test_streams_beyond_32_bits_of_offset():
    T, H, dk = 1_100_003, 16, 128                            # 4.5 GB in, as much out
    q, out = (torch.empty(T, H, dk, dtype=torch.bfloat16, device="cuda") for _ in "io")
    last = torch.randn(1000, H, dk, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(torch.bfloat16)
    q[-1000:] = last
    pos, plan, st = torch.arange(T, device="cuda"), up.up_rope_plan(64), _status()
    up.up_rope(plan, pos, st, q=q, q_out=out)
    assert up.up_read_status(st) == 0
    assert torch.equal(out[-1000:], _call(plan, pos[-1000:].contiguous(), last, None)[0])
