"""Decode attention where the weights and the values' sizes disagree (GPU): rows of zeros that take nearly all the weight,
in ordinary and in tiny company, pages out of range among small values, and columns in which the heaviest row is zero.

Tolerances are those of kv_ref.decode, relative to sum p|v| of each column: no other row's size enters them."""
import numpy as np
import pytest
import torch

from tests import kv_ref
from tests.test_gpu_kvcache import Pages, _bits, _check, _from_bits, _run_decode, _write

pytestmark = pytest.mark.gpu


def _case(seed, n, heavy, nats, size, e4m3, zero, Hq=4, Hkv=1, dk=64, B=16):
    """One request of n rows whose values are about `size`; rows `heavy` score `nats` above the rest's mean for every
    query head, and zero(values, rows) makes what is to be zero in them."""
    rng = np.random.default_rng(seed)
    nb = -(-n // B) + 1
    c = Pages(nb, Hkv, B, dk, e4m3)
    base = rng.choice([-1.0, 1.0], dk)
    q = base + 0.1 * rng.standard_normal((1, Hq, dk))
    k = 0.3 * rng.standard_normal((n, Hkv, dk))
    k[heavy] += base * nats * dk ** -0.5
    v = size * rng.standard_normal((n, Hkv, dk))
    zero(v, heavy)
    qb, kb, vb = (kv_ref.bf16_bits(x.astype(np.float32)) for x in (q, k, v))
    assert _write(c, kb, vb, np.arange(n)) == 0
    return c, np.arange(nb, dtype=np.int32)[None, :], qb


def _rows_of_zeros(v, rows):
    v[rows] = 0.0


def _every_other_column(v, rows):
    v[rows, ..., ::2] = 0.0


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("nats", [0, 5, 14, 40])
@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-5, 1e6])
@pytest.mark.parametrize("n,heavy", [(16, [0]), (200, [0]), (200, [3, 77, 199]), (5000, [0]), (5000, [4000])])
def test_rows_of_zeros_take_weight_and_nothing_else(n, heavy, size, nats, e4m3):
    c, table, qb = _case(n + nats, n, heavy, nats, size, e4m3, _rows_of_zeros)
    _check(c, table, [np.arange(n)], qb, [n])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,dk,B", [(8, 2, 128, 24), (9, 1, 64, 100), (6, 3, 256, 1), (32, 2, 128, 64)])
def test_rows_of_zeros_over_head_layouts_and_pages(Hq, Hkv, dk, B, e4m3):
    n, heavy = 333, [0, 65, 130, 332]
    c, table, qb = _case(dk + B, n, heavy, 10, 1e-4, e4m3, _rows_of_zeros, Hq, Hkv, dk, B)
    _check(c, table, [np.arange(n)], qb, [n])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("value", [0x80, 0x00], ids=["minus", "plus"])
def test_rows_of_zeros_of_either_sign_and_any_scale(value, e4m3):
    """a cache that another program filled: zeros of either sign under whatever scale"""
    n = 100
    c, table, qb = _case(9, n, [5, 50], 12, 1e-3, e4m3, _rows_of_zeros)
    for row, scale in ((5, 200), (50, 127)):
        if e4m3:
            c.v.view(torch.uint8)[row // 16, :, row % 16] = value
            c.vs[row // 16, :, row % 16] = scale
        else:
            c.v.view(torch.int16)[row // 16, :, row % 16] = -32768 if value else 0
    _check(c, table, [np.arange(n)], qb, [n])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("nats", [2, 6, 10])
@pytest.mark.parametrize("n", [100, 1000])
def test_columns_in_which_the_heaviest_row_is_zero(n, nats, e4m3):
    """the other rows' weights, down to about 2^-15 of the heaviest one's, keep the precision they would have alone"""
    c, table, qb = _case(n + nats, n, [7], nats, 1.0, e4m3, _every_other_column)
    _check(c, table, [np.arange(n)], qb, [n])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("size", [1.0, 1e-5])
def test_a_page_out_of_range_counts_as_zeros_among_small_values(size, e4m3):
    n = 100
    c, table, qb = _case(3, n, [], 0, size, e4m3, _rows_of_zeros)
    table[0, 2] = -1
    status, out, _ = _run_decode(c, table, [n], _from_bits(qb))
    assert status == 9
    k, v = c.rows("k", np.arange(n)), c.rows("v", np.arange(n))
    k[32:48] = v[32:48] = 0
    o, _, tol, _ = kv_ref.decode(kv_ref.bf16_value(qb), [k], [v], 64 ** -0.5)
    assert (np.abs(kv_ref.bf16_value(_bits(out)) - o) <= tol).all()


@pytest.mark.parametrize("nats", [13, 16, 20, 30])
@pytest.mark.parametrize("n", [16, 100, 1000])
def test_the_last_bits_of_light_rows_beside_a_heavy_one(n, nats):
    """An e4m3 cache's weights are f16 numbers whose reference lies 2^-7 below the largest weight * value scale W: to half a
    step of f16's subnormals, 2^-25, an error is 2^-32 W and a code's size that of the row's number."""
    c, table, qb = _case(n + nats, n, [7], nats, 1.0, True, _every_other_column)
    status, out, _ = _run_decode(c, table, [n], _from_bits(qb))
    assert status == 0
    rows = np.arange(n)
    k, v, q = c.rows("k", rows), c.rows("v", rows), kv_ref.bf16_value(qb)
    o, _, tol, _ = kv_ref.decode(q, [k], [v], 64 ** -0.5)
    scale = 2.0 ** (c.vs.cpu().numpy()[rows // 16, 0, rows % 16].astype(float) - 127)
    s = q[0] @ k[:, 0].T * 64 ** -0.5
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    largest = (p * scale).max(1)[:, None]                      # W of each head
    tol[0] += (1 + kv_ref.BF16) * 2.0 ** -32 * largest * (np.abs(v[:, 0]) / scale[:, None]).sum(0)
    assert (np.abs(kv_ref.bf16_value(_bits(out)) - o) <= tol).all()
