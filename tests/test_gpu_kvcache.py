"""The paged key-value cache on the GPU: up_kv_write, up_kv_read and up_paged_decode against 64-bit CPU
implementations, over types, head layouts, page sizes, lengths from none to long, windows, orders of the
cache's axes, and whatever lies in rows that nobody attends to."""
import numpy as np
import pytest
import torch

import long_context_prefill_varlen_gb300 as up
from long_context_prefill_varlen_gb300 import _build
from tests import kv_ref
from tests.test_gpu_debug_bounds import library

pytestmark = pytest.mark.gpu


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _as_bits(t):
    return t.view(torch.int16)


def _from_bits(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def _random_rows(rng, T, Hkv, dk):
    """bf16 bits: rows of very different size, some zeros, subnormals, a row of zeros and the largest numbers"""
    x = rng.standard_normal((T, Hkv, dk)) * 2.0 ** rng.integers(-20, 20, (T, Hkv, 1))
    bits = kv_ref.bf16_bits(x.astype(np.float32))
    if T > 8:
        bits[1] = 0
        bits[2, :, ::3] = 0x8000
        bits[3] = rng.integers(0, 0x80, (Hkv, dk))               # subnormal rows
        bits[4, :, 0] = 0x7F7F                                   # the largest finite number
        bits[5] = rng.integers(0x4000, 0x4080, (Hkv, dk))        # maxima around 1.75 * 2^k
        bits[6, :, 1:] = 0
    return bits


class Pages:
    """A cache in the named order of its axes, its tensors filled with NaN everywhere."""

    def __init__(self, num_blocks, Hkv, B, dk, e4m3, order="hnd"):
        dt = torch.uint8 if e4m3 else torch.int16
        fill = 0x7F if e4m3 else 0x7FC0

        def one():
            if order == "hnd":
                t = torch.full((num_blocks, Hkv, B, dk), fill, dtype=dt, device="cuda")
            elif order == "nhd":
                t = torch.full((num_blocks, B, Hkv, dk), fill, dtype=dt, device="cuda").transpose(1, 2)
            else:                                                # rows with room after them, pages last
                t = torch.full((Hkv, B, num_blocks, dk + 32), fill, dtype=dt, device="cuda").permute(2, 0, 1, 3)[..., :dk]
            return t.view(torch.float8_e4m3fn if e4m3 else torch.bfloat16)
        self.e4m3, self.B, self.Hkv, self.dk, self.num_blocks = e4m3, B, Hkv, dk, num_blocks
        self.k, self.v = one(), one()
        rows = (num_blocks, Hkv, up.up_kv_scale_row(B))
        self.ks, self.vs = (torch.full(rows, 255, dtype=torch.uint8, device="cuda") if e4m3 else None for _ in "kv")

    def scales(self):
        return dict(k_scale=self.ks, v_scale=self.vs) if self.e4m3 else {}

    def rows(self, name, slots):
        """64-bit values of the rows of `slots` [n, Hkv, dk]"""
        t = self.k if name == "k" else self.v
        page, off = np.asarray(slots) // self.B, np.asarray(slots) % self.B
        if self.e4m3:
            s = (self.ks if name == "k" else self.vs).cpu().numpy()
            return kv_ref.dequantise(t.view(torch.uint8).cpu().numpy()[page, :, off], s[page, :, off])
        return kv_ref.bf16_value(_bits(t)[page, :, off])


def _write(c, kb, vb, slots, **kw):
    st = _status()
    up.up_kv_write(None if kb is None else _from_bits(kb), None if vb is None else _from_bits(vb),
                   torch.as_tensor(np.asarray(slots)).long().cuda(), c.k, c.v, st, **c.scales(), **kw)
    return up.up_read_status(st)


ORDERS = ["hnd", "nhd", "last"]


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("Hkv,dk,B", [(8, 128, 16), (1, 64, 1), (3, 256, 24), (2, 64, 100), (5, 128, 256)])
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 2, 37, 700])
def test_write_and_read_are_exact(T, e4m3, Hkv, dk, B, order):
    rng = np.random.default_rng(T + 7 * dk + B)
    nb = -(-T // B) + 3
    c = Pages(nb, Hkv, B, dk, e4m3, order)
    slots = rng.permutation(nb * B)[:T].astype(np.int64)
    if T > 2:
        slots[T // 2] = -1
    kb, vb = _random_rows(rng, T, Hkv, dk), _random_rows(rng, T, Hkv, dk)
    assert _write(c, kb, vb, slots) == 0
    live = slots >= 0
    page, off = slots[live] // B, slots[live] % B
    untouched = np.ones((nb, B), dtype=bool)
    untouched[page, off] = False
    for t, s, bits in ((c.k, c.ks, kb), (c.v, c.vs, vb)):
        if e4m3:
            codes, b = kv_ref.quantise(kv_ref.bf16_value(bits[live]))
            got = t.view(torch.uint8).cpu().numpy()
            assert np.array_equal(got[page, :, off], codes)
            assert np.array_equal(s.cpu().numpy()[page, :, off], b)
            assert (got.transpose(0, 2, 1, 3)[untouched] == 0x7F).all()
            s_rows = s.cpu().numpy().transpose(0, 2, 1)
            assert (s_rows[:, :B][untouched] == 255).all() and (s_rows[:, B:] == 255).all()
        else:
            got = _bits(t)
            assert np.array_equal(got[page, :, off], bits[live])
            assert (got.transpose(0, 2, 1, 3)[untouched] == 0x7FC0).all()
    # read it back, in another order, -1 giving zeros
    perm = rng.permutation(T)
    st = _status()
    k, v = (torch.full((T, Hkv, dk), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    up.up_kv_read(c.k, c.v, torch.from_numpy(slots[perm]).cuda(), k, v, st, **c.scales())
    assert up.up_read_status(st) == 0
    for got, bits in ((k, kb), (v, vb)):
        want = bits.copy()
        if e4m3:
            codes, b = kv_ref.quantise(kv_ref.bf16_value(bits))
            with np.errstate(over="ignore"):                     # 248 * 2^120 and more read back as infinity
                want = kv_ref.bf16_bits(kv_ref.dequantise(codes, b).astype(np.float32))
        want[~live] = 0
        assert np.array_equal(_bits(got), want[perm])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hkv,dk", [(8, 64), (4, 128), (2, 256)])
def test_a_long_read_is_that_of_its_pieces(Hkv, dk, e4m3):
    """more tokens than the CTAs of one wave take at once; both sides, and each alone"""
    rng = np.random.default_rng(dk)
    T, B = 50021, 16
    nb = -(-T // B)
    c = Pages(nb, Hkv, B, dk, e4m3)
    slots = rng.permutation(nb * B)[:T].astype(np.int64)
    slots[rng.integers(0, T, 50)] = -1
    kb, vb = (kv_ref.bf16_bits(rng.standard_normal((T, Hkv, dk)).astype(np.float32)) for _ in "kv")
    assert _write(c, kb, vb, slots) == 0
    sl = torch.from_numpy(slots).cuda()
    st = _status()
    new = lambda n: torch.full((n, Hkv, dk), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v, k1, v1 = new(T), new(T), new(T), new(T)
    up.up_kv_read(c.k, c.v, sl, k, v, st, **c.scales())
    up.up_kv_read(c.k, c.v, sl, k1, None, st, **c.scales())
    up.up_kv_read(c.k, c.v, sl, None, v1, st, **c.scales())
    assert torch.equal(_as_bits(k), _as_bits(k1)) and torch.equal(_as_bits(v), _as_bits(v1))
    for t0 in range(0, T, 7000):
        n = min(7000, T - t0)
        kk, vv = new(n), new(n)
        up.up_kv_read(c.k, c.v, sl[t0:t0 + n], kk, vv, st, **c.scales())
        assert torch.equal(_as_bits(kk), _as_bits(k[t0:t0 + n])) and torch.equal(_as_bits(vv), _as_bits(v[t0:t0 + n]))
    assert up.up_read_status(st) == 0
    if not e4m3:
        live = slots >= 0
        assert np.array_equal(_bits(k)[live], kb[live]) and np.array_equal(_bits(v)[live], vb[live])
        assert (_bits(k)[~live] == 0).all()


def test_nonfinite_numbers_become_nan_codes_and_leave_the_rest_of_the_row():
    rng = np.random.default_rng(5)
    bits = kv_ref.bf16_bits(rng.standard_normal((6, 2, 64)).astype(np.float32))
    bits[0, 0, 3], bits[1, 1, 60], bits[2, 0, 0] = 0x7F80, 0xFF80, 0x7FC1
    bits[3] = 0x7FC0
    bits[4, 1, :] = 0xFF80
    c = Pages(2, 2, 16, 64, True)
    slots = np.arange(6)
    assert _write(c, bits, bits, slots) == 0
    x = kv_ref.bf16_value(bits)
    codes, b = kv_ref.quantise(x)
    got = c.k.view(torch.uint8).cpu().numpy()[0, :, :6].transpose(1, 0, 2)
    assert np.array_equal(c.ks.cpu().numpy()[0, :, :6].T, b)
    bad = ~np.isfinite(x)
    assert np.array_equal(got[~bad], codes[~bad]) and ((got[bad] & 0x7F) == 0x7F).all()
    st = _status()
    k = torch.zeros(6, 2, 64, dtype=torch.bfloat16, device="cuda")
    up.up_kv_read(c.k, c.v, torch.from_numpy(slots).cuda(), k, None, st, **c.scales())
    assert up.up_read_status(st) == 0
    assert np.array_equal(np.isnan(kv_ref.bf16_value(_bits(k))), bad)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_write_takes_slices_of_a_fused_projection_one_side_and_a_device_count(e4m3):
    rng = np.random.default_rng(9)
    T, Hq, Hkv, dk, B = 50, 4, 2, 128, 16
    qkv = _from_bits(_random_rows(rng, T, Hq + 2 * Hkv, dk))
    k, v = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    slots = torch.from_numpy(rng.permutation(8 * B)[:T]).cuda()
    a, b = Pages(8, Hkv, B, dk, e4m3), Pages(8, Hkv, B, dk, e4m3)
    st, n = _status(), torch.tensor([33], dtype=torch.int32, device="cuda")
    up.up_kv_write(k, v, slots, a.k, a.v, st, **a.scales(), num_tokens=n)
    up.up_kv_write(k[:33].contiguous(), None, slots[:33].contiguous(), b.k, b.v, st, **b.scales())
    up.up_kv_write(None, v[:33].contiguous(), slots[:33].contiguous(), b.k, b.v, st, **b.scales())
    assert up.up_read_status(st) == 0
    for x, y in ((a.k, b.k), (a.v, b.v)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    if e4m3:
        assert torch.equal(a.ks, b.ks) and torch.equal(a.vs, b.vs)
    got = torch.full((T, Hkv, dk), 3.0, dtype=torch.bfloat16, device="cuda")
    up.up_kv_read(a.k, a.v, slots, None, got, st, **a.scales(), num_tokens=n)
    assert up.up_read_status(st) == 0
    assert (got[33:] == 3.0).all() and not (got[:33] == 3.0).all()
    # a count that does not fit writes nothing and says so
    before = a.k.view(torch.uint8).clone()
    up.up_kv_write(v, k, slots, a.k, a.v, st, **a.scales(), num_tokens=torch.tensor([T + 1], dtype=torch.int32, device="cuda"))
    assert up.up_read_status(st) == 6 and torch.equal(a.k.view(torch.uint8), before)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [-2, 64, 1 << 40, -(1 << 40)])
def test_a_slot_outside_the_cache_is_skipped_and_reported(bad, e4m3):
    rng = np.random.default_rng(3)
    c = Pages(4, 2, 16, 64, e4m3)
    bits = _random_rows(rng, 12, 2, 64)
    slots = np.arange(12)
    slots[7] = bad
    assert _write(c, bits, bits, slots) == 8
    good = np.delete(np.arange(12), 7)
    x = kv_ref.bf16_value(bits)
    want = (kv_ref.dequantise(*kv_ref.quantise(x)) if e4m3 else x)
    assert np.array_equal(c.rows("k", good), want[good]) and np.isnan(c.rows("k", [7])).all()
    st = _status()
    k = torch.full((12, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    up.up_kv_read(c.k, c.v, torch.from_numpy(slots).cuda(), k, None, st, **c.scales())
    assert up.up_read_status(st) == 8
    with np.errstate(over="ignore"):
        want[7] = 0
        assert np.array_equal(_bits(k), kv_ref.bf16_bits(want.astype(np.float32)))


# ------------------------------------------------------------------------------------------ decode

def _decode_case(seed, Hq, Hkv, dk, B, lens, e4m3, window=0, order="hnd", scale=1.0, extra_cols=2):
    """A cache whose attended rows are written by up_kv_write and whose every other row is NaN."""
    rng = np.random.default_rng(seed)
    R = len(lens)
    need = [-(-n // B) for n in lens]
    nb = sum(need) + 3
    c = Pages(nb, Hkv, B, dk, e4m3, order)
    cols = max(1, max(need)) + extra_cols
    table = rng.integers(-(1 << 31), 1 << 31, (R, cols)).astype(np.int32)      # entries nobody uses
    perm, at, slots, rows = rng.permutation(nb), 0, [], []
    for r, n in enumerate(lens):
        table[r, :need[r]] = perm[at:at + need[r]]
        at += need[r]
        lo = max(0, n - window) if window else 0
        table[r, :lo // B] = -7                                                # pages before the window: not read
        pos = np.arange(lo, n)
        s = table[r, pos // B].astype(np.int64) * B + pos % B
        rows.append(s)
        slots.append(s)
    slots = np.concatenate(slots)
    x = rng.standard_normal((2, len(slots), Hkv, dk)) * scale
    x[1] *= 2.0 ** rng.integers(-6, 7, (len(slots), Hkv, 1))
    q = rng.standard_normal((R, Hq, dk))
    bits = kv_ref.bf16_bits(x.astype(np.float32))
    if len(slots):
        assert _write(c, bits[0], bits[1], slots) == 0
    qb = kv_ref.bf16_bits(q.astype(np.float32))
    return c, table, rows, qb


def _run_decode(c, table, lens, q, window=0, sm_scale=None, with_lse=True):
    R, Hq, dk = q.shape
    st = _status()
    out = torch.full((R, Hq, dk), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((R, Hq), 9.0, device="cuda") if with_lse else None
    nbytes = up.up_paged_decode_workspace_bytes(R, Hq, c.Hkv, dk, c.B, table.shape[1], window)
    assert nbytes > 0
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")          # NaN in every fp32 of it
    up.up_paged_decode(q, c.k, c.v, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                       out, ws, st, **c.scales(), lse=lse, window=window, sm_scale=sm_scale)
    return up.up_read_status(st), out, lse


def _check(c, table, rows, qb, lens, window=0, sm_scale=None):
    """Against the reference, as a call of these requests (one launch, where every chunk can have a CTA at once) and
    as one of 40 times as many (persistent CTAs and a join)."""
    status, out, lse = _run_decode(c, table, lens, _from_bits(qb), window, sm_scale)
    assert status == 0
    launches = up.up_kernel_launches()
    status, many, many_lse = _run_decode(c, np.tile(table, (40, 1)), tuple(lens) * 40, _from_bits(np.tile(qb, (40, 1, 1))),
                                         window, sm_scale)
    assert status == 0 and (len(lens) * 40 * c.Hkv < 500 or up.up_kernel_launches() - launches == 2)
    assert torch.equal(many, out.repeat(40, 1, 1)) and torch.equal(many_lse, lse.repeat(40, 1))
    k, v = [c.rows("k", s) for s in rows], [c.rows("v", s) for s in rows]
    scale = qb.shape[2] ** -0.5 if sm_scale is None else sm_scale
    o, l, to, tl = kv_ref.decode(kv_ref.bf16_value(qb), k, v, scale)
    got = kv_ref.bf16_value(_bits(out))
    assert np.isfinite(got).all()
    assert (np.abs(got - o) <= to).all(), float(np.max(np.abs(got - o) - to))
    got_l = lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(l)
    assert np.array_equal(np.isneginf(got_l), empty)
    assert (np.abs(got_l[~empty] - l[~empty]) <= tl[~empty]).all()
    for r, n in enumerate(lens):
        if n == 0:
            assert (got[r] == 0).all()
    return out, lse


LENS = (0, 1, 15, 16, 17, 63, 64, 65, 130, 257, 1000)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("B", [1, 8, 16, 24, 64, 100, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,dk", [(8, 2, 128), (2, 2, 64), (16, 2, 256)])
def test_decode_over_lengths_and_page_sizes(Hq, Hkv, dk, B, e4m3):
    c, table, rows, q = _decode_case(B + dk, Hq, Hkv, dk, B, LENS, e4m3)
    _check(c, table, rows, q, LENS)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("group,Hkv", [(1, 3), (2, 8), (3, 1), (5, 2), (7, 1), (9, 1), (16, 1), (17, 2), (32, 1)])
def test_decode_over_head_groups(group, Hkv, dk, e4m3):
    lens = (300, 0, 77)
    c, table, rows, q = _decode_case(group + dk, group * Hkv, Hkv, dk, 16, lens, e4m3)
    _check(c, table, rows, q, lens)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("B", [16, 24, 100])
@pytest.mark.parametrize("window", [1, 16, 100, 128, 700, 5000])
def test_decode_window(window, B, e4m3):
    lens = LENS + (3001,)
    c, table, rows, q = _decode_case(window + B, 4, 2, 128, B, lens, e4m3, window=window)
    _check(c, table, rows, q, lens, window=window)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("order", ORDERS)
def test_decode_axis_orders(order, e4m3):
    lens = (500, 33, 0, 129)
    c, table, rows, q = _decode_case(4, 8, 2, 128, 16, lens, e4m3, order=order)
    _check(c, table, rows, q, lens)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,dk,n", [(32, 8, 128, 9001), (4, 1, 64, 40000), (16, 8, 256, 6000)])
def test_decode_long_requests(Hq, Hkv, dk, n, e4m3):
    lens = (n, 5, n // 3)
    c, table, rows, q = _decode_case(n, Hq, Hkv, dk, 32, lens, e4m3)
    _check(c, table, rows, q, lens)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [8.0, 1e-4])
def test_decode_peaked_and_flat_scores(scale, e4m3):
    """logits of several hundred (one key takes all the weight) and next to none"""
    lens = (400, 64, 1)
    c, table, rows, q = _decode_case(77, 8, 2, 128, 16, lens, e4m3, scale=scale)
    _check(c, table, rows, q, lens, sm_scale=1.0)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_decode_values_of_very_different_size(e4m3):
    """a token that takes nearly all the weight has values 2^-100 of the others' (an attention sink's)"""
    rng = np.random.default_rng(8)
    n, Hq, Hkv, dk, B = 200, 4, 1, 64, 16
    c = Pages(20, Hkv, B, dk, e4m3)
    table = np.arange(20, dtype=np.int32)[None, :]
    q = rng.standard_normal((1, Hq, dk))
    k = rng.standard_normal((n, Hkv, dk)) * 0.5
    k[3, 0] = q[0].mean(0) * 12.0
    v = rng.standard_normal((n, Hkv, dk))
    v[3] *= 2.0 ** -100
    v[7] *= 2.0 ** 30
    v[9] = 0.0
    qb, kb, vb = (kv_ref.bf16_bits(x.astype(np.float32)) for x in (q, k, v))
    assert _write(c, kb, vb, np.arange(n)) == 0
    _check(c, table, [np.arange(n)], qb, [n])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,dk,B,R", [(8, 2, 128, 16, 40), (9, 1, 64, 24, 70), (4, 4, 256, 64, 33), (34, 2, 128, 16, 6)])
def test_decode_does_not_depend_on_the_tables_width(Hq, Hkv, dk, B, R, e4m3):
    """many requests, most of them short, in a narrow table and in one that could hold far more"""
    rng = np.random.default_rng(R)
    lens = tuple(int(x) for x in np.concatenate([[0, 1, 0, 2500, 0], rng.integers(0, 700, max(0, R - 6)), [0]]))
    c, table, rows, qb = _decode_case(R, Hq, Hkv, dk, B, lens, e4m3)
    out, lse = _check(c, table, rows, qb, lens)
    wide = np.full((R, table.shape[1] + 1280 * 1024 // (B * R * Hkv)), -1, dtype=np.int32)
    wide[:, :table.shape[1]] = table
    status, out2, lse2 = _run_decode(c, wide, lens, _from_bits(qb))
    assert status == 0
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    status, out3, lse3 = _run_decode(c, wide, (0,) * R, _from_bits(qb))
    assert status == 0 and (out3 == 0).all() and torch.isneginf(lse3).all()
    status, out4, _ = _run_decode(c, wide, lens[:-1] + (-5,), _from_bits(qb))
    assert status == 10 and torch.equal(out4[:-1], out[:-1])


def test_decode_requests_share_pages_and_queries_lie_at_a_stride():
    rng = np.random.default_rng(6)
    n, Hq, Hkv, dk, B = 333, 8, 2, 128, 16
    c, table, rows, _ = _decode_case(12, Hq, Hkv, dk, B, (n,), True)
    table = np.repeat(table, 3, axis=0)
    lens = (n, 100, n)
    qkv = _from_bits(kv_ref.bf16_bits(rng.standard_normal((3, Hq + 2 * Hkv, dk)).astype(np.float32)))
    q = qkv[:, :Hq]
    status, out, lse = _run_decode(c, table, lens, q)
    assert status == 0
    ref = _check(c, table, [rows[0], rows[0][:100], rows[0]], _bits(q), lens)
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_decode_does_not_depend_on_the_other_requests_or_the_run(e4m3):
    lens = (2500, 0, 40, 900, 1, 7000)
    c, table, rows, qb = _decode_case(21, 8, 4, 128, 16, lens, e4m3)
    q = _from_bits(qb)
    _, out, lse = _run_decode(c, table, lens, q)
    for _ in range(3):
        _, again, lse2 = _run_decode(c, table, lens, q)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    for r, n in enumerate(lens):
        _, one, l1 = _run_decode(c, table[r:r + 1], (n,), q[r:r + 1].contiguous())
        assert torch.equal(out[r], one[0]) and torch.equal(lse[r], l1[0])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,dk", [(17, 1, 64), (40, 1, 128), (3, 1, 128), (33, 1, 256)])
@pytest.mark.parametrize("R,longest", [(7, 3000), (400, 900), (200, 3000)])
def test_decode_of_many_requests_is_that_of_each_alone(R, longest, Hq, Hkv, dk, e4m3):
    """whatever a CTA worked on before (a head tile of 16 queries, then one of a single query; a request of a hundred
    times larger queries) and however many rows the chunks' join has"""
    rng = np.random.default_rng(R + Hq)
    lens = tuple(int(x) for x in rng.integers(0, longest, R))
    c, table, rows, qb = _decode_case(R + dk, Hq, Hkv, dk, 16, lens, e4m3, extra_cols=0)
    size = torch.from_numpy(10.0 ** rng.integers(-2, 3, (R, 1, 1))).cuda()
    q = (_from_bits(qb).double() * size).to(torch.bfloat16)
    status, out, lse = _run_decode(c, table, lens, q)
    assert status == 0
    for r in [0, R - 1] + [int(x) for x in rng.integers(0, R, 12)]:
        _, one, l1 = _run_decode(c, table[r:r + 1], lens[r:r + 1], q[r:r + 1].contiguous())
        assert torch.equal(out[r], one[0]) and torch.equal(lse[r], l1[0]), r


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,dk,B", [(8, 2, 128, 16), (8, 2, 128, 1), (16, 2, 256, 16), (32, 2, 64, 64)])
def test_decode_of_short_requests_over_and_over(Hq, Hkv, dk, B, e4m3):
    """items of a tile or two, whose queries follow one another at the shortest distance, and calls in turn on two sets of
    inputs, so that a row that keeps another item's or call's numbers differs"""
    sets = []
    for seed in (31, 32):
        c, table, _, qb = _decode_case(seed + dk, Hq, Hkv, dk, B, LENS, e4m3)
        _, out, lse = _run_decode(c, table, LENS, _from_bits(qb))
        sets.append((c, np.tile(table, (40, 1)), _from_bits(np.tile(qb, (40, 1, 1))), out.repeat(40, 1, 1), lse.repeat(40, 1)))
    wrong = 0
    for _ in range(100):
        for c, table, q, out, lse in sets:
            status, o, l = _run_decode(c, table, LENS * 40, q)
            wrong += status != 0 or not torch.equal(o, out) or not torch.equal(l, lse)
    assert wrong == 0


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 1, 100, 333])
@pytest.mark.parametrize("Hq,Hkv,dk,B", [(8, 2, 128, 24), (4, 1, 64, 40), (16, 2, 256, 48), (8, 2, 128, 72), (9, 1, 128, 96),
                                         (2, 2, 256, 112), (8, 2, 64, 120), (8, 2, 128, 200)])
def test_decode_pages_that_do_not_fill_tiles(Hq, Hkv, dk, B, window, e4m3):
    c, table, rows, q = _decode_case(B + dk, Hq, Hkv, dk, B, LENS, e4m3, window=window)
    _check(c, table, rows, q, LENS, window)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hkv,dk", [(1, 64), (2, 128), (3, 256)])
@pytest.mark.parametrize("B", [2, 8, 16, 32])
def test_decode_wherever_keys_and_values_lie(B, Hkv, dk, e4m3):
    """the same cache with keys before values, after them, interleaved by page and by head, and its pages in a wider stride"""
    c, table, rows, qb = _decode_case(B + dk, 4 * Hkv, Hkv, dk, B, LENS, e4m3)
    k, v, n = c.k, c.v, c.num_blocks
    first = _check(c, table, rows, qb, LENS)
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.uint8 if e4m3 else torch.int16, device="cuda").view(k.dtype)
    pair = zeros(2, n, Hkv, B, dk)
    page = zeros(n, 2, Hkv, B, dk)
    head = zeros(n, Hkv, 2, B, dk)
    wide = zeros(2, n, Hkv + 1, B, dk)
    for kk, vv in [(pair[0], pair[1]), (pair[1], pair[0]), (page[:, 0], page[:, 1]), (page[:, 1], page[:, 0]),
                   (head[:, :, 0], head[:, :, 1]), (head[:, :, 1], head[:, :, 0]), (wide[0, :, :Hkv], wide[1, :, 1:])]:
        kk.copy_(k), vv.copy_(v)
        c.k, c.v = kk, vv
        status, out, lse = _run_decode(c, table, LENS, _from_bits(qb))
        assert status == 0 and torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_decode_nan_and_infinity_in_attended_rows(e4m3):
    """NaN keys or values of one KV head reach the rows of that head alone"""
    lens = (100, 90)
    c, table, rows, qb = _decode_case(31, 4, 2, 64, 16, lens, e4m3)
    s = int(rows[0][50])
    t = (c.k if e4m3 else c.v).view(torch.uint8 if e4m3 else torch.int16)
    t[s // 16, 1, s % 16, 5] = 0x7F if e4m3 else 0x7F80                        # NaN key, infinite value
    status, out, _ = _run_decode(c, table, lens, _from_bits(qb))
    o = kv_ref.bf16_value(_bits(out))
    assert status == 0
    assert np.isfinite(o[1]).all() and np.isfinite(o[0, :2]).all()
    assert (~np.isfinite(o[0, 2:])).any()


def test_decode_bad_lengths_and_pages_are_reported():
    lens = (100, 60, 30)
    c, table, rows, qb = _decode_case(41, 4, 2, 64, 16, lens, False)
    cap = table.shape[1] * 16
    status, out, lse = _run_decode(c, table, (100, cap + 1, 30), _from_bits(qb))
    assert status == 10 and (out[1] == 0).all() and torch.isinf(lse[1]).all()
    status, out2, _ = _run_decode(c, table, (100, -1, 30), _from_bits(qb))
    assert status == 10 and torch.equal(out, out2)
    for bad in (-1, c.num_blocks, 1 << 30):
        t = table.copy()
        t[0, 2] = bad
        status, out3, _ = _run_decode(c, t, lens, _from_bits(qb))
        assert status == 9 and torch.equal(out3[2], out[2])
        k, v = c.rows("k", rows[0]), c.rows("v", rows[0])
        k[32:48] = v[32:48] = 0
        o, _, to, _ = kv_ref.decode(kv_ref.bf16_value(qb[:1]), [k], [v], 64 ** -0.5)
        assert (np.abs(kv_ref.bf16_value(_bits(out3[:1])) - o) <= to).all()


def test_decode_in_a_graph_and_on_another_stream():
    lens = (700, 20)
    c, table, rows, qb = _decode_case(51, 8, 2, 128, 16, lens, True)
    q = _from_bits(qb)
    _, want, want_lse = _run_decode(c, table, lens, q)
    R, Hq, dk = q.shape
    tb, n = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse, st = torch.zeros_like(q), torch.zeros(R, Hq, device="cuda"), _status()
    ws = torch.empty(up.up_paged_decode_workspace_bytes(R, Hq, 2, dk, 16, table.shape[1]), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        up.up_paged_decode(q, c.k, c.v, tb, n, out, ws, st, **c.scales(), lse=lse)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        up.up_paged_decode(q, c.k, c.v, tb, n, out, ws, st, **c.scales(), lse=lse)
    out.zero_()
    n.copy_(torch.tensor((700, 0), dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and (out[1] == 0).all() and up.up_read_status(st) == 0


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,dk,B", [(8, 2, 128, 16), (4, 4, 64, 24), (9, 1, 256, 100)])
@pytest.mark.parametrize("times", [1, 60])
def test_bounds_checked_build_is_clean_and_identical(times, Hq, Hkv, dk, B, e4m3):
    lens = (0, 1, 65, 700, 129) * times

    def once():
        c, table, rows, qb = _decode_case(61, Hq, Hkv, dk, B, lens, e4m3, window=400)
        status, out, lse = _run_decode(c, table, lens, _from_bits(qb), window=400)
        st = _status()
        k = torch.zeros(len(rows[3]), Hkv, dk, dtype=torch.bfloat16, device="cuda")
        up.up_kv_read(c.k, c.v, torch.from_numpy(rows[3]).cuda(), k, None, st, **c.scales())
        return status, up.up_read_status(st), out.view(torch.int16), lse, k.view(torch.int16), c.k.view(torch.uint8).contiguous()
    ref = once()
    with library(_build.build(debug_bounds=True)):
        assert up.up_debug_bounds() == 1
        got = once()
    assert ref[:2] == (0, 0) and got[:2] == (0, 0)
    for a, b in zip(ref[2:], got[2:]):
        assert torch.equal(a, b)
