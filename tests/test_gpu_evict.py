"""Eviction on the GPU: up_kv_mass against 64-bit weights, up_kv_evict against a plain sort, up_kv_move bit for bit, and
the three together around up_paged_decode; lengths from none, pages of every size, orders of the cache's axes, NaN wherever
nobody may look, ties, protected rows, bad tables and lists, graphs and streams."""
import math

import numpy as np
import pytest
import torch

import long_context_prefill_varlen_gb300 as up
from long_context_prefill_varlen_gb300 import _build
from tests import evict_ref, kv_ref
from tests.test_gpu_debug_bounds import library
from tests.test_gpu_kvcache import ORDERS, _bits, _decode_case, _from_bits, _run_decode, _status

pytestmark = pytest.mark.gpu

F32 = kv_ref.F32


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------ the weights

def _mass(c, table, lens, q, lse, mass, born, **kw):
    st = _status()
    for name in ("counted", "total"):
        if kw.get(name) is not None:
            kw[name] = _i32(kw[name])
    up.up_kv_mass(q, c.k, c.v, torch.from_numpy(table).cuda(), _i32(lens), lse, mass, born, st, **c.scales(), **kw)
    return up.up_read_status(st)


def _records(c, seed):
    """mass and born with something in every row, used or not"""
    g = torch.Generator("cuda").manual_seed(seed)
    shape = (c.num_blocks, c.Hkv, c.B)
    return (torch.rand(shape, generator=g, device="cuda") * 3,
            torch.randint(0, 1 << 20, shape, generator=g, device="cuda", dtype=torch.int32))


def _check_mass(c, table, rows, qb, lens, decay=1.0, counted=None, total=None, lse=None, sm_scale=None):
    scale = qb.shape[2] ** -0.5 if sm_scale is None else sm_scale
    if lse is None:
        status, _, lse = _run_decode(c, table, lens, _from_bits(qb), sm_scale=sm_scale)
        assert status == 0
    mass, born = _records(c, 1)
    if counted is not None:                        # what lies at new rows does not count, whatever it is
        for r, n in enumerate(counted):
            page, off = rows[r][max(n, 0):] // c.B, rows[r][max(n, 0):] % c.B
            mass[page, :, off] = math.nan
    out, born_before = torch.full_like(mass, 77.0), born.clone()
    assert _mass(c, table, lens, _from_bits(qb), lse, mass, born, mass_out=out, counted=counted, total=total, decay=decay,
                 sm_scale=sm_scale) == 0
    got, old, bn, b0 = (x.cpu().numpy() for x in (out, mass, born, born_before))
    q, l = kv_ref.bf16_value(qb), lse.cpu().numpy().astype(np.float64)
    seen = np.zeros((c.num_blocks, c.B), dtype=bool)
    for r, n in enumerate(lens):
        page, off = rows[r] // c.B, rows[r] % c.B
        seen[page, off] = True
        if n == 0:
            continue
        w, tol = evict_ref.weights(q[r], c.rows("k", rows[r]), l[r], scale)
        new = np.arange(n) >= (n if counted is None else counted[r])
        was = np.where(new[None], 0.0, decay * old[page, :, off].T.astype(np.float64))
        want = was + w
        # the decay as fp32 has it, and one fused product and sum
        assert (np.abs(got[page, :, off].T - want) <= tol + 2 * F32 * np.abs(want) + F32 * np.abs(was)).all()
        want_born = np.where(new[:, None], ((n if total is None else total[r]) - n + np.arange(n))[:, None], b0[page, :, off])
        assert np.array_equal(bn[page, :, off], want_born)
    free = ~seen[:, None].repeat(c.Hkv, 1)
    assert (got[free] == 77.0).all() and np.array_equal(bn[free], b0[free])
    # in place
    same, born2 = mass.clone(), born_before.clone()
    assert _mass(c, table, lens, _from_bits(qb), lse, same, born2, counted=counted, total=total, decay=decay, sm_scale=sm_scale) == 0
    keep = torch.from_numpy(free).cuda()
    assert torch.equal(same[~keep], out[~keep]) and torch.equal(born2, born)
    assert np.array_equal(same[keep].cpu().numpy(), mass[keep].cpu().numpy(), equal_nan=True)
    return out, lse


LENS = (0, 1, 15, 16, 17, 63, 64, 65, 130, 257, 1000)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("B", [1, 8, 16, 24, 64, 100, 256])
@pytest.mark.parametrize("Hq,Hkv,dk", [(8, 2, 128), (2, 2, 64), (16, 2, 256)])
def test_weights_over_lengths_and_page_sizes(Hq, Hkv, dk, B, e4m3):
    c, table, rows, q = _decode_case(B + dk, Hq, Hkv, dk, B, LENS, e4m3)
    _check_mass(c, table, rows, q, LENS)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("group,Hkv", [(1, 3), (3, 1), (7, 2), (8, 1), (9, 1), (16, 1), (17, 2), (32, 1)])
def test_weights_over_head_groups(group, Hkv, dk, e4m3):
    lens = (300, 0, 77)
    c, table, rows, q = _decode_case(group + dk, group * Hkv, Hkv, dk, 16, lens, e4m3)
    _check_mass(c, table, rows, q, lens, decay=0.5, counted=(299, 0, 70), total=(1000, 0, 77))


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("group,Hkv,dk,B", [(33, 1, 128, 16), (64, 1, 64, 24), (71, 2, 128, 16), (40, 1, 256, 100)])
def test_weights_of_more_heads_than_shared_memory_holds(group, Hkv, dk, B, e4m3):
    """beyond 32 query heads a key head the queries come in turns"""
    lens = (300, 0, 77, 1, 64)
    c, table, rows, q = _decode_case(group + dk, group * Hkv, Hkv, dk, B, lens, e4m3)
    _check_mass(c, table, rows, q, lens, decay=0.5, counted=(299, 0, 70, 0, 64), total=(1000, 0, 77, 1, 64))


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("decay,counted", [(0.0, None), (1.0, (0, 0, 0)), (0.9, (400, -3, 50)), (1.0, (900, 1, 16))])
def test_decay_new_rows_and_axis_orders(decay, counted, e4m3, order):
    lens = (400, 1, 50)
    c, table, rows, q = _decode_case(5, 4, 2, 128, 16, lens, e4m3, order=order)
    counted = None if counted is None else tuple(min(x, n) for x, n in zip(counted, lens)) if counted[0] != 900 else counted
    _check_mass(c, table, rows, q, lens, decay=decay, counted=counted, total=(1 << 30, 1, 50))


@pytest.mark.parametrize("scale", [0.25, 4.0])
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_sharp_and_flat_weights(e4m3, scale):
    c, table, rows, q = _decode_case(6, 8, 2, 64, 16, (500, 33), e4m3, scale=scale)
    _check_mass(c, table, rows, q, (500, 33), sm_scale=-0.5 if scale < 1 else 0.125)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,dk", [(8, 2, 128), (20, 1, 64)])
def test_scores_of_large_keys_and_small_queries(Hq, Hkv, dk, e4m3):
    """as ordinary as any, though a product of only some of their factors is beyond 32 bits"""
    lens = (200, 33)
    for up_by in (-115, 115):
        c, table, rows, qb = _decode_case(13, Hq, Hkv, dk, 16, lens, e4m3, scale=2.0 ** up_by)
        _check_mass(c, table, rows, kv_ref.bf16_bits((kv_ref.bf16_value(qb) * 2.0 ** -up_by).astype(np.float32)), lens)


def test_a_head_without_weight_and_one_whose_lse_is_not_a_number():
    lens = (40, 40)
    c, table, rows, q = _decode_case(7, 4, 2, 64, 16, lens, False)
    _, _, lse = _run_decode(c, table, lens, _from_bits(q))
    lse[0, 0] = lse[0, 1] = lse[1, 2] = -math.inf
    _check_mass(c, table, rows, q, lens, lse=lse)
    lse[0, 3] = math.nan
    mass, born = _records(c, 2)
    mass[:] = 0
    assert _mass(c, table, lens, _from_bits(q), lse, mass, born) == 0
    page, off = rows[0] // c.B, rows[0] % c.B
    assert (mass[page, 0, off] == 0).all() and torch.isnan(mass[page, 1, off]).all()
    page, off = rows[1] // c.B, rows[1] % c.B
    assert torch.isfinite(mass[page, :, off]).all()


@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("sm_scale", [None, 0.3, -0.3, -0.088388346])
def test_scores_of_minus_infinity_have_no_weight(sm_scale, dk):
    """as in up_paged_decode, whose lse is that of the other rows; the scale's two parts may be of either sign"""
    lens, gone = (200, 33), ((0, 7, 100, 199), (32,))
    c, table, rows, qb = _decode_case(11, 8, 2, dk, 16, lens, False)
    q = kv_ref.bf16_value(qb)
    q[:, :, 5] = np.abs(q[:, :, 5]) + 0.5
    qb = kv_ref.bf16_bits(q.astype(np.float32))
    q = kv_ref.bf16_value(qb)
    scale = dk ** -0.5 if sm_scale is None else sm_scale
    for r, at in enumerate(gone):
        s = rows[r][list(at)]
        c.k[torch.from_numpy(s // 16).cuda(), :, torch.from_numpy(s % 16).cuda(), 5] = -math.inf if scale > 0 else math.inf
    status, _, lse = _run_decode(c, table, lens, _from_bits(qb), sm_scale=sm_scale)
    assert status == 0 and torch.isfinite(lse).all()
    mass, born = _records(c, 1)
    old = mass.clone()
    assert _mass(c, table, lens, _from_bits(qb), lse, mass, born, sm_scale=sm_scale) == 0
    for r, at in enumerate(gone):
        s, rest = rows[r][list(at)], np.delete(rows[r], at)
        assert torch.equal(mass[s // 16, :, s % 16], old[s // 16, :, s % 16])
        w, tol = evict_ref.weights(q[r], c.rows("k", rest), lse[r].cpu().numpy().astype(np.float64), scale)
        was, got = (x[rest // 16, :, rest % 16].cpu().numpy().T.astype(np.float64) for x in (old, mass))
        assert (np.abs(got - was - w) <= tol + 2 * F32 * (was + w)).all()


def test_many_requests_and_none_of_their_neighbours():
    """a request's weights do not depend on the batch; more requests than a warp has lanes; a long one among them"""
    lens = tuple([0, 3, 100] * 30 + [5000, 0, 0, 64])
    c, table, rows, q = _decode_case(8, 8, 2, 128, 16, lens, True)
    out, lse = _check_mass(c, table, rows, q, lens)
    mass, born = _records(c, 1)
    for r in (1, 2, len(lens) - 4, len(lens) - 1):
        alone = torch.full_like(mass, 77.0)
        assert _mass(c, table[r:r + 1], lens[r:r + 1], _from_bits(q[r:r + 1]), lse[r:r + 1].contiguous(), mass, born, mass_out=alone) == 0
        page, off = rows[r] // c.B, rows[r] % c.B
        assert torch.equal(alone[page, :, off], out[page, :, off])


def test_bad_lengths_and_pages_of_the_weights():
    lens = (40, 50, 60)
    c, table, rows, q = _decode_case(9, 4, 2, 64, 16, lens, True)
    _, _, lse = _run_decode(c, table, lens, _from_bits(q))
    mass, born = _records(c, 3)
    want = torch.full_like(mass, 77.0)
    assert _mass(c, table, lens, _from_bits(q), lse, mass, born, mass_out=want) == 0
    for bad in (-1, table.shape[1] * c.B + 1):
        out = torch.full_like(mass, 77.0)
        assert _mass(c, table, (40, bad, 60), _from_bits(q), lse, mass, born, mass_out=out) == 10
        page, off = rows[1] // c.B, rows[1] % c.B
        assert (out[page, :, off] == 77.0).all()
        for r in (0, 2):
            page, off = rows[r] // c.B, rows[r] % c.B
            assert torch.equal(out[page, :, off], want[page, :, off])
    for bad in (-1, c.num_blocks, 1 << 30):
        t, out = table.copy(), torch.full_like(mass, 77.0)
        t[1, 1] = bad
        assert _mass(c, t, lens, _from_bits(q), lse, mass, born, mass_out=out) == 9
        good = np.delete(rows[1], np.arange(16, 32))
        assert torch.equal(out[good // 16, :, good % 16], want[good // 16, :, good % 16])
        gone = rows[1][16:32]
        assert (out[gone // 16, :, gone % 16] == 77.0).all()


# ------------------------------------------------------------------------------------------ the rows that stay

def _choose(mass, born, table, lens, budget, max_moves=None, total=None, **kw):
    R, Hkv = len(lens), mass.shape[1]
    st = _status()
    room = max(1, max(min(max(b, 0), max(n - b, 0)) for n, b in zip(lens, budget))) if max_moves is None else max_moves
    moves, num = torch.full((R, Hkv, room, 2), -7, dtype=torch.int32, device="cuda"), torch.full((R, Hkv), -7, dtype=torch.int32, device="cuda")
    new_len = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    up.up_kv_evict(mass, born, torch.from_numpy(table).cuda(), _i32(lens), _i32(budget), moves, num, new_len, st,
                   total=None if total is None else _i32(total), **kw)
    return up.up_read_status(st), moves, num, new_len


def _tables(rng, lens, B, extra=2):
    need = [-(-n // B) for n in lens]
    nb = sum(need) + 3
    table = rng.integers(-(1 << 31), 1 << 31, (len(lens), max(1, max(need)) + extra)).astype(np.int32)
    perm, at = rng.permutation(nb), 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, nb


def _check_choice(seed, lens, budget, Hkv=2, B=16, sinks=0, recent=0, values=None, total=None):
    """values(rng, n): a list's masses; rows beyond the lists hold NaN and protected numbers"""
    rng = np.random.default_rng(seed)
    table, nb = _tables(rng, lens, B)
    mass = np.full((nb, Hkv, B), np.nan, dtype=np.float32)
    born = np.zeros((nb, Hkv, B), dtype=np.int32)
    values = values or (lambda rng, n: np.exp(2 * rng.standard_normal(n)))
    lists = {}
    for r, n in enumerate(lens):
        p = np.arange(n)
        t = n if total is None else total[r]
        for h in range(Hkv):
            m = np.asarray(values(rng, n), dtype=np.float32)
            b = p.copy() if total is None else np.sort(rng.choice(t, n, replace=False))
            if total is not None:
                rng.shuffle(b)
            mass[table[r, p // B], h, p % B], born[table[r, p // B], h, p % B] = m, b
            lists[r, h] = m, b, t
    md, bd = torch.from_numpy(mass).cuda(), torch.from_numpy(born).cuda()
    status, moves, num, new_len = _choose(md, bd, table, lens, budget, total=total, sinks=sinks, recent=recent)
    assert status == 0
    assert np.array_equal(new_len.cpu().numpy(), np.minimum(budget, lens))
    mv, nm = moves.cpu().numpy(), num.cpu().numpy()
    for (r, h), (m, b, t) in lists.items():
        want = evict_ref.evict(m, b, t, budget[r], sinks, recent)
        assert nm[r, h] == len(want)
        assert np.array_equal(mv[r, h, :len(want)], np.array(want, dtype=np.int32).reshape(-1, 2))
        assert (mv[r, h, len(want):] == -7).all()
    return md, bd, table, moves, num, new_len


@pytest.mark.parametrize("B", [1, 8, 16, 24, 100, 256])
@pytest.mark.parametrize("Hkv", [1, 2, 5])
@pytest.mark.parametrize("share", [0.0, 0.1, 0.5, 0.9, 1.0])
def test_the_choice_over_lengths_pages_and_budgets(share, Hkv, B):
    lens = (0, 1, 2, 31, 32, 33, 257, 1000, 700)
    budget = [int(n * share) for n in lens[:-1]] + [10_000]
    _check_choice(B + Hkv, lens, budget, Hkv, B)


@pytest.mark.parametrize("R,n", [(1, 4097), (1, 20_000), (2, 9000), (5, 5000), (30, 3001), (200, 300), (300, 40)])
@pytest.mark.parametrize("Hkv", [1, 8])
def test_the_choice_in_clusters_of_every_size(R, n, Hkv):
    rng = np.random.default_rng(R)
    lens = [n] + [int(x) for x in rng.integers(0, n, R - 1)]
    _check_choice(R, lens, [int(x * rng.random()) for x in lens], Hkv, 16, sinks=4, recent=10)


@pytest.mark.parametrize("name", ["equal", "few_values", "last_bits", "zeros"])
def test_ties_of_lists_that_have_a_cta_each(name):
    """more keys with one first digit than the candidates' place holds, without a cluster"""
    _check_choice(7, (6000,) + (30,) * 99, (2500,) + (10,) * 99, values=EDGES[name], sinks=3, recent=20)
    _check_choice(8, (6000, 3000), (5999, 100), Hkv=80, values=EDGES[name])


@pytest.mark.parametrize("wide", [500, 3000, 30_000])
def test_the_choice_does_not_go_by_the_tables_width(wide):
    """many lists, short ones and long ones, under tables of 8K to half a million positions: launches of other forms, the same
    moves"""
    rng = np.random.default_rng(10)
    lens = [0, 1, 5000, 8000] + [int(x) for x in rng.integers(0, 3000, 36)]
    if wide > 500:
        lens += [8192, 8193, 16_384, 16_385, 40_000]
    budget = [int(n * rng.random()) for n in lens]
    md, bd, table, moves, num, new_len = _check_choice(11, lens, budget, Hkv=8, sinks=4, recent=30)
    more = np.full((len(lens), max(wide, table.shape[1])), -1, dtype=np.int32)
    more[:, :table.shape[1]] = table
    status, m, n, l = _choose(md, bd, more, lens, budget, max_moves=moves.shape[2], sinks=4, recent=30)
    assert status == 0 and torch.equal(m, moves) and torch.equal(n, num) and torch.equal(l, new_len)


def test_records_that_are_not_aligned():
    rng = np.random.default_rng(9)
    lens, budget = (700, 5, 2000), (300, 2, 1990)
    table, nb = _tables(rng, lens, 16)
    mass, born = torch.rand(nb, 2, 16, device="cuda"), torch.randint(0, 3000, (nb, 2, 16), device="cuda", dtype=torch.int32)
    want = _choose(mass, born, table, lens, budget, sinks=9, recent=3)
    odd = [torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape) for x in (mass, born)]
    for o, x in zip(odd, (mass, born)):
        o.copy_(x)
    for m, b in ((odd[0], born), (mass, odd[1]), odd):
        got = _choose(m, b, table, lens, budget, sinks=9, recent=3)
        assert got[0] == want[0] == 0 and all(torch.equal(x, y) for x, y in zip(got[1:], want[1:]))


def test_room_for_no_moves():
    mass, born = torch.rand(3, 1, 16, device="cuda"), torch.zeros(3, 1, 16, dtype=torch.int32, device="cuda")
    table = np.array([[0, 1, 2]], dtype=np.int32)
    status, _, num, new_len = _choose(mass, born, table, (40,), (50,), max_moves=0)
    assert status == 0 and int(num) == 0 and int(new_len) == 40
    status, _, num, new_len = _choose(mass, born, table, (40,), (30,), max_moves=0)
    assert status == 12 and int(num) == 0 and int(new_len) == 40


def test_a_list_longer_than_shared_memory():
    for n, k, sinks in ((500_001, 20_000, 100), (500_001, 499_990, 100), (500_001, 50, 400_000)):
        rng = np.random.default_rng(k)
        mass = np.exp(2 * rng.standard_normal(n)).astype(np.float32)
        mass[rng.random(n) < 0.3] = 0
        born = rng.permutation(n).astype(np.int32)
        for R in (1, 160):                        # a cluster of eight, a CTA alone
            lens, budget = [n] + [0] * (R - 1), [k] * R
            table = np.zeros((R, -(-n // 64)), dtype=np.int32)
            table[0] = rng.permutation(table.shape[1])
            md, bd = (torch.zeros(table.shape[1], 1, 64, dtype=t, device="cuda") for t in (torch.float32, torch.int32))
            p = torch.arange(n, device="cuda")
            page = torch.from_numpy(table[0]).cuda().long()[p // 64]
            md[page, 0, p % 64], bd[page, 0, p % 64] = torch.from_numpy(mass).cuda(), torch.from_numpy(born).cuda()
            status, moves, num, new_len = _choose(md, bd, table, lens, budget, sinks=sinks, recent=1000)
            assert status == 0 and int(new_len[0]) == k and (num[1:] == 0).all()
            safe = (born < sinks) | (born >= n - 1000)
            stay = np.zeros(n, dtype=bool)
            stay[np.lexsort((np.arange(n), -mass, ~safe))[:k]] = True
            want = np.stack((np.flatnonzero(stay[k:]) + k, np.flatnonzero(~stay[:k])), 1)
            assert int(num[0, 0]) == len(want) and np.array_equal(moves[0, 0, :len(want)].cpu().numpy(), want)


EDGES = {
    "equal": lambda rng, n: np.full(n, 0.25),
    "zeros": lambda rng, n: np.zeros(n),
    "signed_zeros": lambda rng, n: np.where(rng.random(n) < 0.5, -0.0, 0.0),
    "few_values": lambda rng, n: rng.integers(0, 4, n) * 0.5,
    "nan_and_infinities": lambda rng, n: rng.choice(np.array([math.nan, -math.nan, math.inf, -math.inf, 1.0, -1.0, 1e-45]), n),
    "negative": lambda rng, n: rng.standard_normal(n),
    "subnormal": lambda rng, n: rng.integers(0, 100, n) * 1e-45,
    "last_bits": lambda rng, n: 1 + rng.integers(0, 8, n) * 2.0 ** -23,
    "falling": lambda rng, n: np.arange(n, 0, -1),
    "rising": lambda rng, n: np.arange(n),
}


@pytest.mark.parametrize("name", EDGES)
def test_ties_and_numbers_that_are_none(name):
    _check_choice(3, (777, 64, 5000), (300, 63, 4990), values=EDGES[name], sinks=3, recent=20)


@pytest.mark.parametrize("sinks,recent", [(0, 0), (1, 1), (128, 0), (0, 128), (1 << 30, 0), (0, (1 << 31) - 1), (200, 200)])
def test_protected_rows_that_fit_and_that_do_not(sinks, recent):
    lens = (400, 1000, 2000, 50)
    _check_choice(4, lens, (100, 500, 1, 49), sinks=sinks, recent=recent)
    _check_choice(5, lens, (100, 500, 1999, 7), sinks=sinks, recent=recent, total=(500, 1000, 50_000, 51), values=EDGES["few_values"])


@pytest.mark.parametrize("name,other", [("sinks", "recent"), ("recent", "sinks")])
def test_protected_rows_of_any_number(name, other):
    """beyond 32 bits, too: all rows, which then go by mass, and the other kind of protection makes no difference"""
    lens, budget = (100, 300), (30, 200)
    md, bd, table, *want = _check_choice(12, lens, budget, **{name: (1 << 31) - 1, other: 20})
    few = _check_choice(12, lens, budget, **{other: 20})
    assert not torch.equal(want[0], few[3])
    for number in (1 << 31, 1 << 32, 1 << 40):
        status, *got = _choose(md, bd, table, lens, budget, **{name: number, other: 20})
        assert status == 0 and all(torch.equal(x, y) for x, y in zip(got, want))
    for number in (-1, -(1 << 32)):
        with pytest.raises(up.UpError) as e:
            _choose(md, bd, table, lens, budget, **{name: number})
        assert e.value.code == up.UP_ERR_ARG


def test_requests_that_are_left_as_they_are():
    rng = np.random.default_rng(6)
    lens, B = (100, 200, 300, 50), 16
    table, nb = _tables(rng, lens, B)
    mass, born = torch.rand(nb, 2, B, device="cuda"), torch.zeros(nb, 2, B, dtype=torch.int32, device="cuda")
    ok, moves, num, new_len = _choose(mass, born, table, lens, (60, 100, 30, 25))
    assert ok == 0

    def others_are(result, r, status, length):
        assert result[0] == status and int(result[3][r]) == length and (result[2][r] == 0).all() and (result[1][r] == -7).all()
        for x in set(range(4)) - {r}:
            n = int(num[x].max())
            assert torch.equal(result[2][x], num[x]) and int(result[3][x]) == int(new_len[x])
            assert torch.equal(result[1][x, :, :n], moves[x, :, :n])
    others_are(_choose(mass, born, table, lens, (60, -1, 30, 25), max_moves=100), 1, 11, 200)
    others_are(_choose(mass, born, table, lens, (60, 100, 30, 25), max_moves=99), 1, 12, 200)
    others_are(_choose(mass, born, table, (100, -5, 300, 50), (60, 100, 30, 25), max_moves=100), 1, 10, 0)
    others_are(_choose(mass, born, table, (100, table.shape[1] * B + 1, 300, 50), (60, 100, 30, 25), max_moves=100), 1, 10, 0)
    for bad in (-1, nb, 1 << 30):
        t = table.copy()
        t[2, 7] = bad
        others_are(_choose(mass, born, t, lens, (60, 100, 30, 25), max_moves=100), 2, 9, 300)
    # a row of the table that nobody needs to look at
    t = table.copy()
    t[2] = -1
    assert _choose(mass, born, t, lens, (60, 100, 300, 25), max_moves=100)[0] == 0
    assert _choose(mass, born, t, lens, (60, 100, 0, 25), max_moves=100)[0] == 0


# ------------------------------------------------------------------------------------------ forms of the choice
# (by the tables' width and the number of lists; which form a case takes is tested with the host's rule)

@pytest.mark.parametrize("name", evict_ref.FORMS)
def test_the_choice_in_every_form(name):
    (_, Hkv, n), (_, _, apart, _) = evict_ref.FORMS[name]
    lens, rng = evict_ref.form_lengths(name), np.random.default_rng(n)
    before = up.up_kernel_launches()
    _check_choice(n, lens, [int(x * rng.random()) for x in lens], Hkv, sinks=4, recent=10)
    assert up.up_kernel_launches() == before + 1 + apart
    _check_choice(n + 1, lens, [x - 1 for x in lens], Hkv, total=[x + x // 3 for x in lens], sinks=50, recent=100)


CLUSTERS = ("pairs", "fours", "eights", "pairs_of_32", "fours_of_32", "eights_of_32")
FAR = ("eights_of_32_again", "sixteens", "sixteens_again")


def _clustered(name, short):
    """lists of 13,000 positions at most, which several CTAs share, under the form's tables; or the form's own"""
    (_, Hkv, n), _ = evict_ref.FORMS[name]
    lens = evict_ref.form_lengths(name)
    return ([min(x, 13_000) for x in lens] if short else lens), Hkv, -(-n // 16)


def _check_wide(seed, lens, budget, Hkv, wide, **kw):
    """as _check_choice, and under tables of `wide` entries"""
    md, bd, table, moves, num, new_len = _check_choice(seed, lens, budget, Hkv, **kw)
    more = np.full((len(lens), max(wide, table.shape[1])), -1, dtype=np.int32)
    more[:, :table.shape[1]] = table
    kw.pop("values", None)
    status, m, n, l = _choose(md, bd, more, lens, budget, max_moves=moves.shape[2], **kw)
    assert status == 0 and torch.equal(m, moves) and torch.equal(n, num) and torch.equal(l, new_len)


@pytest.mark.parametrize("form", CLUSTERS)
@pytest.mark.parametrize("name", EDGES)
def test_ties_and_numbers_that_are_none_in_clusters(name, form):
    lens, Hkv, wide = _clustered(form, True)
    assert max(lens) > 6144                       # more than a CTA takes alone
    _check_wide(3, lens, [n // 3 for n in lens], Hkv, wide, values=EDGES[name], sinks=3, recent=20)
    _check_wide(4, lens, [n - 7 for n in lens], Hkv, wide, values=EDGES[name])


@pytest.mark.parametrize("form", FAR)
@pytest.mark.parametrize("name", ["equal", "zeros", "few_values", "last_bits", "nan_and_infinities"])
def test_ties_of_lists_that_eight_ctas_and_more_share(name, form):
    lens, Hkv, wide = _clustered(form, False)
    _check_wide(5, lens, [n // 3 for n in lens], Hkv, wide, values=EDGES[name], sinks=3, recent=20)


@pytest.mark.parametrize("form", CLUSTERS)
@pytest.mark.parametrize("sinks,recent", [(0, 0), (1, 1), (128, 0), (0, 128), (1 << 30, 0), (0, (1 << 31) - 1), (5000, 2000)])
def test_protected_rows_in_clusters(sinks, recent, form):
    lens, Hkv, wide = _clustered(form, True)
    _check_wide(6, lens, [max(1, n // 20) for n in lens], Hkv, wide, sinks=sinks, recent=recent)
    total = [n + n // 2 + 1 for n in lens]
    _check_wide(7, lens, [n - 1 for n in lens], Hkv, wide, sinks=sinks, recent=recent, total=total, values=EDGES["few_values"])


@pytest.mark.parametrize("form", ["pairs", "eights_of_32", "eights_of_32_again", "sixteens"])
def test_a_bad_page_and_a_bad_length_in_clusters(form):
    lens, Hkv, _ = _clustered(form, False)
    rng = np.random.default_rng(8)
    table, nb = _tables(rng, lens, 16)
    mass, born = torch.rand(nb, Hkv, 16, device="cuda"), torch.zeros(nb, Hkv, 16, dtype=torch.int32, device="cuda")
    budget = [n // 2 for n in lens]
    ok, moves, num, new_len = _choose(mass, born, table, lens, budget)
    assert ok == 0
    for at in (0, lens[0] // 32, lens[0] // 16 - 1):             # the first CTA's, one in the middle, the last one's
        t = table.copy()
        t[0, at] = nb
        status, m, n, l = _choose(mass, born, t, lens, budget)
        assert status == 9 and (n[0] == 0).all() and int(l[0]) == lens[0] and (m[0] == -7).all()
        assert torch.equal(m[1:], moves[1:]) and torch.equal(n[1:], num[1:]) and torch.equal(l[1:], new_len[1:])
    for bad in (-1, table.shape[1] * 16 + 1):
        status, m, n, l = _choose(mass, born, table, [bad] + lens[1:], budget, max_moves=moves.shape[2])
        assert status == 10 and (n[0] == 0).all() and int(l[0]) == 0 and (m[0] == -7).all()
        assert torch.equal(m[1:], moves[1:]) and torch.equal(n[1:], num[1:]) and torch.equal(l[1:], new_len[1:])


# ------------------------------------------------------------------------------------------ the moves

def _all_rows(c):
    t = [x.view(torch.uint8) for x in (c.k, c.v)] if c.e4m3 else [x.view(torch.int16) for x in (c.k, c.v)]
    return [x.cpu().numpy() for x in t + ([c.ks, c.vs] if c.e4m3 else [])]


def _move(c, table, moves, num, mass=None, born=None):
    st = _status()
    up.up_kv_move(c.k, c.v, torch.from_numpy(table).cuda(), moves, num, st, **c.scales(), mass=mass, born=born)
    return up.up_read_status(st)


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hkv,dk,B", [(2, 64, 16), (8, 128, 16), (3, 256, 24), (1, 128, 1), (2, 128, 100)])
def test_moves_are_exact(Hkv, dk, B, e4m3, order):
    lens = (0, 3, 200, 1, 1111)
    c, table, rows, _ = _decode_case(dk + B, Hkv, Hkv, dk, B, lens, e4m3, order=order)
    rng = np.random.default_rng(B)
    R, room = len(lens), 400
    lists = np.full((R, Hkv, room, 2), 1 << 30, dtype=np.int32)       # entries past a list's number: not looked at
    num = np.zeros((R, Hkv), dtype=np.int32)
    for r, n in enumerate(lens):
        for h in range(Hkv):
            m = int(rng.integers(0, min(room, n // 2) + 1))
            p = rng.permutation(n)[:2 * m]
            lists[r, h, :m], num[r, h] = p.reshape(2, m).T, m
    mass, born = _records(c, 4)
    want, wm, wb = [x.copy() for x in _all_rows(c)], mass.cpu().numpy().copy(), born.cpu().numpy().copy()
    for r in range(R):
        for h in range(Hkv):
            src, dst = (rows[r][lists[r, h, :num[r, h], j]] for j in (0, 1)) if num[r, h] else (np.zeros(0, int),) * 2
            for x in want + [wm, wb]:
                x[dst // B, h, dst % B] = x[src // B, h, src % B]
    md, nd = torch.from_numpy(lists).cuda(), torch.from_numpy(num).cuda()
    assert _move(c, table, md, nd, mass, born) == 0
    for x, y in zip(_all_rows(c) + [mass.cpu().numpy(), born.cpu().numpy()], want + [wm, wb]):
        assert np.array_equal(x, y)
    # again: sources are where they were, so the same; and without records, which stay
    kept = mass.clone()
    assert _move(c, table, md, nd) == 0 and torch.equal(kept, mass)
    assert all(np.array_equal(x, y) for x, y in zip(_all_rows(c), want))


def test_bad_moves_are_skipped_and_reported():
    lens = (100, 100)
    for bad, status in ((-1, 8), (1 << 20, 8), (None, 9)):
        c, table, rows, _ = _decode_case(1, 2, 2, 64, 16, lens, True)
        lists = np.zeros((2, 2, 3, 2), dtype=np.int32)
        lists[..., 0], lists[..., 1] = (90, 80, 70), (1, 2, 3)
        t = table.copy()
        if bad is None:
            t[1, 80 // 16] = c.num_blocks                             # the page of rows 80 to 95
        else:
            lists[1, 0, 1, 0] = bad
        before = _all_rows(c)
        assert _move(c, t, torch.from_numpy(lists).cuda(), _i32([[3, 3], [3, 3]])) == status
        after = _all_rows(c)
        for x, y in zip(before, after):
            for r in range(2):
                for h in range(2):
                    for src, dst in lists[r, h]:
                        skipped = r == 1 and ((bad is None and src in (90, 80)) or src == bad)
                        d, s = rows[r][dst], rows[r][dst] if skipped else rows[r][src]
                        assert np.array_equal(y[d // 16, h, d % 16], x[s // 16, h, s % 16])
    c, table, rows, _ = _decode_case(1, 2, 2, 64, 16, lens, False)
    before = _all_rows(c)
    assert _move(c, table, torch.zeros(2, 2, 3, 2, dtype=torch.int32, device="cuda"), _i32([[0, 4], [-1, 0]])) == 12
    assert all(np.array_equal(x, y) for x, y in zip(before, _all_rows(c)))


# ------------------------------------------------------------------------------------------ together

def _step(c, table, lens, q, mass, born, budget, state, **kw):
    """decode, weigh, choose, move: the new lengths"""
    status, out, lse = _run_decode(c, table, lens, q)
    assert status == 0
    assert _mass(c, table, lens, q, lse, mass, born, counted=state["counted"], total=state["total"]) == 0
    status, moves, num, new_len = _choose(mass, born, table, lens, budget, total=state["total"], **kw)
    assert status == 0
    assert _move(c, table, moves, num, mass, born) == 0
    return out, [int(x) for x in new_len.cpu()]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,dk,B", [(8, 2, 128, 16), (4, 4, 64, 24), (12, 1, 256, 16)])
def test_decoding_while_rows_go(Hq, Hkv, dk, B, e4m3):
    """Six steps on ragged requests, each with a new row: the rows of every head are followed on the CPU by their numbers in
    the stream, the decode's output has to be attention over exactly those, and the records theirs."""
    lens0, steps, sinks, recent = (0, 30, 300, 900), 6, 2, 5
    full = tuple(n + steps for n in lens0)
    c, table, rows, _ = _decode_case(3, Hq, Hkv, dk, B, full, e4m3)
    R = len(lens0)
    rng = np.random.default_rng(dk)
    stream = [[c.rows(x, s) for s in rows] for x in "kv"]            # every request's tokens, in the stream's order
    raw = [[x[s // B, :, s % B].copy() for s in rows] for x in _all_rows(c)]
    mass = torch.full((c.num_blocks, Hkv, B), math.nan, device="cuda")
    born = torch.full((c.num_blocks, Hkv, B), -9, dtype=torch.int32, device="cuda")
    here = [[list(range(n)) for _ in range(Hkv)] for n in lens0]     # numbers of the rows at positions 0, 1, ...
    weight = {}
    lens, counted = list(lens0), [0] * R
    for step in range(steps):
        # the new token's row, written at the end of what each request has
        arrays = [c.k.view(torch.uint8 if e4m3 else torch.int16), c.v.view(torch.uint8 if e4m3 else torch.int16)] + ([c.ks, c.vs] if e4m3 else [])
        for r in range(R):
            at = rows[r][lens[r]]
            for x, y in zip(arrays, raw):
                x[at // B, :, at % B] = torch.from_numpy(y[r][lens0[r] + step]).cuda()
            for h in range(Hkv):
                here[r][h].append(lens0[r] + step)
            lens[r] += 1
        total = [n + step + 1 for n in lens0]
        budget = [10, 20, 150 - 3 * step, 2000 if step < 2 else 600]
        qb = kv_ref.bf16_bits(rng.standard_normal((R, Hq, dk)).astype(np.float32))
        q64 = kv_ref.bf16_value(qb)
        got, new = _step(c, table, lens, _from_bits(qb), mass, born, budget, dict(counted=counted, total=total), sinks=sinks, recent=recent)
        got = kv_ref.bf16_value(_bits(got))
        m, b = mass.cpu().numpy(), born.cpu().numpy()
        g = Hq // Hkv
        for r in range(R):
            for h in range(Hkv):
                ids = here[r][h]
                k, v = stream[0][r][ids][:, h:h + 1], stream[1][r][ids][:, h:h + 1]
                o, lse, to, _ = kv_ref.decode(q64[r:r + 1, h * g:(h + 1) * g], [k], [v], dk ** -0.5)
                assert (np.abs(got[r, h * g:(h + 1) * g] - o[0]) <= to[0]).all()
                w, tol = evict_ref.weights(q64[r, h * g:(h + 1) * g], k, lse[0], dk ** -0.5)
                for i, x in enumerate(ids):
                    old = weight.get((r, h, x), (0.0, 0.0))
                    # the lse that the kernel was given is off as well (kv_ref.decode's tolerance of it): 2 tol covers both
                    weight[r, h, x] = (old[0] + w[0, i], old[1] + 3 * tol[0, i] + 40 * F32 * (len(ids) + 16) * w[0, i] + 4 * F32 * (old[0] + w[0, i]))
                if new[r] < lens[r]:
                    # the records as they are say who stays (their values are checked against the weights just below)
                    stay = [b[rows[r][p] // B, h, rows[r][p] % B] for p in range(new[r])]
                    assert len(set(stay)) == len(stay) and set(stay) <= set(ids)
                    safe = {x for x in ids if x < sinks or x >= total[r] - recent}
                    if len(safe) <= new[r]:
                        assert safe <= set(stay)
                        gone = [x for x in ids if x not in set(stay)]
                        least = min((weight[r, h, x][0] + weight[r, h, x][1] for x in stay if x not in safe), default=math.inf)
                        assert all(weight[r, h, x][0] - weight[r, h, x][1] <= least for x in gone)
                    here[r][h] = [int(x) for x in stay]
                for p, x in enumerate(here[r][h]):
                    at = rows[r][p]
                    assert b[at // B, h, at % B] == x
                    assert abs(m[at // B, h, at % B] - weight[r, h, x][0]) <= weight[r, h, x][1]
        lens, counted = new, list(new)


def _whole(seed, e4m3):
    lens = (700, 0, 1500, 33)
    c, table, rows, qb = _decode_case(seed, 8, 2, 128, 16, lens, e4m3)
    mass, born = _records(c, seed)
    return c, table, lens, _from_bits(qb), mass, born


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_the_bounds_checked_build_does_the_same(e4m3):
    results = []
    for path in (None, _build.build(debug_bounds=True)):
        c, table, lens, q, mass, born = _whole(5, e4m3)
        state = dict(counted=(600, 0, 1500, 0), total=(900, 0, 1500, 40))
        if path is None:
            out, new = _step(c, table, lens, q, mass, born, (300, 5, 700, 20), state, sinks=4, recent=16)
        else:
            with library(path):
                out, new = _step(c, table, lens, q, mass, born, (300, 5, 700, 20), state, sinks=4, recent=16)
        results.append(_all_rows(c) + [mass.cpu().numpy(), born.cpu().numpy(), _bits(out), np.array(new)])
    for x, y in zip(*results):
        assert np.array_equal(x, y)


def test_a_captured_step_and_one_on_another_stream():
    def calls(c, table, lens, q, lse, mass, born, o, st, stream=None):
        up.up_kv_mass(q, c.k, c.v, table, lens, lse, mass, born, st, **c.scales(), stream=stream)
        up.up_kv_evict(mass, born, table, lens, o["budget"], o["moves"], o["num"], o["new"], st, sinks=4, recent=16, stream=stream)
        up.up_kv_move(c.k, c.v, table, o["moves"], o["num"], st, **c.scales(), mass=mass, born=born, stream=stream)
    results = []
    for how in ("eager", "stream", "graph"):
        c, table, lens, q, mass, born = _whole(6, True)
        _, _, lse = _run_decode(c, table, lens, q)
        o = dict(budget=_i32((300, 5, 700, 20)), moves=torch.zeros(4, 2, 750, 2, dtype=torch.int32, device="cuda"),
                 num=torch.zeros(4, 2, dtype=torch.int32, device="cuda"), new=_i32([0] * 4))
        t, n, st = torch.from_numpy(table).cuda(), _i32(lens), _status()
        torch.cuda.synchronize()
        if how == "eager":
            calls(c, t, n, q, lse, mass, born, o, st)
        elif how == "stream":
            side = torch.cuda.Stream()
            calls(c, t, n, q, lse, mass, born, o, st, side)
            side.synchronize()
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                calls(c, t, n, q, lse, mass, born, o, st)
            assert (o["new"] == 0).all()
            graph.replay()
        torch.cuda.synchronize()
        assert up.up_read_status(st) == 0
        results.append(_all_rows(c) + [mass.cpu().numpy(), born.cpu().numpy(), o["moves"].cpu().numpy(), o["num"].cpu().numpy(), o["new"].cpu().numpy()])
    for other in results[1:]:
        assert all(np.array_equal(x, y) for x, y in zip(results[0], other))


def test_what_the_binding_refuses():
    c, table, lens, q, mass, born = _whole(7, False)
    t, n, lse, st = torch.from_numpy(table).cuda(), _i32(lens), torch.zeros(4, 8, device="cuda"), _status()
    good = dict(q=q, k_cache=c.k, v_cache=c.v, block_table=t, seqused=n, lse=lse, mass=mass, born=born, dev_status=st)
    for bad in (dict(seqused=n.cpu()), dict(seqused=n.long()), dict(lse=lse[:3]), dict(lse=lse.double()), dict(mass=mass[:-1]),
                dict(born=born.long()), dict(mass_out=mass.transpose(0, 1)), dict(block_table=t[:2]), dict(counted=n[:2]), dict(q=q[..., :64])):
        with pytest.raises(AssertionError):
            up.up_kv_mass(**dict(good, **bad))
    o = dict(mass=mass, born=born, block_table=t, seqused=n, budget=n.clone(), moves=torch.zeros(4, 2, 9, 2, dtype=torch.int32, device="cuda"),
             num_moves=torch.zeros(4, 2, dtype=torch.int32, device="cuda"), new_len=_i32([0] * 4), dev_status=st)
    for bad in (dict(born=born[:, :1]), dict(moves=o["moves"][:, :1]), dict(num_moves=o["num_moves"].long()), dict(budget=n[:1]),
                dict(new_len=o["new_len"].cpu()), dict(mass=mass.transpose(0, 1))):
        with pytest.raises(AssertionError):
            up.up_kv_evict(**dict(o, **bad))
    with pytest.raises(up.UpError):
        up.up_kv_evict(**dict(o, new_len=n))
    with pytest.raises(AssertionError):
        up.up_kv_move(c.k, c.v, t, o["moves"][:2], o["num_moves"], st)
    assert up.up_read_status(st) == 0


# ------------------------------------------------------------------------------------------ far and at once

@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_rows_beyond_32_bits_of_offset(e4m3):
    """a cache of five gigabytes a side, of which the last pages are used: against the same rows in a small one"""
    lens, Hkv, B, dk = (300, 0, 77), 8, 16, 128
    small, table, rows, qb = _decode_case(11, 16, Hkv, dk, B, lens, e4m3)
    nb = 5 * (1 << 30) // (Hkv * B * dk * (1 if e4m3 else 2))
    dt = torch.uint8 if e4m3 else torch.int16
    big = type(small).__new__(type(small))
    big.e4m3, big.B, big.Hkv, big.dk, big.num_blocks = e4m3, B, Hkv, dk, nb
    far = nb - small.num_blocks
    big.k, big.v = (torch.empty(nb, Hkv, B, dk, dtype=dt, device="cuda").view(torch.float8_e4m3fn if e4m3 else torch.bfloat16) for _ in "kv")
    big.ks, big.vs = (torch.empty(nb, Hkv, B, dtype=torch.uint8, device="cuda") if e4m3 else None for _ in "kv")
    for x, y in zip((big.k, big.v, big.ks, big.vs), (small.k, small.v, small.ks, small.vs)):
        if y is not None:
            x.view(dt if y.dtype != torch.uint8 else torch.uint8)[far:] = y.view(dt if y.dtype != torch.uint8 else torch.uint8)
    results = []
    for c, up_by in ((small, 0), (big, far)):
        t = np.where((table >= 0) & (table < small.num_blocks), table + up_by, table)
        mass, born = (torch.empty(c.num_blocks, Hkv, B, dtype=x, device="cuda") for x in (torch.float32, torch.int32))
        mass[-small.num_blocks:], born[-small.num_blocks:] = 1.0, 5
        out, new = _step(c, t, lens, _from_bits(qb), mass, born, (100, 3, 40), dict(counted=(250, 0, 0), total=(400, 0, 77)), sinks=2, recent=9)
        rows_of = [x[-small.num_blocks:].clone() for x in (c.k.view(dt), c.v.view(dt), mass, born)]
        results.append((out, new, rows_of + ([c.ks[-small.num_blocks:].clone(), c.vs[-small.num_blocks:].clone()] if e4m3 else [])))
    assert torch.equal(results[0][0], results[1][0]) and results[0][1] == results[1][1]
    assert all(torch.equal(x, y) for x, y in zip(results[0][2], results[1][2]))


def test_records_beyond_32_bits_of_index():
    nb, B = 36_000_000, 64                                   # 2.3 billion records
    mass, born = torch.empty(nb, 1, B, device="cuda"), torch.empty(nb, 1, B, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(1)
    n, k = 1000, 300
    pages = np.concatenate([[nb - 1, 0, 33_600_000, 17_000_000], np.arange(nb - 14, nb - 2)]).astype(np.int32)
    m, p = rng.random(n).astype(np.float32), np.arange(n)
    at = torch.from_numpy(pages).cuda().long()[torch.from_numpy(p).cuda() // B]
    mass[at, 0, torch.from_numpy(p % B).cuda()] = torch.from_numpy(m).cuda()
    born[at, 0, torch.from_numpy(p % B).cuda()] = torch.from_numpy(p.astype(np.int32)).cuda()
    status, moves, num, new_len = _choose(mass, born, pages[None], (n,), (k,), sinks=3, recent=20)
    want = evict_ref.evict(m, p, n, k, 3, 20)
    assert status == 0 and int(new_len[0]) == k and moves[0, 0, :int(num[0, 0])].tolist() == [list(x) for x in want]


def test_two_streams_at_once():
    """two layers' steps side by side, over and over: each as it is alone"""
    alone, at_once = [], []
    for results, streams in ((alone, [None, None]), (at_once, [torch.cuda.Stream(), torch.cuda.Stream()])):
        work = []
        for i, e4m3 in enumerate((False, True)):
            lens = (3000, 0, 1500, 33) if i else (700, 9000, 1)
            c, table, rows, qb = _decode_case(20 + i, 8, 2, 128, 16, lens, e4m3)
            mass, born = _records(c, 20 + i)
            _, _, lse = _run_decode(c, table, lens, _from_bits(qb))
            out = torch.zeros_like(mass)
            n = len(lens)
            o = dict(budget=_i32([x // 2 for x in lens]), moves=torch.zeros(n, 2, 5000, 2, dtype=torch.int32, device="cuda"),
                     num=torch.zeros(n, 2, dtype=torch.int32, device="cuda"), new=_i32([0] * n))
            work.append((c, torch.from_numpy(table).cuda(), _i32(lens), _from_bits(qb), lse, mass, born, out, o, _status()))
        torch.cuda.synchronize()
        for _ in range(10):
            for (c, t, n, q, lse, mass, born, out, o, st), stream in zip(work, streams):
                up.up_kv_mass(q, c.k, c.v, t, n, lse, mass, born, st, **c.scales(), mass_out=out, stream=stream)
                up.up_kv_evict(out, born, t, n, o["budget"], o["moves"], o["num"], o["new"], st, sinks=4, recent=16, stream=stream)
                up.up_kv_move(c.k, c.v, t, o["moves"], o["num"], st, **c.scales(), stream=stream)
        torch.cuda.synchronize()
        for c, t, n, q, lse, mass, born, out, o, st in work:
            assert up.up_read_status(st) == 0
            results.append([out.cpu().numpy(), o["num"].cpu().numpy(), o["new"].cpu().numpy()] + _all_rows(c))
    for x, y in zip(alone, at_once):
        assert all(np.array_equal(a, b, equal_nan=a.dtype.kind == "f") for a, b in zip(x, y))
