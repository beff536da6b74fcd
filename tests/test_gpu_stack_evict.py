"""Eviction and planned rotary positions inside the random-weight decoder stack (GPU).

Each decode step is checked against a float64 CPU recomputation that attends over what the cache holds (read back head by
head through up_kv_read), with the stack tests' tolerances; a budget that takes nothing out changes no bit; a layer's stream and
the sinks stay what they are however often tokens go."""
import numpy as np
import pytest
import torch

from long_context_prefill_varlen_gb300 import layerstack as ls, up_read_status
from synth import cpu as gen
from synth import gpu as sgpu
from synth import recipe
from tests import evict_ref, kv_ref, stack_ref
from tests.test_gpu_generate import A, G, GEOM, L, LENGTHS, REL_FRO, REL_ROW, _read, _ref_decode, n
from tests.test_gpu_kvcache import _bits
from tests.test_gpu_rope import _turns

pytestmark = pytest.mark.gpu


def _prefill(e4m3, drops, weigh, geom=GEOM, lengths=LENGTHS):
    w = recipe.small(lengths=lengths, Hq=geom.Hq, Hkv=geom.Hkv, dk=geom.dk, hdim=geom.d, G=G, n=n, A=A, salt=257)
    d = sgpu.to_device(gen.materialize(w))
    stack = ls.RandomLlamaStack(L, geom, seed=11, device="cuda", init_device="cpu")
    cache = ls.StackCache(L, len(lengths), geom.Hkv, geom.dk, max(lengths) + 8, e4m3=e4m3, weigh=weigh)
    out, info = stack.forward(d["hidden"], d["positions"], d["cu_seqlens"], max(lengths), drops=drops, G=G, n=n, A=A, cache=cache)
    return stack, cache, out, info


def _steps(seed, count, lengths=LENGTHS):
    rng = np.random.default_rng(seed)
    for i in range(count):
        hidden = torch.from_numpy(rng.standard_normal((len(lengths), GEOM.d)).astype(np.float32)).cuda().to(torch.bfloat16)
        yield hidden, torch.tensor(lengths, device="cuda") + i


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("drops", [[], [(1, 0.8)]], ids=["none", "one"])
def test_decoding_from_a_cache_that_rows_leave(drops, e4m3):
    stack, cache, _, _ = _prefill(e4m3, drops, True)
    R, sinks, recent = len(LENGTHS), 4, 16
    budgets = [None, 600, None, torch.tensor([500, 40, 3, 700, 0], dtype=torch.int32, device="cuda"), 20]
    held = [cache.seqused(layer).cpu().numpy().astype(int) for layer in range(L)]
    had = [x.copy() for x in held]
    for step, (hidden, pos) in enumerate(_steps(3, len(budgets))):
        got = stack.decode(hidden, pos, cache).double().cpu()
        cache.check()
        for layer in range(L):
            held[layer] += 1
            had[layer] += 1
            assert np.array_equal(cache.rows(layer, cache.seqused(layer)).cpu().numpy(), held[layer])
        ref = _ref_decode(stack, hidden, pos.cpu(), [_read(cache, layer, list(held[layer])) for layer in range(L)])
        fro = float(torch.linalg.norm(got - ref) / torch.linalg.norm(ref))
        rows = (torch.linalg.norm(got - ref, dim=1) / torch.linalg.norm(ref, dim=1)).max()
        assert fro < REL_FRO and float(rows) < REL_ROW, (step, fro, float(rows))
        for layer in range(L):
            mass, born = (x.cpu().numpy() for x in cache.records[layer])
            for r in range(R):
                p = np.arange(held[layer][r])
                page = cache.block_table[r].cpu().numpy()[p // cache.B]
                b, m = born[page, :, p % cache.B], mass[page, :, p % cache.B]
                assert all(len(set(b[:, h])) == len(p) for h in range(GEOM.Hkv)) and (b < had[layer][r]).all()
                assert np.isfinite(m).all() and (m >= 0).all()
                if step == 0:                      # a head's weights add up to its query heads (twice: the prompt's last
                    assert np.array_equal(b, np.tile(p[:, None], (1, GEOM.Hkv)))               # token had some, too)
                    assert np.allclose(m.sum(0), (2 if len(p) > 1 else 1) * (GEOM.Hq // GEOM.Hkv), rtol=1e-4)
        if budgets[step] is not None:
            cache.evict(budgets[step], sinks=sinks, recent=recent)
            cache.check()
            k = np.full(R, budgets[step]) if isinstance(budgets[step], int) else budgets[step].cpu().numpy()
            for layer in range(L):
                held[layer] = np.minimum(held[layer], k)
                born = cache.records[layer][1].cpu().numpy()
                for r in range(R):
                    p = np.arange(held[layer][r])
                    b = born[cache.block_table[r].cpu().numpy()[p // cache.B], :, p % cache.B]
                    for h in range(GEOM.Hkv):
                        if len(p) >= sinks + recent:
                            t = had[layer][r]
                            assert set(range(min(sinks, t))) | set(range(max(0, t - recent), t)) <= set(b[:, h].tolist())


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_weighing_alone_and_a_large_budget_change_nothing(e4m3):
    outs = []
    for weigh in (False, True):
        stack, cache, _, _ = _prefill(e4m3, [(1, 0.8)], weigh)
        got = []
        for hidden, pos in _steps(5, 3):
            got.append(stack.decode(hidden, pos, cache))
            if weigh:
                cache.evict(10_000, sinks=4, recent=4)
        cache.check()
        outs.append((got, cache))
    for x, y in zip(outs[0][0], outs[1][0]):
        assert torch.equal(x, y)
    for (k0, v0, _), (k1, v1, _) in zip(outs[0][1].layers, outs[1][1].layers):
        assert torch.equal(k0.view(torch.uint8), k1.view(torch.uint8)) and torch.equal(v0.view(torch.uint8), v1.view(torch.uint8))


def test_a_new_prefill_forgets_what_was_evicted():
    stack, cache, _, _ = _prefill(True, [], True)
    for hidden, pos in _steps(6, 2):
        stack.decode(hidden, pos, cache)
        cache.evict(50)
    w = recipe.small(lengths=LENGTHS, Hq=GEOM.Hq, Hkv=GEOM.Hkv, dk=GEOM.dk, hdim=GEOM.d, G=G, n=n, A=A, salt=257)
    d = sgpu.to_device(gen.materialize(w))
    stack.forward(d["hidden"], d["positions"], d["cu_seqlens"], max(LENGTHS), cache=cache)
    fresh = _prefill(True, [], True)[1]
    for hidden, pos in _steps(7, 2):
        a, b = stack.decode(hidden, pos, cache), stack.decode(hidden, pos, fresh)
        assert torch.equal(a, b)
    for layer in range(L):
        rows = cache.rows(layer, cache.seqused(layer)).cpu().numpy()
        for r in range(len(LENGTHS)):
            p = np.arange(rows[r])
            page = cache.block_table[r].cpu().numpy()[p // cache.B]
            for x, y in zip(cache.records[layer], fresh.records[layer]):
                assert np.array_equal(x.cpu().numpy()[page, :, p % cache.B], y.cpu().numpy()[page, :, p % cache.B])


@pytest.mark.parametrize("how", [dict(), dict(layout="pairs", rot=32), dict(scaling="bands", factor=8.0, original_len=512)],
                         ids=["plain", "pairs_of_a_part", "bands"])
def test_the_stacks_planned_positions(how):
    """q and k of a layer are the projections turned by the plan; without scaling, the stack gives what 32-bit angles give, to the
    stack tests' tolerances"""
    geom = ls.with_rope(GEOM, **how)
    stack = ls.RandomLlamaStack(L, geom, seed=11, device="cuda", init_device="cpu")
    base = ls.RandomLlamaStack(L, ls.with_rope(GEOM), seed=11, device="cuda", init_device="cpu")
    w = recipe.small(lengths=LENGTHS, Hq=GEOM.Hq, Hkv=GEOM.Hkv, dk=GEOM.dk, hdim=GEOM.d, G=G, n=n, A=A, salt=257)
    host = gen.materialize(w)
    d = sgpu.to_device(host)
    q0, k0, v0 = base.qkv(0, d["hidden"], torch.zeros_like(d["positions"]))        # position 0 turns nothing
    q, k, v = stack.qkv(0, d["hidden"], d["positions"])
    assert torch.equal(v, v0)
    turns = _turns(geom.rope, d["positions"].tolist())
    for x, x0 in ((q, q0), (k, k0)):
        y, tol = evict_ref.turned(kv_ref.bf16_value(_bits(x0)), turns, geom.rope.gain, how.get("layout", "halves"))
        assert (np.abs(kv_ref.bf16_value(_bits(x)) - y) <= tol).all()
    if not how:
        out, _ = stack.forward(d["hidden"], d["positions"], d["cu_seqlens"], max(LENGTHS))
        hidden = torch.from_numpy(gen.bf16_bits_to_f32(host["hidden"]).astype(np.float64))
        ref = stack_ref.forward(stack, hidden, host["positions"], LENGTHS)
        got = out.double().cpu()
        assert float(torch.linalg.norm(got - ref) / torch.linalg.norm(ref)) < REL_FRO


def test_eviction_makes_room_in_a_full_cache():
    lengths = (16, 40)
    stack, cache, _, _ = _prefill(True, [], True, lengths=lengths)             # three pages of 16 for the longer request
    steps = _steps(8, 20, lengths)
    for _ in range(8):
        stack.decode(*next(steps), cache)
    cache.check()
    cache.evict(np.int64(30), recent=8)
    for _ in range(12):                                                        # 30 tokens grow to 42
        stack.decode(*next(steps), cache)
    cache.check()
    assert cache.rows(0, cache.seqused(0)).tolist() == [16 + 20, 30 + 12] and cache.seqused(0).tolist() == [36, 60]


def test_eviction_right_after_the_prefill():
    """by the weights of each request's last token, which the float64 recomputation of the drop layer's scores has as well"""
    stack, cache, _, info = _prefill(False, [(1, 0.8)], True)
    before = [_read(cache, layer, cache.seqused(layer).tolist()) for layer in range(L)]
    w = recipe.small(lengths=LENGTHS, Hq=GEOM.Hq, Hkv=GEOM.Hkv, dk=GEOM.dk, hdim=GEOM.d, G=G, n=n, A=A, salt=257)
    d = sgpu.to_device(gen.materialize(w))
    _, info = stack.forward(d["hidden"], d["positions"], d["cu_seqlens"], max(LENGTHS), drops=[(1, 0.8)], G=G, n=n, A=A, keep_scored=True)
    q = info[0]["scored"][0].double().cpu()
    mass, _ = cache.records[1]
    for r, N in enumerate(LENGTHS):
        for hq in range(GEOM.Hq if N else 0):
            at = sum(LENGTHS[:r + 1]) - 1
            k = before[1][0][r][:, hq // 2]
            p = torch.softmax(k @ q[at, hq] * GEOM.dk ** -0.5, 0)
            if hq % 2 == 0:
                want = p
            else:
                page = cache.block_table[r].long()[torch.arange(N, device="cuda") // cache.B]
                got = mass[page, hq // 2, torch.arange(N, device="cuda") % cache.B].double().cpu()
                assert torch.allclose(got, want + p, rtol=1e-4, atol=1e-9)
    cache.evict(64, sinks=4, recent=16)
    cache.check()
    for layer in range(L):
        had = torch.tensor([len(x) for x in before[layer][0]])
        assert cache.rows(layer, cache.seqused(layer)).tolist() == had.clamp(max=64).tolist()
    hidden, pos = next(_steps(9, 1))
    got = stack.decode(hidden, pos, cache).double().cpu()
    cache.check()
    rows = [cache.rows(layer, cache.seqused(layer)).tolist() for layer in range(L)]
    ref = _ref_decode(stack, hidden, pos.cpu(), [_read(cache, layer, rows[layer]) for layer in range(L)])
    assert float(torch.linalg.norm(got - ref) / torch.linalg.norm(ref)) < REL_FRO


def test_a_request_that_has_outgrown_the_cache_keeps_its_rows():
    """one step too many, then an eviction: the request's rows and records stay, the other request's go, and the coming steps have
    what they have without the eviction where it takes nothing"""
    lengths, outs = (16, 40), []
    for evict in (False, True):
        stack, cache, _, _ = _prefill(True, [], True, lengths=lengths)         # 48 rows a request
        steps = _steps(8, 11, lengths)
        for _ in range(9):
            stack.decode(*next(steps), cache)
        assert up_read_status(cache.status) != 0                               # 49 tokens
        pages = cache.block_table[1].long()

        def held():
            tensors = [x for k, v, s in cache.layers for x in (k.view(torch.uint8), v.view(torch.uint8), *s.values())]
            return [x[pages].clone() for x in tensors + [x for pair in cache.records for x in pair]]
        before = held()
        if evict:
            cache.evict(20, recent=4)
            assert cache.evicted.tolist() == [[5, 0]] * L and all(torch.equal(x, y) for x, y in zip(before, held()))
            assert [cache.rows(layer, cache.seqused(layer)).tolist() for layer in range(L)] == [[20, 49]] * L
        outs.append([stack.decode(*next(steps), cache) for _ in range(2)])
        with pytest.raises(RuntimeError):
            cache.check()
    for x, y in zip(*outs):
        assert torch.equal(x[1], y[1])


def test_attention_without_the_number_of_tokens():
    """a new row's number is that in the layer's stream, after an eviction too"""
    stack, cache, _, _ = _prefill(True, [], True, lengths=(16, 40))
    stack.decode(*next(_steps(8, 1, (16, 40))), cache)
    cache.evict(10)
    cache.kv_len.add_(1)
    q = torch.randn(2, GEOM.Hq, GEOM.dk, device="cuda").to(torch.bfloat16)
    for layer, how in enumerate(("rows", "seqused", "both")):
        seqused = cache.seqused(layer)
        rows = cache.rows(layer, seqused)
        assert rows.tolist() == [11, 11]
        cache.attend(layer, q, **{"rows": dict(rows=rows), "seqused": dict(seqused=seqused), "both": dict(rows=rows, seqused=seqused)}[how])
        born = cache.records[layer][1][cache.block_table[:, 0].long(), :, 10]
        assert born.tolist() == [[17] * GEOM.Hkv, [41] * GEOM.Hkv] and cache.counted[layer].tolist() == [11, 11]
    cache.check()


def test_a_captured_step_with_its_eviction():
    """replayed, it is what the calls give one after another (positions by a plan: the 32-bit angles' base comes from the host)"""
    lengths, inputs, geom = (16, 40), list(_steps(8, 5, (16, 40))), ls.with_rope(GEOM)
    stack, cache, _, _ = _prefill(True, [(1, 0.8)], True, geom, lengths)
    want = []
    for hidden, pos in inputs:
        want.append(stack.decode(hidden, pos, cache).clone())
        cache.evict(24, sinks=2, recent=8)
    cache.check()
    again = _prefill(True, [(1, 0.8)], True, geom, lengths)[1]
    hidden, pos = inputs[0][0].clone(), inputs[0][1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = stack.decode(hidden, pos, again)
        again.evict(24, sinks=2, recent=8)
    for (h, p), y in zip(inputs, want):
        hidden.copy_(h)
        pos.copy_(p)
        graph.replay()
        assert torch.equal(out, y)
    again.check()
    assert torch.equal(again.evicted, cache.evicted) and torch.equal(again.counted, cache.counted)
    for (m0, b0), (m1, b1), (k0, v0, _), (k1, v1, _) in zip(cache.records, again.records, cache.layers, again.layers):
        assert torch.equal(m0, m1) and torch.equal(b0, b1)
        assert torch.equal(k0.view(torch.uint8), k1.view(torch.uint8)) and torch.equal(v0.view(torch.uint8), v1.view(torch.uint8))
