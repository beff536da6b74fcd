"""Prefill with drops into a paged cache, then decoding from it (GPU): the cache's operators inside the
random-weight decoder stack, UniPrefill section 3.5, Eqs. 16-17.

Each layer's decode is checked against a float64 CPU recomputation that attends over what the cache holds
(read back through up_kv_read), with the stack tests' tolerances for bf16 activations through four layers;
the cached rows are checked against the keys the prefill computed."""
import numpy as np
import pytest
import torch

import long_context_prefill_varlen_gb300 as up
from long_context_prefill_varlen_gb300 import layerstack as ls
from synth import cpu as gen
from synth import gpu as sgpu
from synth import recipe
from tests import stack_ref

pytestmark = pytest.mark.gpu

GEOM = ls.StackGeometry(d=256, Hq=4, Hkv=2, dk=64, ffn=512)
LENGTHS = (1500, 700, 0, 2100, 90)
L, G, n, A = 4, 64, 128, 128
REL_FRO, REL_ROW = 2e-2, 6e-2          # those of test_gpu_stack.py


def _prefill(e4m3, drops, lengths=LENGTHS, B=16, salt=257):
    w = recipe.small(lengths=lengths, Hq=GEOM.Hq, Hkv=GEOM.Hkv, dk=GEOM.dk, hdim=GEOM.d, G=G, n=n, A=A, salt=salt)
    d = sgpu.to_device(gen.materialize(w))
    stack = ls.RandomLlamaStack(L, GEOM, seed=11, device="cuda", init_device="cpu")
    cache = ls.StackCache(L, len(lengths), GEOM.Hkv, GEOM.dk, max(lengths) + 8, B=B, e4m3=e4m3)
    out, info = stack.forward(d["hidden"], d["positions"], d["cu_seqlens"], max(lengths), drops=drops, G=G, n=n, A=A,
                              keep_scored=True, cache=cache)
    cache.check()
    return d, stack, cache, out, info


def _read(cache, layer, lens):
    """what the layer's cache holds for every request: lists of float64 [len, Hkv, dk]"""
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    T = int(sum(lens))
    kc, vc, scales = cache.layers[layer]
    k, v = (torch.empty(T, GEOM.Hkv, GEOM.dk, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    up.up_kv_read(kc, vc, cache.slots(cu, T), k, v, cache.status, **scales)
    cache.check()
    return [[x.double() for x in t.cpu().split(list(lens))] for t in (k, v)]


def _ref_decode(stack, hidden, positions, cached):
    """float64 on the CPU: cached[layer] = (k lists, v lists), the new token's own row included"""
    g, h = stack.g, hidden.double().cpu()
    for layer in range(stack.L):
        a = stack_ref._rms(h, g.eps)
        R = h.shape[0]
        q = stack_ref._rope(torch.matmul(a, stack_ref._w(stack, layer, "wq")).view(R, g.Hq, g.dk), positions, g.dk, g.rope_theta)
        o = torch.zeros(R, g.Hq, g.dk, dtype=torch.float64)
        for r in range(R):
            for hq in range(g.Hq):
                k, v = (cached[layer][i][r][:, hq // (g.Hq // g.Hkv)] for i in (0, 1))
                o[r, hq] = torch.softmax(k @ q[r, hq] * g.dk ** -0.5, 0) @ v
        x = h + torch.matmul(o.view(R, -1), stack_ref._w(stack, layer, "wo"))
        h = stack_ref.ffn_sublayer(stack, layer, x)
    return h


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("drops", [[], [(1, 0.8)], [(0, 0.9), (2, 0.8)]], ids=["none", "one", "two"])
def test_decoding_after_a_prefill_with_drops(drops, e4m3):
    d, stack, cache, _, info = _prefill(e4m3, drops)
    R = len(LENGTHS)
    rng = np.random.default_rng(3)
    # a layer holds what the last drop below it kept
    kept = [np.array(LENGTHS)]
    for layer in range(1, L):
        here = [i for i in info if i["layer"] < layer]
        kept.append(np.array(here[-1]["step"].new_len.cpu().numpy() if here else LENGTHS))
    for layer in range(L):
        assert np.array_equal(cache.seqused(layer).cpu().numpy(), kept[layer])
    for step in range(3):
        hidden = torch.from_numpy(rng.standard_normal((R, GEOM.d)).astype(np.float32)).cuda().to(torch.bfloat16)
        pos = torch.tensor(LENGTHS, device="cuda") + step
        got = stack.decode(hidden, pos, cache).double().cpu()
        cache.check()
        lens = [k + step + 1 for k in kept]
        for layer in range(L):
            assert np.array_equal(cache.seqused(layer).cpu().numpy(), lens[layer])
        ref = _ref_decode(stack, hidden, pos.cpu(), [_read(cache, layer, lens[layer]) for layer in range(L)])
        fro = float(torch.linalg.norm(got - ref) / torch.linalg.norm(ref))
        rows = (torch.linalg.norm(got - ref, dim=1) / torch.linalg.norm(ref, dim=1)).max()
        assert fro < REL_FRO and float(rows) < REL_ROW, (fro, float(rows))


def test_the_cache_holds_the_prefills_keys_and_they_score_alike():
    """bf16 cache: the rows read back are the keys the drop layer was scored on, bit for bit, so the block
    scores of the stream read back from the cache are those of the prefill."""
    d, stack, cache, _, info = _prefill(False, [(1, 0.8)], B=24)
    q, k, x, pos = info[0]["scored"]
    T = k.shape[0]
    kc, vc, _ = cache.layers[1]
    back = torch.empty_like(k)
    up.up_kv_read(kc, vc, cache.slots(d["cu_seqlens"], T), back, None, cache.status)
    cache.check()
    assert torch.equal(back.view(torch.int16), k.contiguous().view(torch.int16))
    step = info[0]["step"]
    again = up.DropStep(d["cu_seqlens"], T, GEOM.Hq, GEOM.Hkv, GEOM.dk, GEOM.d, G=G, n=n, A=A, p=0.8)
    again.score(q, back)
    again.select()
    assert torch.equal(again.block_scores, step.block_scores) and torch.equal(again.token_keep, step.token_keep)


def test_decoding_a_token_equals_prefilling_it():
    """without drops, in a bf16 cache: the output of the last token of a prefill of N + 1 tokens"""
    lengths = (1025, 300, 1)
    w = recipe.small(lengths=lengths, Hq=GEOM.Hq, Hkv=GEOM.Hkv, dk=GEOM.dk, hdim=GEOM.d, G=G, n=n, A=A, salt=77)
    d = sgpu.to_device(gen.materialize(w))
    stack = ls.RandomLlamaStack(L, GEOM, seed=11, device="cuda", init_device="cpu")
    full, _ = stack.forward(d["hidden"], d["positions"], d["cu_seqlens"], max(lengths))
    cu = np.concatenate([[0], np.cumsum(lengths)])
    last = torch.from_numpy(cu[1:] - 1).cuda()
    keep = torch.ones(w.T, dtype=torch.bool)
    keep[torch.from_numpy(cu[1:] - 1)] = False
    short = torch.tensor(np.concatenate([[0], np.cumsum(np.array(lengths) - 1)]), dtype=torch.int32, device="cuda")
    cache = ls.StackCache(L, len(lengths), GEOM.Hkv, GEOM.dk, max(lengths), e4m3=False)
    stack.forward(d["hidden"][keep.cuda()], d["positions"][keep.cuda()], short, max(lengths), cache=cache)
    got = stack.decode(d["hidden"][last], d["positions"][last], cache).double()
    cache.check()
    want = full[last].double()
    fro = float(torch.linalg.norm(got - want) / torch.linalg.norm(want))
    rows = (torch.linalg.norm(got - want, dim=1) / torch.linalg.norm(want, dim=1)).max()
    assert fro < REL_FRO and float(rows) < REL_ROW, (fro, float(rows))


def test_a_cache_that_is_full_reports_it():
    d, stack, cache, _, _ = _prefill(True, [], lengths=(16, 40), salt=5)
    hidden = torch.zeros(2, GEOM.d, dtype=torch.bfloat16, device="cuda")
    for i in range(8):
        stack.decode(hidden, torch.tensor([16 + i, 40 + i], device="cuda"), cache)
    cache.check()                                  # 48 tokens fill the three pages of the longer request
    stack.decode(hidden, torch.tensor([24, 48], device="cuda"), cache)
    with pytest.raises(RuntimeError):
        cache.check()
