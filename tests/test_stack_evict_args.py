"""What a StackCache refuses of an eviction, on the host and before any work (no GPU needed)."""
import pytest
import torch

from long_context_prefill_varlen_gb300 import layerstack as ls


def _cache(weigh):
    return ls.StackCache(3, 2, 1, 64, 16, device="cpu", weigh=weigh)


def test_a_cache_without_records_and_one_without_weights():
    with pytest.raises(ValueError, match="weigh"):
        _cache(False).evict(4)
    with pytest.raises(ValueError, match="weights"):
        _cache(True).evict(4)
    cache = _cache(True)
    cache.weighed = True
    with pytest.raises(ValueError, match="budget"):
        cache.evict(-1)
    cache.start(torch.tensor([0, 3, 7], dtype=torch.int32))
    with pytest.raises(ValueError, match="weights"):
        cache.evict(4)


def test_a_cache_without_records_holds_all_that_its_layers_had():
    n = torch.tensor([3, 4], dtype=torch.int32)
    assert _cache(False).rows(1, n) is n
    cache = _cache(True)
    cache.evicted[1] = torch.tensor([1, 0], dtype=torch.int32)
    assert cache.rows(1, n).tolist() == [2, 4] and cache.rows(0, n).tolist() == [3, 4]
    cache.start(torch.tensor([0, 3, 7], dtype=torch.int32))
    assert cache.rows(1, n).tolist() == [3, 4]


def test_a_geometry_with_a_plan():
    from long_context_prefill_varlen_gb300 import _build
    _build.build()
    geom = ls.with_rope(ls.LLAMA_3_1_8B, scaling="bands", factor=8.0, original_len=8192)
    assert (geom.rope.rot, geom.rope.layout, geom.rope.gain) == (128, 0, 1.0) and ls.LLAMA_3_1_8B.rope is None
    assert geom.d == ls.LLAMA_3_1_8B.d and ls.with_rope(geom, rot=32, layout="pairs").rope.rot == 32


def test_a_prompt_of_no_tokens_weighs_nothing(monkeypatch):
    """(there is no last token to take)"""
    class Cache(ls.StackCache):
        def slots(self, cu, T):
            return None

        def write(self, *a):
            pass

        def check(self, stream=None):
            pass

        def attend(self, *a):
            raise AssertionError("weighed")
    monkeypatch.setattr(ls, "varlen_causal_attention", lambda q, *a: q)
    geom = ls.StackGeometry(d=64, Hq=2, Hkv=1, dk=64, ffn=64)
    cache = Cache(1, 2, 1, 64, 16, device="cpu", weigh=True)
    stack = ls.RandomLlamaStack(1, geom, device="cpu")
    h = torch.empty(0, 64, dtype=torch.bfloat16)
    out, _ = stack.forward(h, torch.empty(0, dtype=torch.int64), torch.zeros(3, dtype=torch.int32), 0, cache=cache)
    assert out.shape == (0, 64) and cache.weighed
    with pytest.raises(AssertionError, match="weighed"):
        stack.forward(torch.zeros(3, 64, dtype=torch.bfloat16), torch.arange(3), torch.tensor([0, 3, 3], dtype=torch.int32), 3,
                      cache=cache)


class _Calls:
    """What an eviction on the CPU asks of the library, answered by up_kv_evict's rules for a request's length."""

    def __init__(self, monkeypatch, had):
        self.budgets, self.rows = [], []
        monkeypatch.setattr(ls, "up_seqused", lambda kept, drop, layer, orig, kv_len, out: out.copy_(torch.tensor(had[layer])))
        monkeypatch.setattr(ls, "up_kv_evict", self.evict)
        monkeypatch.setattr(ls, "up_kv_move", lambda *a, **kw: None)

    def evict(self, mass, born, table, rows, budget, moves, num, new_len, status, total, sinks, recent):
        cap = table.shape[1] * mass.shape[2]
        self.budgets.append(budget.tolist())
        self.rows.append(rows.tolist())
        new_len.copy_(torch.where((rows < 0) | (rows > cap), 0, torch.minimum(rows, budget)))


def test_a_request_that_has_outgrown_the_cache_keeps_its_rows(monkeypatch):
    """(tables of 16 rows)"""
    calls = _Calls(monkeypatch, [[17, 10], [12, 3], [40, 30]])
    cache = _cache(True)
    cache.weighed = True
    cache.evicted[2] = torch.tensor([20, 20], dtype=torch.int32)         # of its 40 tokens a layer still holds 20
    cache.evict(8)
    assert calls.rows == [[17, 10], [12, 3], [20, 10]]
    assert cache.evicted.tolist() == [[0, 2], [4, 0], [20, 22]]
    cache.evict(8)                                                       # nor does it a second time
    assert calls.rows[3:] == [[17, 8], [8, 3], [20, 8]] and cache.evicted.tolist() == [[0, 2], [4, 0], [20, 22]]


@pytest.mark.parametrize("budget", [16, 17, (1 << 31) - 1, 1 << 31, 1 << 40])
def test_a_budget_of_any_size(monkeypatch, budget):
    """more than the cache holds is all of it"""
    calls = _Calls(monkeypatch, [[16, 10], [12, 3], [0, 1]])
    cache = _cache(True)
    cache.weighed = True
    cache.evict(budget)
    assert calls.budgets == [[16, 16]] * 3 and not cache.evicted.any()


@pytest.mark.parametrize("weigh", [False, True])
def test_attention_by_the_rows_or_by_the_tokens(monkeypatch, weigh):
    """either gives the other, what was evicted between them"""
    asked = []
    monkeypatch.setattr(ls, "up_paged_decode_workspace_bytes", lambda *a: 16)
    monkeypatch.setattr(ls, "up_paged_decode", lambda q, k, v, table, rows, *a, sm_scale, **kw: asked.append((rows.tolist(), sm_scale)))
    monkeypatch.setattr(ls, "up_kv_mass", lambda q, k, v, table, rows, *a, sm_scale, counted, total, **kw: asked.append(
        (rows.tolist(), sm_scale, counted.tolist(), total.tolist())))
    cache, q = _cache(weigh), torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    gone = torch.tensor([3, 0], dtype=torch.int32)
    if weigh:
        cache.evicted[1] = gone
    had = torch.tensor([9, 5], dtype=torch.int32)
    rows = had - gone if weigh else had
    for how in (dict(rows=rows), dict(seqused=had), dict(rows=rows, seqused=had)):
        asked.clear()
        cache.attend(1, q, sm_scale=0.5, **how)
        if weigh:
            assert asked == [(rows.tolist(), 0.5), (rows.tolist(), 0.5, [0, 0], had.tolist())]
            assert cache.counted.tolist() == [[0, 0], rows.tolist(), [0, 0]]
            cache.counted.zero_()
        else:
            assert asked == [(rows.tolist(), 0.5)]
    with pytest.raises(ValueError, match="rows or seqused"):
        cache.attend(1, q, sm_scale=0.5)
