"""A StackCache that ran full, and its next prefill (GPU)."""
import pytest
import torch

from long_context_prefill_varlen_gb300 import layerstack as ls

pytestmark = pytest.mark.gpu

GEOM = ls.StackGeometry(d=256, Hq=4, Hkv=2, dk=64, ffn=512)
L = 2


def _prefill(stack, cache, lengths, seed=1):
    g = torch.Generator().manual_seed(seed)
    hidden = torch.randn(sum(lengths), GEOM.d, generator=g).to(torch.bfloat16).cuda()
    positions = torch.cat([torch.arange(n) for n in lengths]).cuda()
    cu = torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32).cuda()
    return stack.forward(hidden, positions, cu, max(lengths), cache=cache)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_a_cache_that_ran_full_takes_the_next_prefill(e4m3):
    stack = ls.RandomLlamaStack(L, GEOM, seed=3, device="cuda", init_device="cpu")
    cache, fresh = (ls.StackCache(L, 2, GEOM.Hkv, GEOM.dk, 32, e4m3=e4m3) for _ in range(2))
    _prefill(stack, cache, (32, 7))
    token = torch.randn(2, GEOM.d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    stack.decode(token, torch.tensor([32, 7], device="cuda"), cache)         # the first request's 33rd
    with pytest.raises(RuntimeError):
        cache.check()
    outs = []
    for c in (cache, fresh):
        _prefill(stack, c, (20, 30), seed=2)
        outs.append(stack.decode(token, torch.tensor([20, 30], device="cuda"), c))
        c.check()
    assert torch.equal(outs[0], outs[1])


def test_a_prefill_longer_than_its_cache_raises():
    stack = ls.RandomLlamaStack(L, GEOM, seed=3, device="cuda", init_device="cpu")
    cache = ls.StackCache(L, 2, GEOM.Hkv, GEOM.dk, 32)
    with pytest.raises(RuntimeError):
        _prefill(stack, cache, (40, 7))
    _prefill(stack, cache, (32, 7))
