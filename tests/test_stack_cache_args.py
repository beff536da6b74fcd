"""What the decoder stack refuses of a StackCache, on the host and before any work (no GPU needed)."""
import pytest
import torch

from long_context_prefill_varlen_gb300 import layerstack as ls

GEOM = ls.StackGeometry(d=64, Hq=2, Hkv=1, dk=64, ffn=64)
L, R = 3, 2


@pytest.fixture(scope="module")
def stack():
    from long_context_prefill_varlen_gb300 import _build
    _build.build()
    return ls.RandomLlamaStack(L, GEOM, device="cpu")


def _cache(L=L, R=R):
    return ls.StackCache(L, R, GEOM.Hkv, GEOM.dk, 16, device="cpu")


def _forward(stack, cache, lengths=(3, 4), **kw):
    cu = torch.tensor((0,) + lengths).cumsum(0).to(torch.int32)
    T = sum(lengths)
    return stack.forward(torch.zeros(T, GEOM.d, dtype=torch.bfloat16), torch.zeros(T, dtype=torch.int64), cu, max(lengths), cache=cache, **kw)


def test_a_prefill_of_the_first_layers_alone(stack):
    """the layers above would decode over rows that nobody wrote"""
    for upto in (0, 1, L - 1):
        with pytest.raises(ValueError, match="upto"):
            _forward(stack, _cache(), upto=upto)


def _decode(stack, cache, rows, positions=None):
    return stack.decode(torch.zeros(rows, GEOM.d, dtype=torch.bfloat16), torch.zeros(positions or rows, dtype=torch.int64), cache)


@pytest.mark.parametrize("lengths", [(5,), (5, 0, 1)])
def test_a_batch_or_a_stack_of_another_size(stack, lengths):
    """one request's lengths would stand for every request's, and a step's slots run past their buffer"""
    cu = torch.tensor((0,) + lengths).cumsum(0).to(torch.int32)
    with pytest.raises(ValueError, match="requests"):
        _cache().start(cu)
    with pytest.raises(ValueError, match="requests"):
        _forward(stack, _cache(), lengths)
    with pytest.raises(ValueError, match="requests"):
        _decode(stack, _cache(), len(lengths))
    with pytest.raises(ValueError, match="layers"):
        _forward(stack, _cache(L=L + 1))
    with pytest.raises(ValueError, match="layers"):
        _decode(stack, _cache(L=L - 1), R)
    with pytest.raises(ValueError, match="positions"):
        _decode(stack, _cache(), R, R + 1)


def test_a_refused_step_leaves_the_cache_as_it_was(stack):
    cache = _cache()
    with pytest.raises(ValueError):
        _decode(stack, cache, R + 1)
    assert (cache.kv_len == 0).all()
