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
