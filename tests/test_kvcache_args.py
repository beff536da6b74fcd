"""What the paged cache's entry points refuse, before anything is launched (no GPU needed), and the 64-bit
reference of their GPU tests against closed forms."""
import ctypes

import numpy as np
import pytest
import torch

from tests import kv_ref


@pytest.fixture(scope="module")
def up():
    from long_context_prefill_varlen_gb300 import _build
    _build.build()
    import long_context_prefill_varlen_gb300 as m
    m.load_library()
    return m


A, ODD = 0x1000, 0x1008        # never dereferenced


def _cache(up, **kw):
    f = dict(k=A, v=A, k_scale=A, v_scale=A, num_blocks=8, stride_block=16 * 2 * 128, stride_head=16 * 128,
             stride_token=128, Hkv=2, B=16, dk=128, format=up.KV_BF16)
    f.update(kw)
    return up._KvCache(*(f[n] for n, _ in up._KvCache._fields_))


BAD_CACHES = [
    (dict(k=None), "ARG"), (dict(v=None), "ARG"), (dict(num_blocks=0), "ARG"), (dict(B=0), "ARG"), (dict(Hkv=0), "ARG"),
    (dict(num_blocks=1 << 31), "ARG"), (dict(format=2), "ARG"), (dict(format=1, k_scale=None), "ARG"),
    (dict(dk=96), "SHAPE"), (dict(k=ODD), "SHAPE"), (dict(v=ODD), "SHAPE"), (dict(stride_token=129), "SHAPE"),
    (dict(stride_head=-128), "SHAPE"), (dict(format=1, v_scale=ODD), "SHAPE"), (dict(format=1, stride_token=136), "SHAPE"),
]


@pytest.mark.parametrize("bad,code", BAD_CACHES, ids=lambda x: str(x))
def test_bad_caches_are_refused_by_every_call(up, bad, code):
    lib, want = up.load_library(), getattr(up, "UP_ERR_" + code)
    c = ctypes.byref(_cache(up, **bad))
    assert lib.up_kv_write(c, A, 256, A, 256, A, 4, None, A, None) == want
    assert lib.up_kv_read(c, A, 4, None, A, A, A, None) == want
    assert lib.up_paged_decode(A, 512, c, A, A, 2, 4, 4, 0.1, 0, A, None, A, 1 << 40, A, None) == want


def test_bad_arguments_of_write_and_read(up):
    lib, c = up.load_library(), ctypes.byref(_cache(up))
    assert lib.up_kv_write(None, A, 256, A, 256, A, 4, None, A, None) == up.UP_ERR_ARG
    assert lib.up_kv_write(c, A, 256, A, 256, None, 4, None, A, None) == up.UP_ERR_ARG
    assert lib.up_kv_write(c, A, 256, A, 256, A, -1, None, A, None) == up.UP_ERR_ARG
    assert lib.up_kv_write(c, A, 256, A, 256, A, 4, None, None, None) == up.UP_ERR_ARG
    assert lib.up_kv_write(c, ODD, 256, A, 256, A, 4, None, A, None) == up.UP_ERR_SHAPE
    assert lib.up_kv_write(c, A, 255, A, 256, A, 4, None, A, None) == up.UP_ERR_SHAPE
    assert lib.up_kv_write(c, A, 256, A, 248, A, 4, None, A, None) == up.UP_ERR_SHAPE      # tokens overlap
    assert lib.up_kv_read(c, A, 4, None, A, ODD, A, None) == up.UP_ERR_SHAPE
    assert lib.up_kv_read(c, None, 4, None, A, A, A, None) == up.UP_ERR_ARG
    # nothing to do: no pointer is needed
    assert lib.up_kv_write(c, None, 0, None, 0, None, 0, None, A, None) == up.UP_OK
    assert lib.up_kv_read(c, None, 0, None, None, None, A, None) == up.UP_OK


def test_bad_arguments_of_decode(up):
    lib, cache = up.load_library(), _cache(up)
    c = ctypes.byref(cache)
    good = dict(q=A, q_stride=512, cache=c, table=A, seqused=A, R=2, max_blocks=4, Hq=4, scale=0.1, window=0, out=A,
                lse=None, ws=A, ws_bytes=1 << 40, status=A, stream=None)

    def call(**kw):
        return lib.up_paged_decode(*dict(good, **kw).values())
    for name in ("q", "cache", "table", "seqused", "out", "ws", "status"):
        assert call(**{name: None}) == up.UP_ERR_ARG, name
    for bad in (dict(R=0), dict(max_blocks=0), dict(Hq=0), dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**bad) == up.UP_ERR_ARG, bad
    for bad in (dict(Hq=3), dict(q=ODD), dict(out=ODD), dict(q_stride=511), dict(q_stride=504), dict(max_blocks=1 << 30)):
        assert call(**bad) == up.UP_ERR_SHAPE, bad
    need = up.up_paged_decode_workspace_bytes(2, 4, 2, 128, 16, 4)
    assert need > 0
    assert call(ws_bytes=need - 1) == up.UP_ERR_WORKSPACE
    assert call(ws=ODD) == up.UP_ERR_WORKSPACE


def test_workspace_sizes(up):
    f = up.up_paged_decode_workspace_bytes
    assert f(2, 4, 2, 100, 16, 4) == 0 and f(0, 4, 2, 128, 16, 4) == 0 and f(2, 4, 3, 128, 16, 4) == 0
    assert f(2, 4, 2, 128, 0, 4) == 0 and f(2, 4, 2, 128, 16, 0) == 0 and f(2, 4, 2, 128, 16, 4, -1) == 0
    assert f(1, 32, 8, 128, 16, 65536) >= f(1, 32, 8, 128, 16, 256) > 0
    assert f(1, 32, 8, 128, 16, 65536, 1024) <= f(1, 32, 8, 128, 16, 65536)
    assert [up.up_kv_scale_row(b) for b in (-1, 0, 1, 16, 17, 100)] == [0, 0, 16, 16, 32, 112]
    for code in (8, 9, 10):
        assert "unknown" not in up.up_status_string(code, True)


def test_the_reference_quantiser_against_torch_and_the_formula():
    rng = np.random.default_rng(1)
    x = rng.uniform(-448, 448, 20000).astype(np.float32)
    x = np.concatenate([x, x * 2.0 ** -12, kv_ref.E4M3[np.isfinite(kv_ref.E4M3)].astype(np.float32)])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv_ref.e4m3_codes(x), want)
    rows = kv_ref.bf16_value(kv_ref.bf16_bits((rng.standard_normal((500, 64)) * 2.0 ** rng.integers(-30, 30, (500, 1))).astype(np.float32)))
    codes, b = kv_ref.quantise(rows)
    top = np.abs(rows).max(-1) / 2.0 ** (b.astype(float) - 127)
    assert (top <= 448).all() and (top > 224).all()
    err = np.abs(kv_ref.dequantise(codes, b) - rows)
    step = 2.0 ** (b.astype(float) - 127)[:, None]
    assert (err <= np.maximum(np.abs(rows) * 2.0 ** -4, step * 2.0 ** -10)).all()


def test_the_reference_attention_against_torch():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((1, 6, 64)), rng.standard_normal((50, 2, 64)), rng.standard_normal((50, 2, 64))
    o, lse, _, _ = kv_ref.decode(q, [k], [v], 0.125)
    tq, tk, tv = (torch.from_numpy(x) for x in (q[0], np.repeat(k, 3, 1), np.repeat(v, 3, 1)))
    a = torch.einsum("hd,nhd->hn", tq, tk) * 0.125
    assert np.allclose(o[0], torch.einsum("hn,nhd->hd", a.softmax(-1), tv).numpy(), atol=1e-12)
    assert np.allclose(lse[0], a.logsumexp(-1).numpy(), atol=1e-12)
