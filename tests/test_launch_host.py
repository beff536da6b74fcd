"""The host side of the library's launches (no GPU): its objects linked with a stand-in for the CUDA runtime, which keeps
attributes per device, refuses what they do not allow and can be told to fail."""
import ctypes
import itertools
import os
import subprocess

import pytest

from long_context_prefill_varlen_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))
A = 0x1000                     # never dereferenced
# the stand-in's devices (the library tells 64 apart): 0, 1, one for each size of cluster, then one that no test had before
CLUSTERS = {1: 2, 2: 3, 4: 4, 8: 5, 16: 6}
fresh_device = itertools.count(7).__next__


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    import long_context_prefill_varlen_gb300 as up
    _build.build()
    objects = [os.path.join(_build.PKG, "_build", s.replace(".cu", ".o")) for s in _build.SOURCES]
    out = str(tmp_path_factory.mktemp("fake") / "libuniprefill_fake.so")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc())))
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", os.path.join(cuda, "include"),
                        "-o", out, os.path.join(HERE, "fake_cudart.cpp")] + objects, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    m = ctypes.CDLL(out)
    for name, (res, args) in up._SIGNATURES.items():
        getattr(m, name).restype, getattr(m, name).argtypes = res, args
    m.fake_launch_name.restype = ctypes.c_char_p
    return m


def _decode(lib, Hq=32, Hkv=8, dk=128, e4m3=False, R=1, max_blocks=256, B=16):
    import long_context_prefill_varlen_gb300 as up
    cache = up._KvCache(A, A, A, A, 8, Hkv * B * dk, B * dk, dk, Hkv, B, dk, up.KV_E4M3 if e4m3 else up.KV_BF16)
    return lib.up_paged_decode(A, Hq * dk, ctypes.byref(cache), A, A, R, max_blocks, Hq, 0.1, 0, A, None, A, 1 << 50, A, None)


def _launched(lib):
    return [(lib.fake_launch_name(i).decode(), lib.fake_launch_cluster(i)) for i in range(lib.fake_launches())]


SHAPES = [(Hq, dk, e4m3) for Hq in (8, 16) for dk in (64, 128, 256) for e4m3 in (False, True)]


@pytest.mark.parametrize("R", [1, 300], ids=["one_launch", "two_launches"])
@pytest.mark.parametrize("Hq,dk,e4m3", SHAPES)
def test_decode_sets_its_kernels_up_on_every_device(lib, Hq, dk, e4m3, R):
    for device in (0, 1):
        for _ in range(2):
            lib.fake_reset(device, 16)
            assert _decode(lib, Hq, 1, dk, e4m3, R) == 0, device
            launched = _launched(lib)
            assert len(launched) == (1 if R == 1 else 2) and "split_kernel" in launched[0][0]


def test_a_set_up_that_failed_is_tried_again(lib):
    device = fresh_device()
    lib.fake_reset(device, 16)
    lib.fake_fail(1, 0)
    assert _decode(lib) != 0 and lib.fake_launches() == 0
    lib.fake_reset(device, 16)
    assert _decode(lib) == 0 and lib.fake_launches() == 1


@pytest.mark.parametrize("tokens", [None, A], ids=["one_pass", "two_pass"])
@pytest.mark.parametrize("R", [1, 5000])
@pytest.mark.parametrize("Hq,Hkv,dk", [(8, 2, 64), (8, 2, 128), (4, 2, 256)])
def test_the_score_sets_its_kernels_up_on_every_device(lib, Hq, Hkv, dk, R, tokens):
    T, G, n = 10000, 64, 128
    nb = lib.up_max_blocks(R, T, G)
    for device in (0, 1):
        lib.fake_reset(device, 16)
        assert lib.up_score_blocks(A, A, A, R, T, Hq, Hkv, dk, G, n, 0.1, A, nb, A, tokens, A, 1 << 50, A, None) == 0, device
        assert any("score_pass_kernel" in name for name, _ in _launched(lib))


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("largest", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("Hq,Hkv,dk,max_blocks,wants", [(32, 8, 128, 16, 1), (32, 8, 128, 32, 2), (32, 8, 128, 64, 4), (32, 8, 128, 128, 8),
                                                        (32, 8, 128, 256, 16), (4, 1, 256, 256, 16)])
def test_a_cluster_that_the_device_cannot_place_gives_two_launches(lib, Hq, Hkv, dk, max_blocks, wants, largest, e4m3):
    """(a partition of a GPU may have room for smaller clusters only)"""
    device = CLUSTERS[largest]
    for _ in range(2):
        lib.fake_reset(device, largest)
        assert _decode(lib, Hq, Hkv, dk, e4m3, 1, max_blocks) == 0
        launched = _launched(lib)
        assert [c for _, c in launched] == ([wants] if wants <= largest else [1, 1])
        assert "split_kernel" in launched[0][0] and (wants <= largest or "join_kernel" in launched[1][0])
    lib.fake_reset(device, largest)
    assert _decode(lib, Hq, Hkv, dk, e4m3, 1, 16) == 0 and lib.fake_launches() == 1      # no error is left behind


@pytest.mark.parametrize("R", [1, 300], ids=["one_launch", "two_launches"])
@pytest.mark.parametrize("attributes,launches", [(1, 0), (0, 1)], ids=["attribute", "launch"])
def test_an_error_of_a_decode_call_is_that_calls_alone(lib, attributes, launches, R):
    device = fresh_device()
    lib.fake_reset(device, 16)
    lib.fake_fail(attributes, launches)
    assert _decode(lib, R=R) == 4                                # UP_ERR_CUDA
    assert _decode(lib, R=R) == 0


def test_an_error_of_a_cache_call_is_that_calls_alone(lib):
    import long_context_prefill_varlen_gb300 as up
    cache = ctypes.byref(up._KvCache(A, A, A, A, 8, 2 * 16 * 128, 16 * 128, 128, 2, 16, 128, up.KV_E4M3))
    for call in (lambda: lib.up_kv_write(cache, A, 256, A, 256, A, 4, None, A, None), lambda: lib.up_kv_read(cache, A, 4, None, A, A, A, None)):
        lib.fake_reset(0, 16)
        lib.fake_fail(0, 1)
        assert call() == 4 and call() == 0


@pytest.mark.parametrize("attributes,launches", [(1, 0), (0, 1)], ids=["attribute", "launch"])
def test_an_error_of_a_drop_step_call_is_that_calls_alone(lib, attributes, launches):
    lib.fake_reset(fresh_device(), 16)
    for call in (lambda: lib.up_score_blocks(A, A, A, 1, 1000, 8, 2, 128, 64, 128, 0.1, A, 100, A, None, A, 1 << 50, A, None),
                 lambda: lib.up_select_topp(A, A, A, 1, 1000, 100, 64, 128, 128, 0.9, A, A, A, None, 0, A, None)):
        lib.fake_fail(attributes, launches)
        assert call() == 4
        assert lib.up_seqused(A, A, 2, 3, 1, A, A, A, None) == 0 and call() == 0
