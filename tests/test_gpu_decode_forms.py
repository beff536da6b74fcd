"""The two forms of a decode call (GPU): one launch of clusters where every chunk can have a CTA at once, CTAs that stay and a
join otherwise.  Which one ran is counted, and both give the same bits."""
import shutil

import numpy as np
import pytest
import torch

import long_context_prefill_varlen_gb300 as up
from tests.test_gpu_debug_bounds import library
from tests.test_gpu_kvcache import _decode_case, _from_bits, _run_decode, _status

pytestmark = pytest.mark.gpu

MOST_CTAS = 6                  # of the decode kernel on an SM


def _both(Hq, Hkv, dk, lens, e4m3, max_blocks, B=16, seed=5):
    c, table, _, qb = _decode_case(seed, Hq, Hkv, dk, B, lens, e4m3, extra_cols=0)
    table = np.pad(table, ((0, 0), (0, max_blocks - table.shape[1])), constant_values=-1)

    def counted(times):
        before = up.up_kernel_launches()
        status, out, lse = _run_decode(c, np.tile(table, (times, 1)), tuple(lens) * times, _from_bits(np.tile(qb, (times, 1, 1))))
        assert status == 0
        return up.up_kernel_launches() - before, out, lse
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    times = MOST_CTAS * sms // (len(lens) * Hkv) + 1             # more rows than CTAs
    launches, out, lse = counted(1)
    assert launches == 1
    launches, many, many_lse = counted(times)
    assert launches == 2
    assert torch.equal(many, out.repeat(times, 1, 1)) and torch.equal(many_lse, lse.repeat(times, 1))


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("max_blocks,chunks", [(16, 1), (32, 2), (48, 3), (64, 4), (80, 5), (128, 8), (200, 13), (256, 16)])
@pytest.mark.parametrize("Hq,Hkv,dk", [(8, 2, 128), (2, 2, 64), (4, 1, 256)])
def test_both_forms_at_every_size_of_cluster(Hq, Hkv, dk, max_blocks, chunks, e4m3):
    _both(Hq, Hkv, dk, (16 * max_blocks - 5,), e4m3, max_blocks)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("group,Hkv", [(1, 3), (2, 8), (3, 1), (5, 2), (7, 1), (9, 1), (16, 1), (17, 2), (32, 1)])
def test_both_forms_over_head_groups(group, Hkv, dk, e4m3):
    _both(group * Hkv, Hkv, dk, (300, 0, 77), e4m3, 20)


@pytest.mark.parametrize("R", [1, 700], ids=["one_launch", "two_launches"])
def test_the_first_call_can_be_captured(R, tmp_path):
    """a copy of the library, whose kernels nobody has set up yet"""
    copy = str(tmp_path / "libuniprefill_copy.so")
    shutil.copy(up.LIB_PATH, copy)
    lens = (300,) * R
    c, table, _, qb = _decode_case(8, 8, 2, 128, 16, (300,), True, extra_cols=0)
    table, q = np.tile(table, (R, 1)), _from_bits(np.tile(qb, (R, 1, 1)))
    _, want, _ = _run_decode(c, table, lens, q)
    tb, n, out, st = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.zeros_like(q), _status()
    ws = torch.empty(up.up_paged_decode_workspace_bytes(R, 8, 2, 128, 16, table.shape[1]), dtype=torch.uint8, device="cuda")
    with library(copy):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            up.up_paged_decode(q, c.k, c.v, tb, n, out, ws, st, **c.scales())
        assert up.up_kernel_launches() == (1 if R == 1 else 2)
    g.replay()
    torch.cuda.synchronize()
    assert up.up_read_status(st) == 0 and torch.equal(out, want)
