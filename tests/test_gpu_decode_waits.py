"""Decode attention when a bounded wait runs out (GPU): a build whose kernels give up after a microsecond.

A call that gave up anywhere reports UP_DEV_WAIT_TIMEOUT; one that reports nothing is right; the context and the
next calls are none the worse."""
import pytest
import torch

from long_context_prefill_varlen_gb300 import _build
from tests.test_gpu_debug_bounds import library
from tests.test_gpu_kvcache import LENS, _decode_case, _from_bits, _run_decode

pytestmark = pytest.mark.gpu

TIMEOUT = 4                                                      # UP_DEV_WAIT_TIMEOUT
# Hq, Hkv, dk, lengths, e4m3: one launch with a cluster a row, then calls of CTAs that stay and a join
CASES = [(32, 8, 128, (4096,), False), (8, 2, 128, LENS, True), (4, 1, 64, (1,), True), (32, 1, 128, (100,) * 3, True),
         (8, 2, 128, LENS * 40, True), (16, 8, 256, (3000,) * 40, False), (32, 8, 128, (9000,) * 30, True)]


@pytest.fixture(scope="module")
def waits_lib():
    return _build.build(wait_limit_ns=1000)


def test_a_wait_that_runs_out_is_reported(waits_lib):
    cases = []
    for Hq, Hkv, dk, lens, e4m3 in CASES:
        c, table, _, qb = _decode_case(5, Hq, Hkv, dk, 16, lens, e4m3)
        q = _from_bits(qb)
        status, out, lse = _run_decode(c, table, lens, q)
        assert status == 0
        cases.append((c, table, lens, q, out, lse))
    ran_out = []
    with library(waits_lib):
        for c, table, lens, q, out, lse in cases:
            ran_out.append(0)
            for _ in range(20):
                status, o, l = _run_decode(c, table, lens, q)
                assert status in (0, TIMEOUT)
                assert status == TIMEOUT or (torch.equal(o, out) and torch.equal(l, lse))
                ran_out[-1] += status == TIMEOUT
    assert max(ran_out) > 0, ran_out                             # else nothing was tested
    for c, table, lens, q, out, lse in cases:
        status, o, l = _run_decode(c, table, lens, q)
        assert status == 0 and torch.equal(o, out) and torch.equal(l, lse)
