"""Failure path of the attention over the quantised cache without a GPU fault.

dsa_test_arm_quant_mla_timeout makes one wait of one role run out, in every other CTA: the kernel records DSA_ERR_TIMEOUT,
every role leaves its loop, MMAs and copies in flight are drained, the CTAs of a cluster still meet and the tensor memory is
freed.  The host reads DSA_ERR_TIMEOUT, the context stays usable and the next call gives the same bits as ever.

Each drain gives up after 0.2 s (4e8 cycles at about 2 GHz) when it waits for something that does not come, so a call that ends
sooner drained what was in flight and nothing else.
"""
import pytest
import torch

from oracle import quant_cache as qc
from test_gpu_quant_mla import Case, _built, dsa  # noqa: F401 (_built is a fixture)

pytestmark = pytest.mark.gpu

LIMIT_NS = 2_000_000  # 2 ms: far longer than the copies in flight take to land
ODD = 8
MMA, COPY, COPY2, ROWS, QUERIES, DECODE, SOFTMAX = range(1, 8)

CALLS = {
    "cluster of 2": dict(H=64, reqs=[(1, 2500)] * 64, k=2048),
    "cluster of 8": dict(H=16, reqs=[(1, 2500)] * 4, k=2048),
    "through memory": dict(H=64, reqs=[(1, 2500)] * 16, k=2048),
    "whole tiles and a rest": dict(H=20, reqs=[(230, 2500)], k=640),
    "every position": dict(H=64, reqs=[(1, 3000), (2, 9000), (1, 77)] * 4, k=None),
}
SITES = ([(MMA, at) for at in range(6)] + [(COPY, at) for at in range(7)] + [(COPY2, at) for at in (0, 1, 2, 3, 5)]
         + [(ROWS, 0), (ROWS, 1), (QUERIES, 0), (DECODE, 0), (DECODE, 3), (SOFTMAX, 0), (SOFTMAX, 1), (SOFTMAX, 4)])


@pytest.mark.parametrize("row", [qc.FP8, qc.FP4])
@pytest.mark.parametrize("call", CALLS)
def test_a_wait_that_runs_out_ends_the_call_and_the_next_is_right(row, call):
    case = Case(row, CALLS[call]["H"], 64, CALLS[call]["reqs"], k=CALLS[call]["k"], seed=1)
    want = case.run()
    torch.cuda.synchronize()
    assert dsa.dsa_check_device_status() == dsa.DSA_OK
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    reached = 0
    for odd in (0, ODD):
        for site, at in SITES:
            dsa.dsa_test_arm_quant_mla_timeout(site + odd, at, LIMIT_NS)
            begin.record()
            case.run()
            end.record()
            status = dsa.dsa_check_device_status()
            torch.cuda.synchronize()
            took = begin.elapsed_time(end) / 1e3
            # (a CTA of few blocks does not come to the later ones, nor 8-bit rows to decoding)
            comes = not (site == DECODE and row == qc.FP8) and at < (1 if site == ROWS else 2)
            assert status in ([dsa.DSA_ERR_TIMEOUT] if comes else [dsa.DSA_OK, dsa.DSA_ERR_TIMEOUT]), (site, odd, at)
            reached += status != dsa.DSA_OK
            assert took < 0.15, (site, odd, at, took)
            assert dsa.dsa_check_device_status() == dsa.DSA_OK    # the status word was cleared
            got = case.run()                                      # the arming was used up
            assert dsa.dsa_check_device_status() == dsa.DSA_OK, (site, odd, at)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (site, odd, at)
    assert reached >= 26


def test_a_disarmed_hook_changes_nothing():
    case = Case(qc.FP8, 16, 64, [(1, 2500)] * 4, k=2048, seed=1)
    want = case.run()
    dsa.dsa_test_arm_quant_mla_timeout(MMA, 0, LIMIT_NS)
    dsa.dsa_test_arm_quant_mla_timeout(MMA, 0, 0)
    got = case.run()
    assert dsa.dsa_check_device_status() == dsa.DSA_OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
