"""Failure path of the shared-prefix attention without a GPU fault.

Every wait of the attention kernel is bounded.  dsa_test_arm_prefix_mla_timeout makes one wait of
one role run out (in one CTA of every pair): the kernel records DSA_ERR_TIMEOUT, every role of both
CTAs leaves its loop, MMAs and copies in flight are drained and the tensor memory is freed.  The
host reads DSA_ERR_TIMEOUT, the context stays usable and the next call gives the same bits as ever.

Each drain gives up after 0.2 s (4e8 cycles at about 2 GHz) when it waits for something that does
not come, so a call that ends sooner drained what was in flight and nothing else.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("sparse_attention_token_gb300")

LIMIT_NS = 2_000_000   # 2 ms: far longer than the copies in flight take to land
ODD = 8


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def _batch(requests, H, prefix, new, own, page=64):
    """(arguments, keywords) of a dsa_prefix_mla call: pages one after another."""
    g = torch.Generator(device="cuda").manual_seed(requests + H)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    shared, per = prefix // page, -(-(prefix % page + own) // page)
    pages = shared + 1 + requests * per
    bt = torch.zeros((requests, shared + per), dtype=torch.int32)
    bt[:, :shared] = torch.arange(shared)
    bt[:, shared:] = shared + 1 + torch.arange(requests * per).view(requests, per)
    lens = prefix + own - torch.arange(requests) % min(own - new + 1, 50)
    cu = torch.arange(requests + 1) * new
    i32 = lambda t: t.to(torch.int32).cuda()
    q = rnd(requests * new, H, 576)
    return ((q[..., :512], q[..., 512:], rnd(pages, page, 512), rnd(pages, page, 64), bt.cuda(), i32(cu), i32(lens),
             i32(torch.arange(shared + 1))), dict(prefix_len=prefix, scale=576 ** -0.5))


BATCHES = {
    "shared tiles": dict(requests=40, H=64, prefix=2900, new=1, own=250),   # several pieces a pair, joined
    "own tiles": dict(requests=6, H=128, prefix=1500, new=40, own=700),     # causal borders, cleared rows
}
# the issuer stopping at a block leaves the copies of it, and those behind it, in flight
SITES = ([(1, at) for at in range(7)] + [(2, 0), (3, 0), (4, 1), (5, 0)]
         + [(2 + ODD, 0), (3 + ODD, 0), (4 + ODD, 1), (5 + ODD, 0)]) * 3


@pytest.mark.parametrize("batch", BATCHES)
def test_a_wait_that_runs_out_ends_the_call_and_the_next_is_right(batch):
    args, kw = _batch(**BATCHES[batch])
    ref = dsa.dsa_prefix_mla(*args, **kw)
    assert dsa.dsa_check_device_status() == dsa.DSA_OK
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for site, at in SITES:
        dsa.dsa_test_arm_prefix_mla_timeout(site, at, LIMIT_NS)
        begin.record()
        dsa.dsa_prefix_mla(*args, **kw)
        end.record()
        status = dsa.dsa_check_device_status()
        torch.cuda.synchronize()
        took = begin.elapsed_time(end) / 1e3
        assert status == dsa.DSA_ERR_TIMEOUT, (site, at)
        assert took < 0.15, (site, at, took)
        assert dsa.dsa_check_device_status() == dsa.DSA_OK        # the status word was cleared
        got = dsa.dsa_prefix_mla(*args, **kw)                     # the arming was used up
        assert dsa.dsa_check_device_status() == dsa.DSA_OK, (site, at)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]), (site, at)


def test_a_disarmed_hook_changes_nothing():
    args, kw = _batch(**BATCHES["shared tiles"])
    ref = dsa.dsa_prefix_mla(*args, **kw)
    dsa.dsa_test_arm_prefix_mla_timeout(2, 0, LIMIT_NS)
    dsa.dsa_test_arm_prefix_mla_timeout(2, 0, 0)
    got = dsa.dsa_prefix_mla(*args, **kw)
    assert dsa.dsa_check_device_status() == dsa.DSA_OK
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
