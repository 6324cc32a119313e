"""Refusals of the shared-prefix entry points that need no GPU, beside those of test_prefix_step.py."""
import pytest


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__ as g
    g.build()
    import sparse_attention_token_gb300 as m
    return m


@pytest.mark.parametrize("site,limit,ok", [(1, 1000, True), (5, 0, True), (13, 1000, True), (0, 1000, False), (6, 1000, False),
                                           (8, 1000, False), (9, 1000, False), (14, 1000, False), (-1, 1000, False),
                                           (17, 1000, False), (1, 2_000_000_000, False)])
def test_timeout_hook_sites(dsa, site, limit, ok):
    want = dsa.DSA_OK if ok else dsa.DSA_ERR_INVALID_ARGUMENT
    assert dsa.lib().dsa_test_arm_prefix_mla_timeout(site, 0, limit) == want
    assert dsa.lib().dsa_test_arm_prefix_mla_timeout(1, 0, 0) == dsa.DSA_OK  # disarmed again
