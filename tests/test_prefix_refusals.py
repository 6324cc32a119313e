"""Refusals and workspace sizes of the shared-prefix entry points, which need no GPU."""
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


@pytest.mark.parametrize("B,H", [(1, 64), (64, 64), (128, 16), (1024, 16), (4096, 8), (4096, 1)])
def test_workspace_follows_the_rows(dsa, B, H):
    """Two slots of 128 x 514 fp32 for each pair of SMs, whatever the batch; two results of that row
    size for every row that two tiles may share, in blocks of 128; and the plan's records: at most
    64 bytes a query, 40 a tile and 4 a request."""
    alone = dsa.dsa_prefix_mla_workspace_size(1, 1, 128, prefix_len=1000)
    row = 514 * 4
    blocks, tiles = -(-B * H // 128), 2 * (B * H // 128 + 1) + B + 1
    most = alone + 2 * blocks * 128 * row + 64 * B + 40 * tiles + 4 * B + 4096
    assert dsa.dsa_prefix_mla_workspace_size(B, B, H, prefix_len=1000) <= most
