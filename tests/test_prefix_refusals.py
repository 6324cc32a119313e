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


@pytest.mark.parametrize("short", [1, 4096])
def test_a_workspace_that_is_too_small(dsa, short):
    import ctypes
    from test_prefix_step import _attend_args
    n = ctypes.c_size_t(0)
    assert dsa.lib().dsa_prefix_mla_workspace_size(ctypes.byref(_attend_args(dsa)), ctypes.byref(n)) == dsa.DSA_OK
    a = _attend_args(dsa, workspace_bytes=n.value - short)
    assert dsa.lib().dsa_prefix_mla(ctypes.byref(a), None) == dsa.DSA_ERR_WORKSPACE
    for bad in (dict(workspace=None), dict(workspace=(1 << 20) + 8)):
        a = _attend_args(dsa, workspace_bytes=n.value, **bad)
        assert dsa.lib().dsa_prefix_mla(ctypes.byref(a), None) == dsa.DSA_ERR_WORKSPACE


def test_the_size_helper_answers_for_the_call(dsa):
    import ctypes
    from test_prefix_step import _attend_args
    for B, T, H, prefix, page in ((1, 1, 128, 0, 16), (5, 9, 20, 1000, 128), (64, 64, 64, 8192, 64), (2, 900, 17, 33, 32)):
        n = ctypes.c_size_t(0)
        a = _attend_args(dsa, B=B, total_q=T, H=H, prefix_len=prefix, page_size=page, num_prefix_pages=-(-prefix // page),
                         max_pages_per_seq=77)
        assert dsa.lib().dsa_prefix_mla_workspace_size(ctypes.byref(a), ctypes.byref(n)) == dsa.DSA_OK
        assert dsa.dsa_prefix_mla_workspace_size(B, T, H, prefix_len=prefix) == n.value
    assert dsa.dsa_prefix_mla_workspace_size(3, 0, 64, prefix_len=10) == 0
    with pytest.raises(dsa.DsaError):
        dsa.dsa_prefix_mla_workspace_size(3, 4, 129, prefix_len=10)


def test_strides_of_dimensions_of_size_one_do_not_count(dsa):
    import ctypes
    from test_prefix_step import _attend_args
    # the workspace is asked for last: what gets there was accepted so far
    call = lambda **kw: dsa.lib().dsa_prefix_mla(ctypes.byref(_attend_args(dsa, workspace_bytes=0, **kw)), None)
    odd = dict(qn_stride_t=577, qr_stride_t=65)
    assert call(total_q=1, **odd) == dsa.DSA_ERR_WORKSPACE
    assert call(total_q=2, **odd) == dsa.DSA_ERR_INVALID_ARGUMENT
    odd = dict(qn_stride_h=577, qr_stride_h=65)
    assert call(H=1, **odd) == dsa.DSA_ERR_WORKSPACE
    assert call(H=2, **odd) == dsa.DSA_ERR_INVALID_ARGUMENT
    assert call(total_q=1, H=2, **odd) == dsa.DSA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("big", [dict(total_q=1 << 24), dict(total_q=(1 << 31) - 1, H=1), dict(total_q=(1 << 31) - 1, H=128),
                                 dict(num_pages=1 << 25), dict(prefix_len=(1 << 31) - 128, num_prefix_pages=1 << 25)])
def test_sizes_that_pass_32_bits(dsa, big):
    """Refused by the call and by its workspace size alike (a size from overflown tile counts would be
    of no use to anybody)."""
    import ctypes
    from test_prefix_step import _attend_args
    a = _attend_args(dsa, **{"H": 128, **big})
    n = ctypes.c_size_t(5)
    assert dsa.lib().dsa_prefix_mla_workspace_size(ctypes.byref(a), ctypes.byref(n)) == dsa.DSA_ERR_UNSUPPORTED
    assert n.value == 5
    a.workspace_bytes = 0  # the workspace is asked for last
    assert dsa.lib().dsa_prefix_mla(ctypes.byref(a), None) == dsa.DSA_ERR_UNSUPPORTED
