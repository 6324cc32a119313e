"""Sizes and values of the quantised latent cache's calls that are past what they can do: refused, without a GPU."""
import pytest

from test_quant_refusals import MLA, READ, _call, _size, dsa  # noqa: F401 (dsa is a fixture)


@pytest.mark.parametrize("width", [0x7FFFFF01, 0x7FFFFFC1, 0x7FFFFFFF])
def test_selections_whose_blocks_pass_32_bits(dsa, width):  # noqa: F811
    assert _call(dsa, "dsa_quant_mla", MLA, dict(topk_width=width, total_q=1)) == dsa.DSA_ERR_UNSUPPORTED


def test_the_widest_selection_is_cut_like_others(dsa):  # noqa: F811
    sizes = [_size(dsa, topk_width=k, total_q=1, H=64) for k in (1 << 20, 0x7FFFFF00)]
    assert sizes[0] == sizes[1]


@pytest.mark.parametrize("scale", [float("inf"), -float("inf")])
def test_a_scale_that_is_not_finite(dsa, scale):  # noqa: F811
    assert _call(dsa, "dsa_quant_mla", MLA, dict(scale=scale)) == dsa.DSA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("strides", [dict(c_stride=0), dict(c_stride=504), dict(r_stride=0), dict(r_stride=56)], ids=str)
def test_rows_that_lie_over_one_another_are_not_written(dsa, strides):  # noqa: F811
    """Two rows of an output would be written to the same place by two warps; one row's stride leads nowhere."""
    assert _call(dsa, "dsa_mla_quant_read", READ, strides) == dsa.DSA_ERR_INVALID_ARGUMENT
    assert _call(dsa, "dsa_mla_quant_read", READ, dict(strides, total=0)) == dsa.DSA_OK


@pytest.mark.parametrize("kw", [dict(total_q=1, H=64, topk_width=65536), dict(total_q=16, H=64, topk_width=2048),
                                dict(total_q=17, H=64, topk_width=2048), dict(total_q=33, H=16, topk_width=2048),
                                dict(total_q=4, H=128, topk_width=8192), dict(total_q=33, H=64, topk_width=256)], ids=str)
def test_tiles_are_not_cut_less_for_the_sake_of_a_cluster(dsa, kw):  # noqa: F811
    """Few tiles of many keys are cut for all SMs: their pieces go through memory, so the call takes a workspace of their size
    (148 SMs where there is none to ask, two pieces of 64 x 512 fp32 a CTA)."""
    tiles = kw["total_q"] * -(-kw["H"] // 64)
    blocks = -(-kw["topk_width"] // 64)
    pieces = tiles * min(148 // tiles, blocks // 2)
    assert _size(dsa, **kw) >= 2 * pieces * 64 * 512 * 4


@pytest.mark.parametrize("kw", [dict(total_q=4, H=16, topk_width=2048), dict(total_q=64, H=64, topk_width=2048),
                                dict(total_q=30, H=32, topk_width=512)], ids=str)
def test_pieces_of_a_cluster_take_no_workspace(dsa, kw):  # noqa: F811
    assert _size(dsa, **kw) == 0


@pytest.mark.parametrize("site,limit,good", [(1, 1000, True), (7, 10 ** 9, True), (15, 1000, True), (0, 1000, False), (8, 1000, False),
                                             (16, 1000, False), (-1, 1000, False), (1, 10 ** 9 + 1, False)])
def test_arguments_of_the_failure_hook(dsa, site, limit, good):  # noqa: F811
    want = dsa.DSA_OK if good else dsa.DSA_ERR_INVALID_ARGUMENT
    assert dsa.lib().dsa_test_arm_quant_mla_timeout(site, 0, limit) == want
    assert dsa.lib().dsa_test_arm_quant_mla_timeout(1, 0, 0) == dsa.DSA_OK  # disarmed again
