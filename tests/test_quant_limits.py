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
