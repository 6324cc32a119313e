"""Calls of the quantised latent cache at the edges of what the documentation allows."""
import pytest
import torch

from oracle import quant_cache as qc
from test_gpu_quant_mla import Case, I32, _built, _ok, dsa  # noqa: F401 (_built is a fixture)

pytestmark = pytest.mark.gpu

FORMATS = [qc.FP8, qc.FP4]


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("k", [None, 70])
def test_without_requests_all_rows_are_padding(row, k):
    """cu_q_lens has one entry then, and no length belongs to it, whatever it holds."""
    for end in (0, 2, 7):
        case = Case(row, 20, 16, [], k=k, pad=3)
        case.cu = I32([end])
        out, lse = case.run()
        _ok()
        assert not out.any() and (lse == -float("inf")).all()


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("H,k,queries", [(64, 2048, 16), (16, 2048, 16), (16, 2048, 15), (64, 2048, 17), (20, 2048, 33), (32, 2048, 24),
                                         (64, 20000, 1), (128, 9000, 2), (8, 700, 45), (64, 384, 192)])
def test_cuts_of_few_tiles(row, H, k, queries):
    """On both sides of the rule that takes a cluster or memory for the pieces of a tile."""
    Case(row, H, 64, [(queries, max(k, 2500))], k=k, seed=k + queries).check()
