"""Attention over the quantised cache where one key stands far ahead of many that matter together.

The 64-bit oracle and the errors E of the logits are those of test_gpu_quant_mla.py.  A key's probability is held in two
terms, 2^-7 of it off at most, and fp16's 2^-11; what it weighs must not depend on how far behind the first key it stands, as
long as the keys behind it count in the output.
"""
import numpy as np
import pytest
import torch

from oracle import quant_cache as qc
from test_gpu_quant_mla import Case, I32, _built, _ok, dsa  # noqa: F401 (_built is a fixture)

pytestmark = pytest.mark.gpu

FORMATS = [qc.FP8, qc.FP4]
P = 2.0 ** -7 + 2.0 ** -11


def _logits_by_rope(case, leads, c=None, seed=8):
    """Rows whose logit is `leads[position]` (bf16) for every query and head, latent rows c (random about 1 when not given)."""
    case.q[:] = 0
    case.q[..., 512] = 1.0
    case.scale = 1.0
    n = case.pages * case.page
    g = torch.Generator(device="cuda").manual_seed(seed)
    if c is None:
        c = 1 + 0.25 * torch.randn((case.reqs[0][1], 512), generator=g, device="cuda")
    pos = torch.arange(len(leads), device="cuda")
    at = case.bt[0].long()[pos // case.page] * case.page + pos % case.page
    r = torch.zeros((len(leads), 64), dtype=torch.bfloat16, device="cuda")
    r[:, 0] = torch.as_tensor(leads, device="cuda").to(torch.bfloat16)
    dsa.dsa_mla_quant_append(c[: len(leads)].to(torch.bfloat16), r, at, case.cache)
    return n


def _one_query(case):
    """The reference of the first query and head: all see the same keys."""
    q, topk, cu, T, H = case.q, case.topk, case.cu, case.T, case.H
    case.q, case.cu, case.T = case.q[:1, :1], I32([0, 1]), 1
    case.topk = None if topk is None else topk[:1]
    ref = case.reference()
    case.q, case.topk, case.cu, case.T = q, topk, cu, T
    return ref


def _logit_error(ref):
    return 2.0 ** -20 * ref["small"] + 2.0 ** -13 * ref["reach"] + 2.0 ** -16 + ref["n"][:, None] * 2.0 ** -22


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("queries,k", [(160, 2048), (3, 2048), (1, 70), (1, None)])
@pytest.mark.parametrize("ahead", [9.5, 10.25, 10.5, 12.0, 16.0, 24.0])
def test_rows_of_zeros_ahead(row, queries, k, ahead):
    """A row of zeros adds nothing to the output, so the keys behind it are all there is of it, held as any others: 2^-7 and
    2^-11 of each, the output's rounding and the logits' errors, relative to the sum of magnitudes, whatever the gap."""
    n = 2300
    case = Case(row, 16, 64, [(queries, n)], k=k, seed=6, spread=0.0)
    if k is None:
        case.reqs = [(1, n)]
    lead = torch.zeros(n)
    first = torch.arange(k or n)
    zero = [0, 63, 64, (k or n) - 1]  # in the first block, at its end, in the last
    lead[zero[:1]] = ahead
    lead[zero[1:]] = ahead - 1
    c = 1 + 0.25 * torch.randn((n, 512), generator=torch.Generator(device="cuda").manual_seed(8), device="cuda")
    c[zero] = 0
    _logits_by_rope(case, lead, c)
    if k is not None:
        case.topk = first.to(torch.int32).cuda().repeat(case.T, 1).contiguous()
    out, lse = case.run()
    _ok()
    ref = _one_query(case)
    E = _logit_error(ref)[0]
    o = out.double().cpu().numpy()
    assert (np.abs(o - ref["out"][0, 0]) <= (P + 2 * E + 2.0 ** -18) * ref["cond"][0, 0] + 2.0 ** -8 * np.abs(ref["out"][0, 0])).all()
    assert np.abs(lse.double().cpu().numpy() - ref["lse"][0, 0]).max() <= E + 2.0 ** -17
    one = Case(row, 16, 64, [(1, 5)], k=3, seed=1, spread=0.0)  # nothing but rows of zeros, and one
    _logits_by_rope(one, torch.tensor([ahead, 0.0, 1.0, 0.0, 0.0]), torch.zeros((5, 512), device="cuda"))
    for keys, want in (([0, 1, 2], np.log(np.exp(ahead) + 1 + np.e)), ([2, -1, -1], 1.0)):
        one.topk = I32([keys])
        out, lse = one.run()
        _ok()
        assert not out.any() and np.abs(lse.double().cpu().numpy() - want).max() <= 2.0 ** -15


@pytest.mark.parametrize("row", FORMATS)
def test_rows_whose_scale_is_one(row):
    """Rows of scale 2^0 that are not zeros, among them one whose only code is its last, beside rows of zeros."""
    case = Case(row, 20, 16, [(3, 300), (1, 90)], k=128, seed=4, spread=0.0, scale=2e-3)
    n = case.pages * case.page
    g = torch.Generator(device="cuda").manual_seed(3)
    c = 300 * torch.sign(torch.randn((n, 512), generator=g, device="cuda")) * torch.rand((n, 512), generator=g, device="cuda")
    c[:, 5] = 400
    c[::7] = 0
    c[3::7, :511] = 0
    c[3::7, 511] = -420
    c[5::14] = -0.0
    r = torch.randn((n, 64), generator=g, device="cuda").to(torch.bfloat16)
    dsa.dsa_mla_quant_append(c.to(torch.bfloat16), r, torch.arange(n, device="cuda"), case.cache)
    case.check(random=False)
