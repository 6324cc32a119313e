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


def _many(row, n, ahead, lead_size, pattern=0, heads=128, requests=76):
    """`requests` x `heads` rows over the same n positions (as many tiles as SMs: each stays in one piece), one key in front of
    n - 1 that weigh alike: 64 pages, named again and again.  (out, lse, ref, cond, tail2 as in the oracle, E)."""
    g = torch.Generator(device="cuda").manual_seed(8)
    page, kinds = 64, 64
    cache = torch.full((1 + kinds, page, row), 255, dtype=torch.uint8, device="cuda")
    c = 1 + 0.25 * torch.randn(((1 + kinds) * page, 512), generator=g, device="cuda")
    if pattern:
        c *= torch.where((torch.arange(len(c), device="cuda") % pattern) < pattern // 2, 1.0, -1.0)[:, None]
    c[0] *= lead_size
    r = torch.zeros((len(c), 64), device="cuda")
    r[0, 0] = ahead
    dsa.dsa_mla_quant_append(c.to(torch.bfloat16), r.to(torch.bfloat16), torch.arange(len(c), device="cuda"), cache)
    cols = -(-n // page)
    order = torch.cat([torch.zeros(1, dtype=torch.int32), (1 + torch.arange(cols - 1) % kinds).to(torch.int32)])
    bt = order.cuda().repeat(requests, 1).contiguous()
    q = torch.zeros((requests, heads, 576), dtype=torch.bfloat16, device="cuda")
    q[..., 512] = 1.0
    out, lse = dsa.dsa_quant_mla(q[..., :512], q[..., 512:], cache, bt, I32(list(range(requests + 1))), I32([n] * requests), scale=1.0)
    _ok()
    rows = dsa.dsa_mla_quant_read(cache, torch.arange(1 + kinds, dtype=torch.int32, device="cuda")[None], I32([0, len(c)]), total=len(c))[0].double()
    # how often each row is seen: whole pages, and the last one up to its place
    times = torch.bincount(order[:-1].long(), minlength=1 + kinds).double()[:, None].repeat(1, page)
    times[order[-1], : n - (cols - 1) * page] += 1
    times = times.flatten().cuda()
    weight = times.clone()
    weight[0] *= float(np.exp(np.float64(torch.tensor(ahead).to(torch.bfloat16))))
    total = weight.sum()
    raw = cache.view(-1, row)
    if row == qc.FP8:
        S = raw[:, 640:644].contiguous().view(torch.float32)[:, 0].double()
    else:
        S = torch.exp2(((raw[:, 384:392] >> 7).long() << torch.arange(8, device="cuda")).sum(1).double() - 128)
    top = (torch.where(times > 0, weight / times.clamp(min=1), 0.0) / total * S).max()
    p = weight / total
    return (out.double(), lse.double(), p @ rows, p @ rows.abs(), top ** 2 * (times[:, None] * (rows / S[:, None]) ** 2).sum(0),
            torch.log(total), 8 * 2.0 ** -24 * (ahead * 1.4427 + 140))


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("n", [65536 + 37, 1 << 20])
@pytest.mark.parametrize("lead_size", [0.125, 1.0, 8.0])
@pytest.mark.parametrize("share", [16.0, 1.0, 0.125])
def test_a_long_tail_in_one_piece(row, n, lead_size, share):
    """All of the tail weighs `share` of the first key.  Its keys are as small as 2^-30 of that; their mean is held as that of
    large ones: 2^-7 and 2^-11 of them, which equal keys may be off alike.  Around the mean each value is off by the roundings of
    its own keys, at most a whole step of the second term, 2^-12 (and fp16's, 2^-16) against a largest p of 2^5 in units of c / S:
    eight root sums of squares of them.  Sums: fp32, each addition off by half a step, 2^-24 of the sum so far.  The sum of p has one
    addition of a block of 64 keys (and 2^3 within it), so n 2^-30; O one of every 32 keys for each term, a whole step off if it is
    cut instead of rounded, so n / 16 of 2^-23."""
    ahead = float(torch.tensor(np.log(n / share)).to(torch.bfloat16))
    out, lse, ref, cond, tail2, total, E = _many(row, n, ahead, lead_size)
    assert (lse - total).abs().max() <= E + 2.0 ** -17 + n * 2.0 ** -30
    T, sums = 2.0 ** -17 + 2.0 ** -21, n * 2.0 ** -30 + n * 2.0 ** -27
    assert ((out - ref).abs() <= (P + 2 * E + 2.0 ** -14 + sums) * cond + 2.0 ** -8 * ref.abs() + 8 * T * tail2.sqrt()).all()
    assert ((out.mean(2) - ref.mean()).abs() <= (P + 2 * E + 2.0 ** -14 + 2.0 ** -11 + sums) * cond.mean()).all()


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("pattern", [2, 4, 8, 16, 32, 64])
@pytest.mark.parametrize("share", [1.0, 0.02])
def test_a_tail_whose_values_go_with_the_place(row, pattern, share):
    """The values change their sign every few positions: a rounding that goes with the place would show as their sum."""
    n = 65536
    ahead = float(torch.tensor(np.log(n / share)).to(torch.bfloat16))
    out, lse, ref, cond, tail2, total, E = _many(row, n, ahead, 1 / 64, pattern=pattern)
    T = 2.0 ** -17 + 2.0 ** -21
    assert ((out - ref).abs() <= (P + 2 * E + 2.0 ** -14) * cond + 2.0 ** -8 * ref.abs() + 8 * T * tail2.sqrt()).all()
    assert ((out.mean(2) - ref.mean()).abs() <= (P + 2 * E + 2.0 ** -14 + 2.0 ** -11) * cond.mean()).all()


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("sink", [0.0, 0.03125, 8.0])
@pytest.mark.parametrize("ahead", [9.0, 9.5, 10.25, 10.5, 12.0, 13.0])
def test_the_mean_of_selected_tails(row, sink, ahead):
    """One key ahead of 2047 selected ones alike: the output's mean is right to what equal keys may be off alike, 2^-7 and 2^-11,
    whatever the first key's row holds."""
    case = Case(row, 16, 64, [(160, 2300)], k=2048, seed=6, spread=0.0)
    lead = torch.zeros(2048)
    lead[0] = ahead
    g = torch.Generator(device="cuda").manual_seed(8)
    c = 1 + 0.25 * torch.randn((2048, 512), generator=g, device="cuda")
    c[0] *= sink
    _logits_by_rope(case, lead, c)
    case.topk = torch.arange(2048, dtype=torch.int32, device="cuda").repeat(case.T, 1).contiguous()
    out, lse = case.run()
    _ok()
    ref = _one_query(case)
    o, want = out.double().cpu().numpy(), ref["out"][0, 0]
    E = 8 * 2.0 ** -24 * (ahead * 1.4427 + 140)
    assert np.abs(lse.double().cpu().numpy() - ref["lse"][0, 0]).max() <= E + 2.0 ** -17
    assert (np.abs(o.mean(2) - want.mean()) <= (P + 2 * E + 2.0 ** -11) * np.abs(want).mean()).all()
