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


@pytest.mark.parametrize("row", FORMATS)
def test_the_sign_of_zeros(row):
    """-0 is written as -0 by rows that are taken once and by those, one in some 100, that are taken again."""
    n = 1200
    g = torch.Generator().manual_seed(1)
    c = torch.randn((n, 512), generator=g).to(torch.bfloat16)
    c[:, ::3] = -0.0
    c[:, 1::3] = 0.0
    w = 1 + 0.1 * torch.randn(512, generator=g)
    cache = torch.zeros((1, n, row), dtype=torch.uint8, device="cuda")
    dsa.dsa_mla_quant_append(c.cuda(), torch.zeros((n, 64), dtype=torch.bfloat16, device="cuda"), torch.arange(n).cuda(), cache,
                             norm_weight=w.cuda())
    _ok()
    got = cache[0].cpu().numpy()
    lc, lr = qc.latent(c, torch.zeros((n, 64), dtype=torch.bfloat16), norm_weight=w)
    want = [qc.encode_row(a, b, row) for a, b in zip(lc, lr)]
    assert (got == want).all()


@pytest.mark.parametrize("row", FORMATS)
def test_read_leaves_rows_before_the_first_request(row):
    """Offsets that begin behind other rows of the output: those are no request's, and starts do not move into them."""
    case = Case(row, 1, 16, [(1, 40), (1, 25)], seed=2)
    every = dsa.dsa_mla_quant_read(case.cache, case.bt, I32([0, 12, 17]), total=17, starts=I32([20, 3]))
    c, r = torch.full((40, 512), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((40, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_mla_quant_read(case.cache, case.bt, I32([10, 22, 27]), total=40, starts=I32([20, 3]), c_kv=c, k_rope=r)
    _ok()
    assert (c[:10] == 9).all() and (r[:10] == 9).all() and (c[27:] == 9).all() and (r[27:] == 9).all()
    assert torch.equal(c[10:27], every[0]) and torch.equal(r[10:27], every[1])


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-30])
@pytest.mark.parametrize("power", [-45, -52, -66, -75, -100, -125])
def test_norms_of_small_rows(row, eps, power):
    """Rows whose squares fp32 cannot hold: the norm is that of the values all the same, or what the epsilon leaves of them."""
    g = torch.Generator().manual_seed(-power)
    c = torch.ldexp(torch.randn((7, 512), generator=g), torch.tensor(power)).to(torch.bfloat16)
    c[3] = 0
    r = torch.randn((7, 64), generator=g).to(torch.bfloat16)
    w = 1 + 0.1 * torch.randn(512, generator=g)
    cache = torch.zeros((1, 7, row), dtype=torch.uint8, device="cuda")
    dsa.dsa_mla_quant_append(c.cuda(), r.cuda(), torch.arange(7).cuda(), cache, norm_weight=w.cuda(), norm_eps=eps)
    _ok()
    got = cache[0].cpu().numpy()
    live = [0, 1, 2, 4, 5, 6]
    lc, lr = qc.latent(c[live], r[live], norm_weight=w, norm_eps=eps)
    assert (got[live] == [qc.encode_row(a, b, row) for a, b in zip(lc, lr)]).all()
    assert not qc.decode_row(got[3])[0].any()


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("norm,n", [(True, 2047), (True, 2048), (True, 2051), (True, 8191), (True, 8195), (False, 4095), (False, 4097),
                                    (False, 16383), (False, 16387)])
def test_the_number_of_tokens_a_warp_does_not_matter(row, norm, n):
    """Both sides of the rule for one, two and four tokens a warp: the same bytes as from calls of a few rows."""
    g = torch.Generator(device="cuda").manual_seed(n)
    c = torch.randn((n, 512), generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn((n, 64), generator=g, device="cuda").to(torch.bfloat16)
    kw = dict(norm_weight=1 + 0.1 * torch.randn(512, generator=g, device="cuda")) if norm else {}
    slots = torch.randperm(n + 9, generator=g, device="cuda")[:n]
    slots[::11] = -1
    one, many = (torch.full((-(-(n + 9) // 64), 64, row), 3, dtype=torch.uint8, device="cuda") for _ in range(2))
    dsa.dsa_mla_quant_append(c, r, slots.contiguous(), one, **kw)
    for i in range(0, n, 1000):
        dsa.dsa_mla_quant_append(c[i: i + 1000], r[i: i + 1000], slots[i: i + 1000].contiguous(), many, **kw)
    _ok()
    assert torch.equal(one, many)
