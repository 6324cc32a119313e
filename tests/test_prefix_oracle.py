"""Pins of the shared-prefix attention's oracle where pages are not there."""
import numpy as np
import torch

from oracle import prefix_step


def _args(seed=4):
    g = torch.Generator().manual_seed(seed)
    cc, cr = torch.randn((9, 4, 8), generator=g), torch.randn((9, 4, 4), generator=g)
    qn, qr = torch.randn((2, 3, 8), generator=g), torch.randn((2, 3, 4), generator=g)
    return qn, qr, cc, cr, torch.tensor([[4, 7, 1, 0]]), torch.tensor([0, 2]), torch.tensor([14]), torch.tensor([4, 2])


def _keys(a, where):
    """out, lse of every query over the rows (page, row, position) that it sees."""
    qn, qr, cc, cr = (t.double() for t in a[:4])
    out, lse = [], []
    for t, n in ((0, 13), (1, 14)):
        rows = [(p, i) for p, i, s in where if s < n]
        c, r = torch.stack([cc[p, i] for p, i in rows]), torch.stack([cr[p, i] for p, i in rows])
        x = (qn[t] @ c.T + qr[t] @ r.T) * 0.3
        out.append(torch.softmax(x, 1) @ c)
        lse.append(torch.logsumexp(x, 1))
    return torch.stack(out).numpy(), torch.stack(lse).numpy()


PREFIX = [(4, 0, 0), (4, 1, 1), (4, 2, 2), (4, 3, 3), (2, 0, 4), (2, 1, 5)]
OWN = [(7, 2, 6), (7, 3, 7), (1, 0, 8), (1, 1, 9), (1, 2, 10), (1, 3, 11), (0, 0, 12), (0, 1, 13)]


def _same(a, where):
    got = prefix_step.prefix_mla(*a, prefix_len=6, scale=0.3)
    out, lse = _keys(a, where)
    assert np.allclose(got["out"], out, atol=1e-12) and np.allclose(got["lse"], lse, atol=1e-12)
    return got


def test_every_page_there():
    assert _same(_args(), PREFIX + OWN)["n"].tolist() == [13, 14]


def test_pages_outside_the_cache_are_left_out():
    for bad in (-1, 9, 1 << 20):
        a = _args()
        a[4][0, 2] = bad
        assert _same(a, PREFIX + [w for w in OWN if w[0] != 1])["n"].tolist() == [9, 10]
        a = _args()
        a[7][0] = bad
        assert _same(a, [w for w in PREFIX if w[0] != 4] + OWN)["n"].tolist() == [9, 10]


def test_positions_past_the_table_are_left_out():
    a = list(_args())
    a[4] = a[4][:, :3].contiguous()
    assert _same(a, PREFIX + OWN[:6])["n"].tolist() == [12, 12]
    a[7] = a[7][:1].contiguous()
    assert _same(a, PREFIX[:4] + OWN[:6])["n"].tolist() == [10, 10]


def test_no_page_there_sees_nothing():
    a = _args()
    a[4].fill_(-1)
    a[7].fill_(-1)
    got = prefix_step.prefix_mla(*a, prefix_len=6, scale=0.3)
    assert np.all(got["out"] == 0) and np.all(np.isneginf(got["lse"])) and got["n"].tolist() == [0, 0]
