"""GPU parity of the attention over the quantised latent cache with the 64-bit oracle.

The rows are read back from the cache exactly (tested by itself), so what is compared is the attention alone.  Its errors:
  logits  a query row is held in two e4m3 terms: exact within 2^13 of its largest value, else off by 2^-21 of that at most
          (with fp16's own 2^-24: `small` times 2^-20 covers both); 576 exact products are summed in fp32 in two planes, at
          most 2 * 576 * 2^-23 relative to `reach`, the largest scaled sum of |q k|; a few fp32 roundings of the logit and of
          its row's exponent: 8 * 2^-24 of (reach log2(e) + 140)
  P       an e4m3 term and an e5m2 term of what it leaves: 2^-4 * 2^-3 of p, and fp16's 2^-11.  Below e4m3's normal numbers
          (p < 2^-6, where the largest is 2^5 at least) the first term is off by up to 2^-10, and the second by a whole step
          of it, 2^-2, as it is rounded up for some of 16 keys and down for others: 2^-12, with fp16's and e5m2's smallest
          steps 2^-17 each, against 2^5 in units of c / S:  `tail` times  T = 2^-17 + 2^-21
  sums    n fp32 additions in O, L and the joins: n * 2^-22, the exponentials 2^-20; the output is rounded once, 2^-8.  So
    |lse - ref| <= E + 2^-19 + 2^-22 |ref|,   E = 2^-20 small + 2^-13 reach + 2^-16 + n 2^-22
    |out - ref| <= (2 E + 2^-7 + 2^-11 + 2^-19) cond + T tail + 2^-8 |ref|
With random rows the roundings of P differ from key to key, each at most (2^-7 + 2^-11) p |c| or T, and no more than that over
sqrt(3) in the root mean square: eight of their root sums of squares stand in place of the sums.
"""
import numpy as np
import pytest
import torch

from oracle import quant_cache as qc

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("sparse_attention_token_gb300")

FORMATS = [qc.FP8, qc.FP4]
I32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def _ok():
    torch.cuda.synchronize()
    assert dsa.dsa_check_device_status() == dsa.DSA_OK


class Case:
    """A batch: requests (queries, length) over a cache of random rows; k selected keys a query, or all (None)."""

    def __init__(self, row, H, page, reqs, k=None, pad=0, seed=0, amp=1.0, spread=1.0, scale=0.07, extra_cols=1, spare=2):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.row, self.H, self.page, self.reqs, self.k, self.scale = row, H, page, reqs, k, scale
        B = len(reqs)
        need = [-(-n // page) for _, n in reqs]
        width = max(need + [0]) + extra_cols
        self.pages = sum(need) + spare
        perm = torch.randperm(self.pages, generator=torch.Generator().manual_seed(seed))
        bt, at = torch.full((B, width), -9, dtype=torch.int32), 0
        for b, m in enumerate(need):
            bt[b, :m] = perm[at: at + m].to(torch.int32)
            at += m
        self.bt = bt.cuda()
        self.cu = I32([0] + np.cumsum([q for q, _ in reqs]).tolist())
        self.lens = I32([n for _, n in reqs])
        self.live = sum(q for q, _ in reqs)
        self.T = self.live + pad
        rows = self.pages * page
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
        each = torch.exp(spread * rnd(rows, 1)) * amp
        self.cache = torch.full((self.pages, page, row), 255, dtype=torch.uint8, device="cuda")
        # rows of the spare pages and behind the sequences' ends keep bytes that are NaN in every part
        owned = torch.zeros((self.pages, page), dtype=torch.bool)
        for b, (_, n) in enumerate(reqs):
            for p in range(need[b]):
                owned[int(bt[b, p]), : min(page, n - p * page)] = True
        slots = torch.where(owned.view(-1), torch.arange(rows), torch.tensor(-1)).cuda()
        dsa.dsa_mla_quant_append((rnd(rows, 512) * each).to(torch.bfloat16), rnd(rows, 64).to(torch.bfloat16), slots, self.cache)
        self.q = rnd(self.T, H, 584).to(torch.bfloat16)
        if pad:
            self.q[self.live:] = float("nan")
        self.topk = None
        if k is not None:
            tk, gen = torch.full((self.T, k), -1, dtype=torch.int32), torch.Generator().manual_seed(seed + 2)
            t = 0
            for q, n in reqs:
                for i in range(q):
                    seen = max(0, n - q + i + 1)
                    sel = torch.randperm(seen, generator=gen)[: k].to(torch.int32)
                    tk[t, torch.randperm(k, generator=gen)[: len(sel)]] = sel
                    t += 1
            if pad:
                tk[self.live:] = 1
            self.topk = tk.cuda()

    def run(self, **kw):
        return dsa.dsa_quant_mla(self.q[..., :512], self.q[..., 512:576], self.cache, self.bt, self.cu, self.lens, self.topk,
                                 scale=self.scale, **kw)

    def reference(self):
        n = self.pages * self.page
        c, r = dsa.dsa_mla_quant_read(self.cache, torch.arange(self.pages, dtype=torch.int32, device="cuda")[None], I32([0, n]), total=n)
        raw = self.cache.view(n, self.row)
        if self.row == qc.FP8:
            S = raw[:, 640:644].contiguous().view(torch.float32)[:, 0].double()
        else:
            S = torch.exp2(((raw[:, 384:392] >> 7).long() << torch.arange(8, device="cuda")).sum(1).double() - 128)
        S = torch.where(torch.isfinite(S) & (S > 0) & (S < 1e30), S, 1.0).cpu().numpy()
        return qc.quant_mla(self.q[..., :512], self.q[..., 512:576], (qc.f64(c), qc.f64(r), S), self.bt, self.cu, self.lens, self.topk,
                            scale=float(np.float32(self.scale)), page_size=self.page, num_pages=self.pages)

    def check(self, random=True, ok=True, **kw):
        out, lse = self.run(**kw)
        if ok:
            _ok()
        ref = self.reference()
        compare(out, lse, ref, random)
        return out, lse, ref


def compare(out, lse, ref, random):
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    E = 2.0 ** -20 * ref["small"] + 2.0 ** -13 * ref["reach"] + 2.0 ** -16 + ref["n"][:, None] * 2.0 ** -22
    empty = ref["n"] == 0
    assert not o[empty].any() and (l[empty] == -np.inf).all()
    some = ~empty
    assert (np.abs(l[some] - ref["lse"][some]) <= (E + 2.0 ** -19 + 2.0 ** -22 * np.abs(ref["lse"]))[some]).all()
    p, T = 2.0 ** -7 + 2.0 ** -11, 2.0 ** -17 + 2.0 ** -21
    each, tail = p * ref["cond"], T * ref["tail"]
    if random:
        each, tail = np.minimum(each, 8 * 3 ** -0.5 * p * np.sqrt(ref["square"])), np.minimum(tail, 8 * 3 ** -0.5 * T * np.sqrt(ref["tail2"]))
    room = (2 * E[..., None] + 2.0 ** -19) * ref["cond"] + each + tail + 2.0 ** -8 * np.abs(ref["out"])
    assert np.isfinite(o).all()
    if random and some.sum() * o.shape[1] >= 64:  # and over all: the root mean squares of the roundings, half as much again
        sq = 2.0 ** -16 / 3 * np.mean(ref["out"] ** 2) + p * p / 3 * np.mean(ref["square"]) + T * T / 3 * np.mean(ref["tail2"])
        rest = 2.0 ** -17 * ref["reach"].max() * np.sqrt(np.mean(ref["cond"] ** 2))
        assert np.sqrt(np.mean((o - ref["out"]) ** 2)) <= 1.5 * np.sqrt(sq) + rest
    assert (np.abs(o - ref["out"]) <= room)[some].all()


REQS = [[(1, 1)], [(1, 64), (1, 65), (1, 63)], [(3, 3), (0, 70), (1, 129), (2, 200)], [(0, 0), (5, 130), (0, 0), (1, 700)]]


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("H,k", [(1, 1), (3, 7), (16, 64), (20, 65), (64, 130), (65, 333), (128, 128)])
@pytest.mark.parametrize("reqs", REQS, ids=range(len(REQS)))
def test_selected_keys(row, H, k, reqs):
    Case(row, H, 16, reqs, k=k, seed=H + k).check()


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("H,page", [(1, 1), (7, 24), (16, 64), (64, 16), (100, 96), (128, 7)])
@pytest.mark.parametrize("reqs", REQS, ids=range(len(REQS)))
def test_every_position(row, H, page, reqs):
    Case(row, H, page, reqs, seed=H + page).check()


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("k", [None, 96, 900])
@pytest.mark.parametrize("pad", [1, 40])
def test_padded_batches(row, k, pad):
    """Padding rows hold NaN queries and selections of their own: zeros and -inf all the same."""
    out, lse, _ = Case(row, 20, 32, [(2, 77), (0, 5), (1, 40)], k=k, pad=pad, seed=pad).check()
    assert not out[3:].any() and (lse[3:] == -float("inf")).all()


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("H,k,queries", [(16, 2048, 1), (128, 2048, 3), (64, 1001, 80), (64, 130, 200), (20, 64, 310), (128, 640, 90),
                                         (64, 640, 215), (64, 1001, 30), (20, 2048, 10), (1, 2048, 2), (33, 700, 5), (128, 1500, 60)])
def test_schedules(row, H, k, queries):
    """One tile in many pieces, rounds of whole tiles with a rest in pieces, rests that are not cut; pieces that go through
    memory and those of clusters of 2, 4 and 8."""
    Case(row, H, 64, [(queries, 2500)], k=k, seed=k).check()


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("H,reqs", [(16, [(1, 30000)]), (128, [(1, 20011), (1, 64)]), (64, [(1, 500 + 37 * i) for i in range(90)]),
                                    (20, [(70, 1000), (1, 5)]), (64, [(1, 1)] * 400), (16, [(2, 9000), (1, 1), (0, 3), (1, 4097)])])
def test_lines_of_every_position(row, H, reqs):
    Case(row, H, 64, reqs, seed=len(reqs)).check()


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("H,scale,spread", [(4, 0.1, 0.3), (13, 0.1, 0.3), (64, 0.1, 0.3), (64, 0.5, 1.0), (4, 0.5, 1.0)])
def test_a_maximum_that_keeps_rising(row, H, scale, spread):
    """Keys in the order of their logits, so that the reference moves in every block, for few heads and for all."""
    case = Case(row, H, 64, [(1, 1500)], k=1400, seed=H, scale=scale, spread=spread)
    first = case.q[0, 0, :576].double()
    n = case.pages * case.page
    c, r = dsa.dsa_mla_quant_read(case.cache, torch.arange(case.pages, dtype=torch.int32, device="cuda")[None], I32([0, n]), total=n)
    case.q[0, :] = case.q[0, 0]                      # every head rises
    pos = torch.arange(1500, device="cuda")
    at = case.bt[0].long()[pos // 64] * 64 + pos % 64
    logit = c[at].double() @ first[:512] + r[at].double() @ first[512:]
    case.topk = logit.argsort()[-1400:].to(torch.int32)[None].contiguous()
    up = case.check(random=False)
    case.topk = case.topk.flip(1).contiguous()       # and falls: the first block holds the maximum
    down = case.check(random=False)
    assert torch.allclose(up[1], down[1], rtol=1e-5, atol=1e-4)


@pytest.mark.parametrize("row", FORMATS)
def test_rows_of_very_different_scales(row):
    """Scales over 2^+-40 while logits stay moderate: the output is led by rows of little weight, the sum by others."""
    case = Case(row, 8, 16, [(3, 300), (1, 90)], k=128, seed=4, spread=9.0, scale=1e-3)
    case.q[..., :512] *= 1e-11
    case.check(random=False)


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("power", [-130, -70, 40, 90])
def test_large_and_small_queries(row, power):
    case = Case(row, 20, 16, [(2, 100)], k=64, seed=9)
    case.q = torch.ldexp(case.q.float(), torch.tensor(power, device="cuda")).to(torch.bfloat16)
    case.scale = 0.05 * 2.0 ** -power if abs(power) < 120 else 1.0
    case.check()


@pytest.mark.parametrize("row", FORMATS)
def test_equal_keys_and_one_key(row):
    """k copies of one row, named many times: out is the row itself (p cancels up to its rounding), lse = x + ln k."""
    case = Case(row, 64, 16, [(1, 200)], k=150, seed=3)
    case.topk[:] = 137
    out, lse, ref = case.check(random=False)
    assert ref["n"][0] == 150
    case.topk[:, 1:] = -1
    one, l1, _ = case.check(random=False)
    # one key: p = 2^5 exactly, so the row comes out as it stands
    assert np.array_equal(one.double().cpu().numpy(), case.reference()["out"].astype(np.float32).astype(np.float64))
    assert np.allclose((lse - l1).cpu().numpy(), np.log(150), atol=1e-4)


@pytest.mark.parametrize("row", FORMATS)
def test_sums_of_tails(row):
    """One key far ahead and 2000 behind it that together weigh as much: small p must not be lost."""
    case = Case(row, 16, 64, [(1, 2001)], k=2001, seed=6, spread=0.0, scale=1.0)
    case.q[:] = 0
    case.q[..., 512] = 1.0
    n = case.pages * case.page
    r = torch.zeros((n, 64), dtype=torch.bfloat16, device="cuda")
    slot0 = int(case.bt[0, 0]) * 64
    r[slot0, 0] = float(torch.tensor(np.log(2000.0)).to(torch.bfloat16))
    g = torch.Generator(device="cuda").manual_seed(8)
    c = torch.randn((n, 512), generator=g, device="cuda").to(torch.bfloat16)
    dsa.dsa_mla_quant_append(c, r, torch.arange(n, device="cuda"), case.cache)
    case.check(random=False)


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("sink", [0.0, 0.03125, 1.0])
@pytest.mark.parametrize("ahead", [9.0, 9.125, 9.3125, 9.5, 10.25])
def test_a_long_tail_of_equal_keys(row, ahead, sink):
    """One key ahead of 2047 equal ones that stand for a part of the output together: their roundings, a tenth of each, must
    not add up.  Over 16 keys the mean of the roundings is right to a 32nd of a step of 2^-2, 2^-7 of p.  Behind that stands
    fp16's smallest half step, 2^-17 against a largest p of 2^5: with 2^5 * exp(-ahead) * S / S_sink for p it is 2^-11 of p or
    less where the sink's own row is small, but counts where it is zeros, whose scale is 1."""
    case = Case(row, 16, 64, [(160, 2300)], k=2048, seed=6, spread=0.0, scale=1.0)  # enough queries that tiles stay whole
    case.q[:] = 0
    case.q[..., 512] = 1.0
    n = case.pages * case.page
    r = torch.zeros((n, 64), dtype=torch.bfloat16, device="cuda")
    r[int(case.bt[0, 0]) * 64, 0] = ahead
    g = torch.Generator(device="cuda").manual_seed(8)
    c = (1 + 0.25 * torch.randn((n, 512), generator=g, device="cuda")).to(torch.bfloat16)
    at = int(case.bt[0, 0]) * 64
    c[at] = sink * c[at]
    dsa.dsa_mla_quant_append(c, r, torch.arange(n, device="cuda"), case.cache)
    case.topk = (torch.arange(2048, dtype=torch.int32, device="cuda") + torch.arange(160, dtype=torch.int32, device="cuda")[:, None] * 0).contiguous()
    out, lse = case.run()
    _ok()
    case.q, case.topk = case.q[:1], case.topk[:1]    # every query sees the same keys
    case.cu, case.T = I32([0, 1]), 1
    ref = case.reference()
    err = np.abs(out.double().cpu().numpy() - ref["out"])
    T = 2.0 ** -17 + 2.0 ** -21
    assert (err <= (2.0 ** -7 + 2.0 ** -8 + 2.0 ** -10) * ref["cond"] + 8 * 3 ** -0.5 * T * np.sqrt(ref["tail2"])).all()
    E = [qc.row_exponent(x, row) for x in qc.f64(c[:200])]
    tail = 2.0 ** 5 * np.exp(-ahead) * 2.0 ** (min(E) - qc.row_exponent(qc.f64(c[at]), row))
    assert np.abs((out.double().mean().item() / ref["out"].mean() - 1)) <= 2.0 ** -7 + 2.0 ** -9 + 2.0 ** -17 / tail


@pytest.mark.parametrize("row", FORMATS)
def test_selections_outside_a_sequence_are_skipped(row):
    case = Case(row, 20, 16, [(2, 50), (1, 33)], k=70, seed=1)
    case.topk[0, :5] = torch.tensor([50, 51, 1 << 30, -7, -1 << 31], dtype=torch.int32, device="cuda")
    case.topk[1] = -1
    case.topk[2, 3:9] = 33
    out, lse, ref = case.check()
    assert ref["n"][1] == 0 and ref["n"][0] > 0


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("k", [None, 60])
@pytest.mark.parametrize("what", ["page", "table", "no pages", "no columns"])
def test_pages_that_are_not_there(row, k, what):
    case = Case(row, 20, 16, [(1, 90), (2, 40)], k=k, seed=2)
    if what == "page":
        case.bt[0, 2], case.bt[1, 0] = case.pages, -1
    elif what == "table":
        case.bt = case.bt[:, :4].contiguous()
    elif what == "no columns":
        case.bt = case.bt[:, :0].contiguous()
    else:
        case.cache, case.pages = case.cache[:0], 0
    out, lse = case.run()
    assert dsa.dsa_check_device_status() == dsa.DSA_ERR_DEVICE_CHECK
    if what in ("page", "table"):
        compare(out, lse, case.reference(), True)
    else:
        assert not out.any() and (lse == -float("inf")).all()


@pytest.mark.parametrize("k", [None, 64])
def test_odd_batches(k):
    row = qc.FP8
    assert Case(row, 8, 16, [(0, 20), (0, 0)], k=k).run()[0].shape == (0, 8, 512)
    case = Case(row, 8, 16, [(0, 20)], k=k, pad=3)           # nothing but padding
    out, lse, _ = case.check()
    case = Case(row, 8, 16, [], k=k, pad=2)                  # no requests
    out, lse = case.run()
    _ok()
    assert not out.any() and (lse == -float("inf")).all()
    case = Case(row, 8, 16, [(4, 2), (3, -1 + 1)], k=k)      # more queries than tokens: the first see nothing
    if k is None:
        case.check()


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("k", [None, 700])
def test_strides_and_own_buffers(row, k):
    case = Case(row, 24, 32, [(2, 900), (1, 1000)], k=k, seed=12)
    out, lse = case.run()
    flat = dsa.dsa_quant_mla(case.q[..., :512].contiguous(), case.q[..., 512:576].contiguous(), case.cache, case.bt, case.cu, case.lens,
                             case.topk, scale=case.scale)
    assert torch.equal(out, flat[0]) and torch.equal(lse, flat[1])
    heads = case.q.transpose(0, 1).contiguous().transpose(0, 1)  # heads further apart than tokens
    again = dsa.dsa_quant_mla(heads[..., :512], heads[..., 512:576], case.cache, case.bt, case.cu, case.lens, case.topk, scale=case.scale)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    need = dsa.dsa_quant_mla_workspace_size(case.T, case.H, k=k or 0)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    o, l = torch.full_like(out, float("nan")), torch.full_like(lse, float("nan"))
    got = case.run(out=o, lse=l, workspace=ws[:need])
    assert got[0] is o and torch.equal(o, out) and torch.equal(l, lse) and (ws[need:] == 255).all()
    _ok()


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("k", [None, 512])
def test_the_result_does_not_depend_on_the_run(row, k):
    case = Case(row, 64, 64, [(1, 3000), (2, 1500)] * 8, k=k, seed=20)
    first = case.run()
    for _ in range(5):
        out, lse = case.run()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    _ok()


def test_streams_and_graphs():
    """Two captured calls of different sizes share a workspace, replayed in turn with changed inputs, beside another stream."""
    cases = [Case(qc.FP8, 64, 64, [(1, 2000)] * 6, seed=1), Case(qc.FP4, 20, 32, [(3, 700), (1, 40)], k=300, seed=2),
             Case(qc.FP8, 16, 64, [(1, 4000)], k=2048, seed=3)]
    want = [c.run() for c in cases]
    ws = torch.empty(max(dsa.dsa_quant_mla_workspace_size(c.T, c.H, k=c.k or 0) for c in cases), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side, graphs, outs = torch.cuda.Stream(), [], []
    for c in cases:
        o, l = torch.empty((c.T, c.H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((c.T, c.H), device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(out=o, lse=l, workspace=ws)
        graphs.append(g)
        outs.append((o, l))
    other = Case(qc.FP8, 64, 64, [(1, 1000)] * 40, seed=5)
    alone = other.run()
    torch.cuda.synchronize()
    for _ in range(3):
        beside = other.run(stream=side)
        for i in (0, 1, 2, 0, 2, 1):
            outs[i][0].fill_(7), outs[i][1].fill_(7)
            graphs[i].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
        assert torch.equal(beside[0], alone[0])
    cases[0].lens.fill_(77)                      # a replay sees the lengths as they are then
    graphs[0].replay()
    _ok()
    cases[0].reqs = [(1, 77)] * 6
    compare(outs[0][0], outs[0][1], cases[0].reference(), True)


def test_offsets_past_32_bits():
    """A cache of more than 4 GB: rows at its end are written, read and attended to."""
    row, page = qc.FP8, 64
    pages = (5 << 30) // (row * page)
    cache = torch.empty((pages, page, row), dtype=torch.uint8, device="cuda")
    n = 500
    g = torch.Generator(device="cuda").manual_seed(1)
    c, r = torch.randn((n, 512), generator=g, device="cuda").to(torch.bfloat16), torch.randn((n, 64), generator=g, device="cuda").to(torch.bfloat16)
    bt = torch.arange(pages - 1, pages - 9, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    pos = torch.arange(n, device="cuda")
    slots = bt[0].long()[pos // page] * page + pos % page
    assert int(slots.max()) * row > 1 << 32
    dsa.dsa_mla_quant_append(c, r, slots, cache)
    small = torch.zeros((8, page, row), dtype=torch.uint8, device="cuda")
    dsa.dsa_mla_quant_append(c, r, pos, small)
    near = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    cu = I32([0, n])
    far_rows, near_rows = (dsa.dsa_mla_quant_read(x, t, cu, total=n) for x, t in ((cache, bt), (small, near)))
    assert torch.equal(far_rows[0], near_rows[0]) and torch.equal(far_rows[1], r)
    q = torch.randn((2, 40, 576), generator=g, device="cuda").to(torch.bfloat16)
    tk = torch.randint(0, n, (2, 200), generator=g, device="cuda", dtype=torch.int32)
    for topk in (None, tk):
        a, b = (dsa.dsa_quant_mla(q[..., :512], q[..., 512:], x, t, I32([0, 2]), I32([n]), topk, scale=0.05)
                for x, t in ((cache, bt), (small, near)))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    _ok()


@pytest.mark.parametrize("row", FORMATS)
def test_a_serving_run(row):
    """Pages planned, a prompt and then single tokens written, keys chosen by the indexer, attended to from the codes; the same
    steps over the bf16 rows that are read back agree to what the two attentions round."""
    g = torch.Generator(device="cuda").manual_seed(row)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    B, H, page, width, k, scale = 3, 16, 64, 7, 64, 0.06
    pages = B * width
    cache = torch.full((pages, page, row), 255, dtype=torch.uint8, device="cuda")
    kc, bt = torch.zeros((pages, page, 128), dtype=torch.bfloat16, device="cuda"), torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    w = 1 + 0.1 * rnd(512)
    ang = torch.rand((width * page, 32), generator=g, device="cuda") * 6.28
    lens, used = [0] * B, 0
    for q_lens in ([200, 70, 1], [1, 1, 1], [2, 0, 40], [1, 1, 1]):
        lens = [n + q for n, q in zip(lens, q_lens)]
        T = sum(q_lens)
        cu, slots, pos, n_used = dsa.dsa_page_plan(I32(q_lens), I32(lens), bt, free[used:].contiguous(), page_size=page, total_q=T)
        used += int(n_used)
        kv = rnd(T, 576).to(torch.bfloat16)
        dsa.dsa_mla_quant_append(kv[:, :512], kv[:, 512:], slots, cache, norm_weight=w, rope_cos=ang.cos(), rope_sin=ang.sin(), positions=pos)
        dsa.dsa_indexer_cache_append(rnd(T, 128).to(torch.bfloat16), slots, kc)
        topk = dsa.dsa_indexer(rnd(T, 32, 128).to(torch.bfloat16), rnd(T, 32), kc, cu, I32(lens), bt, max_seq_len=max(lens), topk_limit=k)
        q = rnd(T, H, 576).to(torch.bfloat16)
        qn, qr = q[..., :512].contiguous(), q[..., 512:].contiguous()
        seq = I32(lens)
        ends = I32([0] + np.cumsum(lens).tolist())
        own = torch.zeros((pages, page, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((pages, page, 64), dtype=torch.bfloat16, device="cuda")
        rows, rope = dsa.dsa_mla_quant_read(cache, bt, ends, total=int(ends[-1]))
        at = torch.cat([bt[b].long()[torch.arange(n, device="cuda") // page] * page + torch.arange(n, device="cuda") % page for b, n in enumerate(lens)])
        own[0].view(-1, 512)[at], own[1].view(-1, 64)[at] = rows, rope
        assert torch.isfinite(rows).all()
        _ok()
        # logits: the bound of this one and the other's 576 * 2^-23, on the largest sum of |q k| that there is
        reach = scale * (qn.abs().double().flatten(0, 1) @ rows.abs().double().T + qr.abs().double().flatten(0, 1) @ rope.abs().double().T).max()
        E = float(reach) * (2.0 ** -13 + 576 * 2.0 ** -23) + 2.0 ** -15
        for sel in (topk, None):
            out, lse = dsa.dsa_quant_mla(q[..., :512], q[..., 512:], cache, bt, cu, seq, sel, scale=scale)
            if sel is None:
                want, wl = dsa.dsa_prefix_mla(qn, qr, own[0], own[1], bt, cu, seq, prefix_len=0, scale=scale)
                assert (lse - wl).abs().max() <= E
            else:
                want = dsa.dsa_sparse_mla(qn, qr, own[0], own[1], bt, cu, seq, sel, scale=scale)
            _ok()
            # the roundings of P and of the output: 2^-7 + 2^-11 + 2^-8 here and 2^-7 there, of max |c| at most
            assert (out.float() - want.float()).abs().max() <= (2.0 ** -6 + 2.0 ** -8 + 2.0 ** -11 + 4 * E) * rows.abs().max().float()


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("k", [None, 90, 700])
def test_nan_in_a_query_stays_in_its_row(row, k):
    case = Case(row, 70, 16, [(2, 800), (1, 77)], k=k, seed=3)
    want = case.run()
    case.q[1, 66, 100] = float("nan")
    case.q[2, 3, 530] = float("nan")
    out, lse = case.run()
    _ok()
    for t, h in ((1, 66), (2, 3)):
        assert torch.isnan(lse[t, h]) and torch.isnan(out[t, h]).all()
        out[t, h], lse[t, h] = want[0][t, h], want[1][t, h]
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("args", [[], ["--bits", "4", "--requests", "3", "--heads", "20", "--prompt", "150", "--topk", "64", "--steps", "3"]])
def test_the_example_runs(args):
    import os
    import subprocess
    import sys
    script = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "quantised_cache_step.py")
    got = subprocess.run([sys.executable, script] + args, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stderr[-2000:]
    assert "decode:" in got.stdout and "nan" not in got.stdout
