"""GPU parity of the shared-prefix step (page plan, latent append, prefix attention) with the
64-bit oracle.

The plan is whole numbers: equal.  The append rounds once to bf16 (half a step, 2^-8) after a few
fp32 operations (2^-20 covers the 512-term sum, the root and the products).  Attention: the
logits are fp32 sums of 576 exact products, at most 576 * 2^-23 relative to `reach` (the largest
scaled sum of |q k|), which moves every probability by that much relatively, numerator and
denominator; probabilities enter P.V rounded to bf16 (2^-8 of each); n terms are summed in fp32
(n * 2^-23); the exponentials and the joins of partial sums are within 2^-20; the output is
rounded once (2^-8).  So
    |out - ref| <= (2^-8 + 2 E + 2^-20) * sum_s p_s |c_s| + 2^-8 |ref|,   E = 576 * 2^-23 * reach + n * 2^-23
    |lse - ref| <= E + 2^-20 + 2^-22 |ref|.
Cases with exact answers pin what those bounds could hide.
"""
import math

import numpy as np
import pytest
import torch

from oracle import prefix_step

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("sparse_attention_token_gb300")

H16, E23 = 2.0 ** -8, 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def _ok():
    torch.cuda.synchronize()
    assert dsa.dsa_check_device_status() == dsa.DSA_OK


# ---------------------------------------------------------------- page plan

def _plan_case(pairs, page, shared, extra_cols, seed, spare=3):
    """Requests (new, total after the step): tables holding what they held before, a free list."""
    g = torch.Generator().manual_seed(seed)
    width = max([1] + [-(-n // page) for _, n in pairs] + [shared]) + extra_cols
    perm = torch.randperm(sum(-(-n // page) + 2 for _, n in pairs) + shared + spare + 8, generator=g).to(torch.int32)
    prefix, at = perm[:shared], shared
    bt = torch.full((len(pairs), width), -7, dtype=torch.int32)
    need = 0
    for b, (q, n) in enumerate(pairs):
        held, have = -(-(n - q) // page), -(-n // page)
        own = max(held - shared, 0)
        bt[b, shared: shared + own] = perm[at: at + own]
        at += own
        need += max(have, shared) - max(held, shared) if n else 0
    return bt, prefix.contiguous(), perm[at: at + need + spare].contiguous()


def _check_plan(pairs, page, shared=0, extra_cols=0, pad=0, seed=0, spare=3, offset=0):
    bt, prefix, free = _plan_case(pairs, page, shared, extra_cols, seed, spare)
    q, n = [p[0] for p in pairs], [p[1] for p in pairs]
    total = sum(q) + pad
    ref = prefix_step.page_plan(q, n, bt, free, page_size=page, total_q=total, prefix_pages=prefix)
    dev = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
    gbt = torch.zeros(bt.numel() + offset, dtype=torch.int32, device="cuda")[offset:].view(bt.shape)
    gbt.copy_(bt)
    cu, slots, pos, used = dsa.dsa_page_plan(dev(q), dev(n), gbt, free.cuda(), page_size=page, total_q=total,
                                             prefix_pages=prefix.cuda() if shared else None)
    _ok()
    assert gbt.tolist() == ref[0]
    assert (cu.tolist(), slots.tolist(), pos.tolist(), used.item()) == (ref[1], ref[2], ref[3], ref[4])


@pytest.mark.parametrize("page", [1, 16, 24, 64])
def test_plan_decode(page):
    _check_plan([(1, 1), (1, 64), (1, 65), (1, 128), (1, 1000), (1, 129)], page, seed=page)


@pytest.mark.parametrize("shared", [1, 5])
@pytest.mark.parametrize("extra_cols", [0, 1, 2, 3])
def test_plan_prefix_and_widths(shared, extra_cols):
    s = 16 * shared
    _check_plan([(3, s + 3), (1, s + 1), (0, s), (0, 0), (40, s + 90), (1, s + 33)], 16, shared=shared,
                extra_cols=extra_cols, pad=5, seed=shared, offset=extra_cols)


def test_plan_prompts_and_padding():
    _check_plan([(700, 700), (1, 1), (5000, 5000), (64, 64), (0, 40)], 64, extra_cols=30, pad=100, seed=8)


@pytest.mark.parametrize("B", [255, 256, 257, 700])
def test_plan_many_requests(B):
    g = torch.Generator().manual_seed(B)
    q = torch.randint(0, 4, (B,), generator=g).tolist()
    n = [a + int(x) for a, x in zip(q, torch.randint(0, 300, (B,), generator=g))]
    _check_plan(list(zip(q, n)), 16, extra_cols=2, seed=B)


def test_plan_one_long_request():
    _check_plan([(20001, 50001)], 32, shared=4, extra_cols=7, seed=9)


def test_plan_no_requests_and_no_tokens():
    i32 = dict(dtype=torch.int32, device="cuda")
    e = torch.empty(0, **i32)
    cu, slots, pos, used = dsa.dsa_page_plan(e, e, torch.empty((0, 4), **i32), e, page_size=16, total_q=3)
    _ok()
    assert (cu.tolist(), slots.tolist(), pos.tolist(), used.tolist()) == ([0], [-1] * 3, [-1] * 3, [0])
    _check_plan([(0, 17), (0, 0)], 16)


def test_plan_short_free_list_is_reported_and_the_rest_is_right():
    bt, _, free = _plan_case([(20, 20), (20, 20), (20, 20)], 16, 0, 0, 4, spare=0)
    free = free[:3]  # six wanted
    ref = prefix_step.page_plan([20] * 3, [20] * 3, bt, free, page_size=16, total_q=60)
    g = bt.cuda()
    v = torch.full((3,), 20, dtype=torch.int32, device="cuda")
    cu, slots, pos, used = dsa.dsa_page_plan(v, v, g, free.cuda(), page_size=16, total_q=60)
    assert dsa.dsa_check_device_status() == dsa.DSA_ERR_DEVICE_CHECK
    assert g.tolist() == ref[0] and slots.tolist() == ref[2] and used.item() == 6


def test_plan_bad_lengths_are_reported_and_stay_inside():
    i32 = dict(dtype=torch.int32, device="cuda")
    guard = torch.full((4, 4), 5, **i32)
    q, n = torch.tensor([2, -1, 900], **i32), torch.tensor([1, 3, 1 << 30], **i32)
    out = torch.full((70,), -3, dtype=torch.int64, device="cuda")
    dsa.dsa_page_plan(q, n, guard[:3], torch.arange(20, **i32), page_size=16, total_q=64, slot_mapping=out[:64])
    assert dsa.dsa_check_device_status() == dsa.DSA_ERR_DEVICE_CHECK
    assert guard[3].tolist() == [5] * 4 and out[64:].tolist() == [-3] * 6


# ---------------------------------------------------------------- latent append

@pytest.mark.parametrize("n", [1, 2, 7, 64, 301])
@pytest.mark.parametrize("norm,rope,interleaved,views", [(True, True, False, True), (True, True, True, False),
                                                         (False, True, False, False), (True, False, False, True),
                                                         (False, False, False, True)])
def test_latent_append(n, norm, rope, interleaved, views):
    g = torch.Generator().manual_seed(n)
    page, pages = 16, 24
    kv = torch.randn((n, 640), generator=g).to(torch.bfloat16)
    c, r = kv[:, :512], kv[:, 512:576]
    if not views:
        c, r = c.contiguous(), r.contiguous()
    cc = torch.randn((pages, page, 512), generator=g).to(torch.bfloat16)
    cr = torch.randn((pages, page, 64), generator=g).to(torch.bfloat16)
    slots = torch.randperm(page * pages, generator=g)[:n]
    slots[1::5] = -1
    pos = torch.randint(0, 500, (n,), generator=g, dtype=torch.int32)
    ang = torch.rand((500, 32), generator=g) * 6.28
    kw = dict(norm_weight=1 + 0.1 * torch.randn(512, generator=g) if norm else None,
              rope_cos=ang.cos() if rope else None, rope_sin=ang.sin() if rope else None,
              positions=pos if rope else None, rope_interleaved=interleaved)
    ref_c, ref_r = prefix_step.latent_append(c, r, slots, cc, cr, **kw)
    gc, gr = cc.cuda(), cr.cuda()
    gkv = kv.cuda()
    dc, dr = (gkv[:, :512], gkv[:, 512:576]) if views else (c.cuda(), r.cuda())
    dsa.dsa_mla_cache_append(dc, dr, slots.cuda(), gc, gr,
                             **{k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in kw.items()})
    _ok()
    gc, gr = gc.double().cpu().numpy(), gr.double().cpu().numpy()
    assert np.all(np.abs(gc - ref_c) <= (H16 + 2.0 ** -20) * np.abs(ref_c) + 1e-30)
    # a pair's turn loses at most 2^-22 of the pair's length before it is rounded
    assert np.all(np.abs(gr - ref_r) <= H16 * np.abs(ref_r) + 2.0 ** -22 * np.abs(ref_r).max())
    live = np.zeros(page * pages, dtype=bool)
    live[slots[slots >= 0].numpy()] = True
    assert np.array_equal(gc.reshape(-1, 512)[~live], cc.double().numpy().reshape(-1, 512)[~live])
    if not norm:
        assert np.array_equal(gc, ref_c)


@pytest.mark.parametrize("n", [8195, 16387])
@pytest.mark.parametrize("interleaved", [False, True])
def test_latent_append_many_tokens(n, interleaved):
    # several tokens a warp: every row against the oracle's formula, written with numpy at once
    g = torch.Generator(device="cuda").manual_seed(n)
    page, pages = 32, 600
    kv = torch.randn((n, 576), generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.randperm(page * pages, generator=g, device="cuda")[:n]
    slots[3::1000] = -1
    pos = torch.randint(0, 300, (n,), generator=g, device="cuda", dtype=torch.int32)
    ang = torch.rand((300, 32), generator=g, device="cuda") * 6.28
    w = 1 + 0.1 * torch.randn(512, generator=g, device="cuda")
    gc = torch.full((pages, page, 512), 9.0, dtype=torch.bfloat16, device="cuda")
    gr = torch.full((pages, page, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_mla_cache_append(kv[:, :512], kv[:, 512:], slots, gc, gr, norm_weight=w, rope_cos=ang.cos(),
                             rope_sin=ang.sin(), positions=pos, rope_interleaved=interleaved)
    _ok()
    c, r = kv[:, :512].double().cpu().numpy(), kv[:, 512:].double().cpu().numpy()
    c = c / np.sqrt((c * c).mean(1, keepdims=True) + 1e-6) * w.double().cpu().numpy()
    p = pos.cpu().numpy()
    cos, sin = ang.cos().double().cpu().numpy()[p], ang.sin().double().cpu().numpy()[p]
    ia, ib = (np.arange(0, 64, 2), np.arange(1, 64, 2)) if interleaved else (np.arange(32), np.arange(32, 64))
    out = r.copy()
    out[:, ia], out[:, ib] = r[:, ia] * cos - r[:, ib] * sin, r[:, ia] * sin + r[:, ib] * cos
    sl = slots.cpu().numpy()
    live = sl >= 0
    fc, fr = gc.double().cpu().numpy().reshape(-1, 512), gr.double().cpu().numpy().reshape(-1, 64)
    assert np.all(np.abs(fc[sl[live]] - c[live]) <= (H16 + 2.0 ** -20) * np.abs(c[live]) + 1e-30)
    assert np.all(np.abs(fr[sl[live]] - out[live]) <= H16 * np.abs(out[live]) + 2.0 ** -22 * np.abs(out).max())
    rest = np.ones(len(fc), dtype=bool)
    rest[sl[live]] = False
    assert np.all(fc[rest] == 9) and np.all(fr[rest] == 9)


def test_latent_append_without_positions_uses_the_token_row():
    g = torch.Generator().manual_seed(2)
    kv = torch.randn((9, 576), generator=g).to(torch.bfloat16)
    ang = torch.rand((12, 32), generator=g)
    cc, cr = torch.zeros((1, 16, 512), dtype=torch.bfloat16), torch.zeros((1, 16, 64), dtype=torch.bfloat16)
    slots = torch.arange(9)
    _, ref = prefix_step.latent_append(kv[:, :512], kv[:, 512:], slots, cc, cr, rope_cos=ang.cos(), rope_sin=ang.sin())
    d = kv.cuda()
    gc, gr = cc.cuda(), cr.cuda()
    dsa.dsa_mla_cache_append(d[:, :512], d[:, 512:], slots.cuda(), gc, gr, rope_cos=ang.cos().cuda(),
                             rope_sin=ang.sin().cuda())
    _ok()
    assert np.all(np.abs(gr.double().cpu().numpy() - ref) <= H16 * np.abs(ref) + 2.0 ** -22 * np.abs(ref).max())


def test_latent_append_zero_row_and_bad_slots():
    d = torch.zeros((4, 576), dtype=torch.bfloat16, device="cuda")
    d[1:] = 1
    gc = torch.full((2, 16, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    gr = torch.full((2, 16, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(512, device="cuda")
    cos = torch.ones((5, 32), device="cuda")
    pos = torch.tensor([0, 1, 5, -1], dtype=torch.int32, device="cuda")   # two positions outside the tables
    slots = torch.tensor([0, 32, 2, 3], device="cuda")                    # one slot past the cache
    dsa.dsa_mla_cache_append(d[:, :512], d[:, 512:], slots, gc, gr, norm_weight=w, rope_cos=cos,
                             rope_sin=torch.zeros_like(cos), positions=pos)
    assert dsa.dsa_check_device_status() == dsa.DSA_ERR_DEVICE_CHECK
    assert torch.all(gc.view(-1, 512)[0] == 0) and torch.all(gr.view(-1, 64)[0] == 0)
    assert torch.all(gc.view(-1, 512)[1:] == 3) and torch.all(gr.view(-1, 64)[1:] == 3)


# ---------------------------------------------------------------- attention

class Case:
    def __init__(self, H, page, prefix, reqs, pad=0, seed=0, junk=None):
        """reqs: (new tokens, total length) of every request; junk: value of every cache row
        that no position below a sequence's length names."""
        g = torch.Generator().manual_seed(seed)
        self.prefix, self.scale, self.page = prefix, 576 ** -0.5, page
        n_pre = -(-prefix // page)
        per = [-(-n // page) for _, n in reqs]
        pages = n_pre + sum(per) + 2
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        self.pp = perm[:n_pre].contiguous()
        self.bt = torch.full((len(reqs), max([1] + per) + 1), -1, dtype=torch.int32)
        at = n_pre
        for b, k in enumerate(per):
            first = prefix // page  # whole prefix pages lie in front, as the page plan leaves them
            self.bt[b, :min(first, k)] = self.pp[:min(first, k)]
            self.bt[b, first:k] = perm[at: at + max(0, k - first)]
            at += max(0, k - first)
        cu = [0]
        for q, _ in reqs:
            cu.append(cu[-1] + q)
        T = cu[-1] + pad
        self.cu, self.lens = torch.tensor(cu, dtype=torch.int32), torch.tensor([n for _, n in reqs], dtype=torch.int32)
        rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
        self.cc, self.cr = rnd(pages, page, 512), rnd(pages, page, 64)
        self.qn, self.qr = rnd(T, H, 512), rnd(T, H, 64)
        if junk is not None:
            used = torch.zeros((pages, page), dtype=torch.bool)
            longest = max([n for _, n in reqs] + [0])
            for s in range(min(prefix, longest)):
                used[self.pp[s // page], s % page] = True
            for b, (_, n) in enumerate(reqs):
                for s in range(prefix, n):
                    used[self.bt[b, s // page], s % page] = True
            self.cc[~used], self.cr[~used] = junk, junk

    def gpu(self, **kw):
        d = lambda t: t.cuda()
        out, lse = dsa.dsa_prefix_mla(kw.pop("qn", d(self.qn)), kw.pop("qr", d(self.qr)), d(self.cc), d(self.cr),
                                      d(self.bt), d(self.cu), d(self.lens), d(self.pp), prefix_len=self.prefix,
                                      scale=self.scale, **kw)
        _ok()
        return out, lse

    def oracle(self):
        return prefix_step.prefix_mla(self.qn, self.qr, self.cc, self.cr, self.bt, self.cu, self.lens, self.pp,
                                      prefix_len=self.prefix, scale=self.scale)

    def check(self, got=None):
        out, lse = got or self.gpu()
        out, lse, ref = out.double().cpu().numpy(), lse.double().cpu().numpy(), self.oracle()
        empty = np.isneginf(ref["lse"])
        assert np.array_equal(np.isneginf(lse), empty)
        assert np.all(out[empty] == 0)
        err = 576 * E23 * ref["reach"] + E23 * ref["n"][:, None]
        tol = (H16 + 2 * err + 2.0 ** -20)[:, :, None] * ref["cond"] + H16 * np.abs(ref["out"])
        d = np.abs(out - ref["out"])
        assert np.all(d <= tol), f"{(d - tol).max():.3e} over the bound at {np.unravel_index((d - tol).argmax(), d.shape)}"
        live = ~empty
        dl = np.abs(lse[live] - ref["lse"][live])
        assert np.all(dl <= err[live] + 2.0 ** -20 + 2.0 ** -22 * np.abs(ref["lse"][live])), dl.max()


@pytest.mark.parametrize("H,page,prefix,reqs", [
    (16, 64, 1000, [(1, 1001), (1, 1065), (1, 1200)]),
    (64, 16, 129, [(3, 132), (0, 134), (1, 259), (0, 0)]),
    (128, 32, 513, [(2, 515), (1, 1200)]),
    (20, 128, 127, [(1, 128), (5, 204)]),
    (8, 64, 0, [(1, 1), (4, 300)]),
    (64, 64, 64, [(150, 214), (70, 464)]),
    (128, 64, 128, [(40, 168), (3, 131), (1, 700)]),
    (1, 16, 33, [(1, 34)]),
    (32, 32, 300, [(1, 301 + 17 * i) for i in range(9)]),
    (64, 128, 2000, [(1, 2001)]),
    (17, 16, 256, [(13, 280), (33, 300)]),
    (128, 64, 20000, [(1, 20001)]),
    (16, 16, 9000, [(1, 9001), (3, 9003), (1, 9777), (2, 9129)]),
    (48, 32, 640, [(1, 641 + 31 * i) for i in range(40)]),
    (100, 64, 1280, [(2, 1290), (9, 1400), (1, 1281)]),
    (2, 128, 384, [(200, 584), (1, 385), (64, 500)]),
], ids=str)
def test_attend(H, page, prefix, reqs):
    Case(H, page, prefix, reqs, seed=H + prefix).check()


@pytest.mark.parametrize("H,prefix", [(128, 20), (16, 40), (64, 0)])
def test_attend_more_requests_queries_and_tiles_than_a_plan_thread_each(H, prefix):
    # 1100 requests: own tiles, packed tiles, and no prefix; some idle, some seeing nothing
    reqs = [(1 if i % 7 else i % 3, prefix + 1 + i % 5 if i % 11 else 0) for i in range(1100)]
    reqs = [(q, max(n, q) if n else 0) for q, n in reqs]
    Case(H, 16, prefix, reqs, pad=3, seed=H).check()


@pytest.mark.parametrize("prefix", [127, 128, 129, 255, 256, 257])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_attend_around_tile_borders(prefix, page):
    Case(16, page, prefix, [(1, prefix + 1), (1, prefix + 127), (2, prefix + 129), (1, prefix + 64)], seed=prefix).check()


def test_attend_sequences_shorter_than_the_prefix_and_empty_rows():
    # positions before 0 see nothing; a sequence may end inside the prefix
    Case(32, 16, 100, [(1, 40), (3, 2), (2, 0), (1, 100), (1, 150)], pad=4, seed=5).check()


@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("H", [16, 64])
def test_attend_rows_nobody_sees_may_hold_anything(junk, H):
    Case(H, 64, 70, [(1, 71), (2, 200), (1, 133), (60, 190)], seed=6, junk=junk).check()


@pytest.mark.parametrize("H,prefix,reqs", [
    (128, 0, [(1, 100), (2, 90), (1, 1)]),          # tiles of one block, written without a join
    (64, 500, [(130, 700), (70, 900)]),             # tiles of a request, joined
    (16, 500, [(1, 501), (3, 700), (1, 800)]),      # tiles of several requests, joined with their own
], ids=str)
def test_attend_a_nan_in_a_query_stays_with_its_row(H, prefix, reqs):
    c = Case(H, 32, prefix, reqs, seed=12)
    out, lse = c.gpu()
    t, h = 2, H - 3
    for q in (c.qn, c.qr):
        q[t, h, 5] = math.nan
        got, got_lse = c.gpu()
        assert torch.all(torch.isnan(got[t, h])) and torch.isnan(got_lse[t, h])
        rest = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
        rest[t, h] = False
        assert torch.equal(got[rest], out[rest]) and torch.equal(got_lse[rest], lse[rest])


@pytest.mark.parametrize("H,prefix", [(128, 0), (64, 200), (16, 200)])
def test_attend_a_nan_in_a_key_reaches_every_row_of_its_request(H, prefix):
    c = Case(H, 32, prefix, [(1, prefix + 90), (1, prefix + 70)], seed=13)
    s = prefix + 60
    c.cr[int(c.bt[0, s // 32]), s % 32, 7] = math.nan
    out, lse = c.gpu()
    assert torch.all(torch.isnan(out[0])) and torch.all(torch.isnan(lse[0]))
    assert torch.all(torch.isfinite(out[1])) and torch.all(torch.isfinite(lse[1]))


def test_attend_one_key_is_its_row():
    c = Case(64, 16, 0, [(1, 1), (1, 1), (1, 1)], seed=7)
    out, lse = c.gpu()
    for b in range(3):
        assert torch.equal(out[b].cpu(), c.cc[int(c.bt[b, 0]), 0].expand(64, 512))


def test_attend_equal_logits_average():
    c = Case(16, 64, 500, [(1, 700), (3, 900)], seed=8)
    c.qn.zero_()
    c.qr.zero_()
    out, lse = c.gpu()
    ref = c.oracle()
    d = np.abs(out.double().cpu().numpy() - ref["out"])
    assert np.all(d <= (H16 + 2.0 ** -20) * np.abs(ref["out"]) + 1000 * E23 * ref["cond"])  # p = 1 exactly
    assert np.all(np.abs(lse.double().cpu().numpy() - ref["lse"]) <= 2.0 ** -20)


def test_attend_large_logits_and_late_maxima():
    # keys grow along the sequence, so the running maximum moves in every tile; logits of hundreds
    c = Case(16, 64, 700, [(1, 900), (2, 1500)], seed=9)
    grow = torch.linspace(0.5, 8.0, 700)
    for s in range(700):
        c.cc[int(c.pp[s // 64]), s % 64] = (c.cc[int(c.pp[s // 64]), s % 64].float() * grow[s]).to(torch.bfloat16)
    c.scale = 1.0
    c.check()


def test_attend_strided_queries():
    c = Case(20, 32, 90, [(2, 100), (1, 300)], seed=10)
    T, H = c.qn.shape[:2]
    q = torch.empty((H, T, 640), dtype=torch.bfloat16, device="cuda")  # heads outermost, rows padded
    q[:, :, :512], q[:, :, 512:576] = c.qn.transpose(0, 1).cuda(), c.qr.transpose(0, 1).cuda()
    c.check(c.gpu(qn=q[:, :, :512].transpose(0, 1), qr=q[:, :, 512:576].transpose(0, 1)))


def test_attend_is_the_same_every_time_and_in_a_graph_and_on_a_stream():
    c = Case(64, 64, 900, [(1, 950), (2, 1400), (1, 901)], seed=11)
    d = lambda t: t.cuda()
    args = [d(t) for t in (c.qn, c.qr, c.cc, c.cr, c.bt, c.cu, c.lens, c.pp)]
    kw = dict(prefix_len=c.prefix, scale=c.scale)
    first = dsa.dsa_prefix_mla(*args, **kw)
    again = dsa.dsa_prefix_mla(*args, **kw)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = dsa.dsa_prefix_mla(*args, stream=s, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = dsa.dsa_prefix_mla(*args, **kw)
    args[6].sub_(1)  # lengths are read on the device: the captured step follows them
    g.replay()
    torch.cuda.synchronize()
    _ok()
    for o in (again, other):
        assert torch.equal(first[0], o[0]) and torch.equal(first[1], o[1])
    shorter = dsa.dsa_prefix_mla(*args, **kw)
    assert torch.equal(held[0], shorter[0]) and torch.equal(held[1], shorter[1])
    assert not torch.equal(held[1], first[1])


def test_attend_bad_pages_are_reported_and_skipped():
    c = Case(16, 16, 64, [(1, 100), (1, 90)], seed=12)
    good = c.oracle()
    c.bt[0, 5] = 1 << 20
    c.bt[1, 4] = -1
    d = lambda t: t.cuda()
    out, lse = dsa.dsa_prefix_mla(d(c.qn), d(c.qr), d(c.cc), d(c.cr), d(c.bt), d(c.cu), d(c.lens), d(c.pp),
                                  prefix_len=c.prefix, scale=c.scale)
    assert dsa.dsa_check_device_status() == dsa.DSA_ERR_DEVICE_CHECK
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    assert np.all(lse.double().cpu().numpy() <= good["lse"] + 1e-4)     # fewer keys, smaller sums
    # a length past the table: what the table covers is used
    c = Case(16, 16, 64, [(1, 100)], seed=13)
    c.lens += 16 * c.bt.shape[1]
    dsa.dsa_prefix_mla(d(c.qn), d(c.qr), d(c.cc), d(c.cr), d(c.bt), d(c.cu), d(c.lens), d(c.pp), prefix_len=c.prefix,
                       scale=c.scale)
    assert dsa.dsa_check_device_status() == dsa.DSA_ERR_DEVICE_CHECK


def test_attend_far_pages_of_a_long_cache():
    # 4.6 GB of latent rows: element offsets pass 32 bits
    c = Case(16, 64, 130, [(1, 200), (1, 131)], seed=14)
    pages = 70000
    cc = torch.empty((pages, 64, 512), dtype=torch.bfloat16, device="cuda")
    cr = torch.empty((pages, 64, 64), dtype=torch.bfloat16, device="cuda")
    n = c.cc.shape[0]
    cc[-n:], cr[-n:] = c.cc.cuda(), c.cr.cuda()
    move = lambda t: torch.where(t >= 0, t + (pages - n), t).cuda()
    got = dsa.dsa_prefix_mla(c.qn.cuda(), c.qr.cuda(), cc, cr, move(c.bt), c.cu.cuda(), c.lens.cuda(), move(c.pp),
                             prefix_len=c.prefix, scale=c.scale)
    _ok()
    c.check(got)
    # the append writes there too
    kv = torch.randn((1, 576), device="cuda").to(torch.bfloat16)
    dsa.dsa_mla_cache_append(kv[:, :512], kv[:, 512:], torch.tensor([pages * 64 - 1], device="cuda"), cc, cr)
    _ok()
    assert torch.equal(cc[-1, -1], kv[0, :512]) and torch.equal(cr[-1, -1], kv[0, 512:])


def test_a_whole_step_behind_a_shared_prompt():
    """plan -> append -> attend over three decode steps, against the oracle on the written cache."""
    g = torch.Generator().manual_seed(15)
    page, H, prompt, B = 16, 16, 53, 3
    shared = prompt // page
    pages = 40
    cc, cr = torch.zeros((pages, page, 512), dtype=torch.bfloat16).cuda(), torch.zeros((pages, page, 64), dtype=torch.bfloat16).cuda()
    free = torch.randperm(pages, generator=g).to(torch.int32).cuda()
    prefix, free = free[:shared].contiguous(), free[shared:].contiguous()
    rows = torch.randn((prompt, 576), generator=g).to(torch.bfloat16).cuda()
    at = prefix.long()[torch.arange(shared * page, device="cuda") // page] * page + torch.arange(shared * page, device="cuda") % page
    dsa.dsa_mla_cache_append(rows[: shared * page, :512], rows[: shared * page, 512:], at, cc, cr)
    bt = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), shared * page, dtype=torch.int32, device="cuda")
    for step, new in enumerate([[7, 12, 40], [1, 1, 1], [1, 0, 2]]):
        q = torch.tensor(new, dtype=torch.int32, device="cuda")
        lens = lens + q
        T = sum(new)
        cu, slots, pos, used = dsa.dsa_page_plan(q, lens, bt, free, page_size=page, total_q=T, prefix_pages=prefix)
        kv = torch.randn((T, 576), generator=g).to(torch.bfloat16).cuda()
        dsa.dsa_mla_cache_append(kv[:, :512], kv[:, 512:], slots, cc, cr, norm_weight=torch.ones(512, device="cuda"))
        qq = torch.randn((T, H, 576), generator=g).to(torch.bfloat16).cuda()
        c = Case.__new__(Case)
        c.prefix, c.scale, c.page = shared * page, 576 ** -0.5, page
        c.qn, c.qr, c.cc, c.cr, c.bt, c.cu, c.lens, c.pp = (t.cpu() for t in (
            qq[..., :512], qq[..., 512:], cc, cr, bt, cu, lens, prefix))
        c.check(dsa.dsa_prefix_mla(qq[..., :512], qq[..., 512:], cc, cr, bt, cu, lens, prefix,
                                   prefix_len=shared * page, scale=c.scale))
        free = free[used.item():].contiguous()
    _ok()
