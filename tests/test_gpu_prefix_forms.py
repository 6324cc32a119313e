"""Forms of the shared-prefix attention beside those of test_gpu_prefix_step.py, with its bounds:
batches of many requests, of mixed requests and of long prompts, the caller's own buffers, calls
side by side, pages and lengths that are not there, and sizes that pass 32 bits in the plan."""
import pytest
import torch

from test_gpu_prefix_step import Case, dsa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("H,requests", [(8, 300), (20, 131), (1, 400)])
def test_many_requests_with_keys_of_their_own(H, requests):
    # whole own tiles of few rows that straddle the blocks of 128 rows which their results stand in
    reqs = [(1 + i % 3 if i % 7 else 0, 201 + (37 * i) % 400) for i in range(requests)]
    Case(H, 16, 200, reqs, pad=2, seed=H).check()


MIXED = [
    (16, 300, [(1, 301 + 3 * i) for i in range(40)] + [(130, 450)]),             # one chunk among single tokens
    (16, 300, [(130, 450)] + [(1, 301 + 3 * i) for i in range(40)]),
    (64, 140, [(1, 150)] * 3 + [(90, 300), (1, 141), (0, 200), (77, 230)]),
    (20, 129, [(2, 140)] * 12 + [(0, 0)] * 5 + [(100, 229)] + [(0, 131)] * 4),
    (16, 200, [(0, 210)] * 20 + [(160, 400)] + [(0, 0)] * 20),                   # idle requests around one prompt
    (16, 200, [(1, 230)] * 2 + [(250, 470), (240, 450)]),                        # hardly any empty rows: own tiles
]


@pytest.mark.parametrize("H,prefix,reqs", MIXED, ids=range(len(MIXED)))
@pytest.mark.parametrize("pad", [0, 37])
def test_mixed_requests(H, prefix, reqs, pad):
    Case(H, 32, prefix, reqs, pad=pad, seed=H + prefix).check()


def _ms(call, n=20):
    for _ in range(3):
        call()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    for _ in range(n):
        call()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n


def test_a_chunk_among_single_tokens_shares_the_prefix():
    """127 single tokens x 16 heads fill 16 tiles of 128 rows, a chunk of 800 tokens 100.  Apart they
    cost 16 and 100 walks of the prefix, together they need 116; with a tile for every single token
    they would be 227."""
    prefix, page, H = 32768, 64, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    i32 = lambda t: torch.as_tensor(t).to(torch.int32).cuda()
    shared, per = prefix // page, 13
    cc, cr = rnd(shared + 128 * per, page, 512), rnd(shared + 128 * per, page, 64)

    def batch(new):
        own = shared + torch.arange(len(new) * per).view(-1, per)
        bt = torch.cat([torch.arange(shared).expand(len(new), -1), own], 1)
        cu = torch.cat([torch.zeros(1, dtype=torch.int64), torch.tensor(new).cumsum(0)])
        q = rnd(sum(new), H, 576)
        args = (q[..., :512], q[..., 512:], cc, cr, i32(bt), i32(cu), i32(prefix + torch.tensor(new)),
                i32(torch.arange(shared)))
        return _ms(lambda: dsa.dsa_prefix_mla(*args, prefix_len=prefix, scale=576 ** -0.5))

    apart = batch([1] * 127) + batch([800])
    together = batch([1] * 127 + [800])
    assert dsa.dsa_check_device_status() == dsa.DSA_OK
    assert together < 1.3 * apart, (together, apart)


def _check_reported(c):
    """The call reports what is not there, and its results are those of the keys that are."""
    d = lambda t: t.cuda()
    got = dsa.dsa_prefix_mla(d(c.qn), d(c.qr), d(c.cc), d(c.cr), d(c.bt), d(c.cu), d(c.lens), d(c.pp),
                             prefix_len=c.prefix, scale=c.scale)
    assert dsa.dsa_check_device_status() == dsa.DSA_ERR_DEVICE_CHECK
    c.check(got)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("H", [16, 128])  # prefix tiles shared by the requests, and tiles of their own
@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_pages_that_are_not_there_are_left_out(page, H, bad):
    prefix = 3 * page + 5
    reqs = [(1, prefix + 200), (3, prefix + 150), (1, prefix + 1), (2, prefix + 2 * page)]
    c = Case(H, page, prefix, reqs, seed=page)
    c.bt[0, 4] = bad                    # a whole page of one request
    c.bt[1, (prefix + 149) // page] = bad  # its newest keys
    c.bt[3, 3] = bad                    # the page that begins with the prefix's last keys
    _check_reported(c)
    c = Case(H, page, prefix, reqs, seed=page + 1)
    c.pp[1] = bad                       # a page of the prefix, for all of them
    _check_reported(c)
    c = Case(H, page, prefix, [(1, 3)] + reqs[1:], seed=page + 2)
    c.pp[0] = len(c.cc)                 # the first page behind the cache: all that a short request sees
    _check_reported(c)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("H", [16, 128])
def test_lengths_past_the_table_are_cut(page, H):
    prefix = 2 * page
    c = Case(H, page, prefix, [(1, prefix + page), (2, prefix + 50), (4, prefix + 3 * page)], seed=page)
    width = c.bt.shape[1]
    c.bt[0, 3:] = torch.arange(1, width - 2)   # the request's table is full: every page somebody's
    c.lens[0] = width * page + 7               # and its length beyond it
    c.lens[2] = width * page + 2               # some of its queries see all of the table, some less
    c.bt[2, c.bt[2] < 0] = 0
    _check_reported(c)


def test_the_callers_buffers():
    c = Case(20, 32, 300, [(1, 301 + 40 * i) for i in range(9)] + [(30, 400)], pad=3, seed=21)
    ref = c.gpu()
    T, H = c.qn.shape[:2]
    need = dsa.dsa_prefix_mla_workspace_size(len(c.lens), T, H, prefix_len=c.prefix)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((T + 2, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 2, H), 7.0, device="cuda")
    got = c.gpu(out=out[1:-1], lse=lse[1:-1], workspace=ws[:need])
    assert got[0].data_ptr() == out[1].data_ptr() and got[1].data_ptr() == lse[1].data_ptr()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    # nothing written beside them
    assert torch.all(ws[need:] == 0xA5)
    assert torch.all(out[0] == 7) and torch.all(out[-1] == 7) and torch.all(lse[0] == 7) and torch.all(lse[-1] == 7)
    # a workspace that another batch left behind
    ws[:need] = 0xFF
    again = c.gpu(out=out[1:-1], lse=lse[1:-1], workspace=ws[:need])
    assert torch.equal(again[0], ref[0]) and torch.equal(again[1], ref[1])
    with pytest.raises(dsa.DsaError) as e:
        c.gpu(workspace=ws[: need - 1])
    assert e.value.status == dsa.DSA_ERR_WORKSPACE


def test_a_long_prompt_behind_a_prefix():
    Case(8, 64, 200, [(1000, 1200), (1, 260), (333, 533)], seed=22).check()
    Case(128, 32, 0, [(300, 300)], seed=23).check()


def test_calls_side_by_side_on_two_streams():
    cases = [Case(64, 64, 900, [(1, 950), (2, 1400), (1, 901)], seed=24),
             Case(16, 32, 500, [(1, 501 + i) for i in range(40)], seed=25)]
    d = lambda t: t.cuda()
    args = [[d(t) for t in (c.qn, c.qr, c.cc, c.cr, c.bt, c.cu, c.lens, c.pp)] for c in cases]
    kw = [dict(prefix_len=c.prefix, scale=c.scale) for c in cases]
    ref = [dsa.dsa_prefix_mla(*a, **k) for a, k in zip(args, kw)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        for a, k, s in zip(args, kw, streams):
            got.append(dsa.dsa_prefix_mla(*a, stream=s, **k))
    torch.cuda.synchronize()
    assert dsa.dsa_check_device_status() == dsa.DSA_OK
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, ref[i % 2][0]) and torch.equal(lse, ref[i % 2][1])


@pytest.mark.parametrize("H,reqs,width", [
    (128, [(140, 190)], 16_000_000),                               # own tiles, written without a join
    (80, [(5, 60 + 9 * i) for i in range(20)], 15_000_000),       # shared tiles
])
def test_tables_so_wide_that_the_plan_counts_in_64_bits(H, reqs, width):
    """Tables of 15 million pages of 128 rows: 2^31 blocks of keys and more over the tiles there is
    room for, whatever the lengths turn out to be."""
    c = Case(H, 128, 40, reqs, seed=26)
    wide = torch.full((len(reqs), width), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.bt.shape[1]] = c.bt.cuda()
    d = lambda t: t.cuda()
    got = dsa.dsa_prefix_mla(d(c.qn), d(c.qr), d(c.cc), d(c.cr), wide, d(c.cu), d(c.lens), d(c.pp),
                             prefix_len=c.prefix, scale=c.scale)
    assert dsa.dsa_check_device_status() == dsa.DSA_OK
    c.check(got)


@pytest.mark.slow
def test_so_many_blocks_that_the_plan_cuts_them_in_64_bits():
    """1024 tiles behind 7.3 million keys (some 57000 blocks each; about a second): more than 2^32
    places times parts.  The keys are 1024 rows over and over, so query i sees each of them
    `times` - 1 times and the first i + 1 once more, and the sums are known.

    A running sum takes one fp32 addition a block, 57000 * 2^-24 = 0.0034 relative at most, the
    logits 576 * 2^-23 * reach; a lost, doubled or misplaced piece moves lse by far more."""
    times, rows, H, page = 7130, 1024, 128, 128
    prefix = times * rows
    g = torch.Generator(device="cuda").manual_seed(27)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    cc, cr, q = rnd(rows // page, page, 512), rnd(rows // page, page, 64), rnd(rows, H, 576)
    i32 = lambda t: t.to(torch.int32).cuda()
    scale = 576 ** -0.5
    out, lse = dsa.dsa_prefix_mla(q[..., :512], q[..., 512:], cc, cr, torch.full((1, 1), -1, dtype=torch.int32, device="cuda"),
                                  i32(torch.tensor([0, rows])), i32(torch.tensor([prefix])),
                                  i32(torch.arange(prefix // page) % (rows // page)), prefix_len=prefix, scale=scale)
    assert dsa.dsa_check_device_status() == dsa.DSA_OK
    k = torch.cat([cc.view(rows, 512), cr.view(rows, 64)], 1).double()
    for i in range(0, rows, 64):
        qi = q[i: i + 64].double()
        x = torch.einsum("thd,sd->ths", qi, k) * scale
        reach = (qi.abs().float().flatten(0, 1) @ k.abs().float().T).amax(1).view(64, H).double() * scale * 1.001
        count = (times - 1) + (torch.arange(rows, device="cuda") <= torch.arange(i, i + 64, device="cuda")[:, None]).double()
        m = x.amax(2, keepdim=True)
        e = torch.exp(x - m) * count[:, None, :]
        total = e.sum(2, keepdim=True)
        ref = (m + total.log())[:, :, 0]
        tol = 576 * 2.0 ** -23 * reach + 57100 * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * ref.abs()
        assert torch.all((lse[i: i + 64].double() - ref).abs() <= tol)
        if i % 256:
            continue
        p = e / total
        # 8 fp32 additions a block into the tile's sums, each of at most 2^-23 of what is there
        cond = torch.einsum("ths,sd->thd", p, k[:, :512].abs())
        o = torch.einsum("ths,sd->thd", p, k[:, :512])
        bound = (2.0 ** -8 + 2 * tol.amax() + 8 * 57100 * 2.0 ** -23) * cond + 2.0 ** -8 * o.abs()
        assert torch.all((out[i: i + 64].double() - o).abs() <= bound)


def test_one_token_and_one_head_in_tensors_of_odd_strides():
    g = torch.Generator(device="cuda").manual_seed(28)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    # one token's row in a tensor whose rows are no multiples of 16 bytes apart
    kv = rnd(1, 577)
    gc, gr = torch.zeros((2, 16, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 16, 64), dtype=torch.bfloat16, device="cuda")
    dsa.dsa_mla_cache_append(kv[:, :512], kv[:, 512:576], torch.tensor([19], device="cuda"), gc, gr)
    assert dsa.dsa_check_device_status() == dsa.DSA_OK
    assert torch.equal(gc[1, 3], kv[0, :512]) and torch.equal(gr[1, 3], kv[0, 512:576])
    for H, reqs in ((16, [(1, 200)]), (1, [(3, 200), (1, 150)])):
        c = Case(H, 32, 90, reqs, seed=29)
        T = c.qn.shape[0]
        store = torch.zeros(T * H * 600 + 8, dtype=torch.bfloat16, device="cuda")
        # rows 592 apart; the stride of the dimension of size 1 is 577
        st, sh = (577, 592) if T == 1 else (592, 577)
        qn, qr = store.as_strided((T, H, 512), (st, sh, 1)), store.as_strided((T, H, 64), (st, sh, 1), 512)
        qn.copy_(c.qn)
        qr.copy_(c.qr)
        c.check(c.gpu(qn=qn, qr=qr))


@pytest.mark.slow
@pytest.mark.parametrize("H,reqs", [(1, [(1, 300)]), (16, [(1, 300), (2, 200)])])
def test_a_length_at_the_end_of_32_bits(H, reqs):
    """A table of 2^24 + 2 pages of 128 rows covers 2^31 + 256 positions; a length of 2^31 - 1 is cut
    where the block counts still fit, and the pages that are there give the result."""
    c = Case(H, 128, 140, reqs, seed=30)
    wide = torch.full((len(reqs), (1 << 24) + 2), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.bt.shape[1]] = c.bt.cuda()
    c.lens[0] = (1 << 31) - 1
    d = lambda t: t.cuda()
    got = dsa.dsa_prefix_mla(d(c.qn), d(c.qr), d(c.cc), d(c.cr), wide, d(c.cu), d(c.lens), d(c.pp),
                             prefix_len=c.prefix, scale=c.scale)
    assert dsa.dsa_check_device_status() == dsa.DSA_ERR_DEVICE_CHECK
    c.lens[0] = c.bt.shape[1] * 128  # the oracle: all that the pages hold
    c.check(got)
