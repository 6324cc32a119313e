"""GPU parity of the quantised latent cache's writing and reading with the 64-bit oracle.

Codes and scales are whole decisions: equal, byte by byte, wherever no value lies within 2^-40 of a border (the inputs
are chosen or drawn so).  The rotary part is rounded once to bf16 after an fp32 rotation (half a step, 2^-8, and 2^-22 of
the pair's length); without a rotation it is exact.  Reading back rounds nothing.
"""
import numpy as np
import pytest
import torch

from oracle import quant_cache as qc

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("sparse_attention_token_gb300")

FORMATS = [qc.FP8, qc.FP4]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def _ok():
    torch.cuda.synchronize()
    assert dsa.dsa_check_device_status() == dsa.DSA_OK


def _split(rows, row):
    """(codes and scales, rotary part as bf16) of rows of bytes."""
    at = 512 if row == qc.FP8 else 256
    return np.concatenate([rows[:, :at], rows[:, at + 128:]], 1), rows[:, at:at + 128].copy().view(np.uint16)


def _bf16(u16):
    return (u16.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def _append_and_compare(c, r, slots, row, page=16, pages=24, tail=(), **kw):
    """Writes the rows through the library into a cache of known bytes and compares every byte of it."""
    g = torch.Generator().manual_seed(5)
    cache = torch.randint(0, 256, (pages, page, row), generator=g, dtype=torch.uint8)
    dev = cache.cuda()
    to = lambda v: v.cuda() if isinstance(v, torch.Tensor) else v
    dsa.dsa_mla_quant_append(to(c), to(r), slots.cuda(), dev, **{k: to(v) for k, v in kw.items()})
    _ok()
    got, want = dev.cpu().numpy().reshape(-1, row), cache.numpy().reshape(-1, row).copy()
    lc, lr = qc.latent(c, r, **kw)
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s] = qc.encode_row(lc[t], lr[t], row)
    if row == qc.FP8:  # the twelve bytes behind a row's scale are written as zeros
        assert not got[slots[slots >= 0].numpy(), 644:].any()
    gc, gr = _split(got, row)
    wc, wr = _split(want, row)
    assert np.array_equal(gc, wc)
    if kw.get("rope_cos") is None:
        assert np.array_equal(gr, wr)
    else:
        live = slots >= 0
        s = slots[live].numpy()
        untouched = np.ones(len(got), bool)
        untouched[s] = False
        assert np.array_equal(gr[untouched], wr[untouched])
        scale = np.array([2.0 ** -qc.row_exponent(lc[t], row) for t in np.nonzero(live.numpy())[0]])[:, None]
        ref = lr[live.numpy()] * scale
        length = np.abs(qc.f64(r)[live.numpy()]).max(1, keepdims=True) * 2 * scale
        assert (np.abs(_bf16(gr[s]) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * length).all()
    return dev


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("n", [1, 2, 5, 67, 301])
@pytest.mark.parametrize("norm,rope,interleaved,views", [(True, True, False, True), (True, True, True, False),
                                                         (False, True, False, False), (True, False, False, True),
                                                         (False, False, False, True)])
def test_append(row, n, norm, rope, interleaved, views):
    g = torch.Generator().manual_seed(n + row)
    kv = torch.randn((n, 640), generator=g).to(torch.bfloat16)
    c, r = kv[:, :512], kv[:, 512:576]
    if not views:
        c, r = c.contiguous(), r.contiguous()
    slots = torch.randperm(16 * 24, generator=g)[:n]
    slots[1::5] = -1
    ang = torch.rand((500, 32), generator=g) * 6.28
    kw = dict(norm_weight=1 + 0.1 * torch.randn(512, generator=g)) if norm else {}
    if rope:
        kw.update(rope_cos=ang.cos(), rope_sin=ang.sin(), rope_interleaved=interleaved,
                  positions=torch.randint(0, 500, (n,), generator=g, dtype=torch.int32))
    if views:
        kw_dev = kv.cuda()
        assert not kw_dev[:, :512].is_contiguous() or n == 1
    _append_and_compare(c, r, slots, row, **kw)


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("shift", [-58, -9, 0, 7, 40])
def test_codes_at_borders(row, shift):
    """Without a norm: every midpoint between two codes of both grids, every exponent's border, at many scales."""
    vals = [0.0, -0.0, 448.0, 432.0, 434.0, 447.0, 450.0]
    vals += [(a + b) / 2 for a, b in zip(qc.E4M3[:-1], qc.E4M3[1:])] + list(qc.E4M3)
    vals = np.array([v for v in vals if v <= 448] + [-v for v in vals if v <= 432])
    rng = np.random.default_rng(shift + 60)
    rows = []
    for top in (448.0, 432.0, 446.0, 450.0, 256.0, 3.5):
        for _ in range(3):
            v = rng.choice(vals, 512)
            v[np.abs(v) > top] = 0
            v[rng.integers(512)] = top
            rows.append(v)
    c = torch.from_numpy(np.array(rows) * 2.0 ** shift).to(torch.bfloat16)
    n = len(c)
    r = torch.randn((n, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    _append_and_compare(c, r, torch.randperm(384, generator=torch.Generator().manual_seed(2))[:n], row)


def test_scales_and_codes_of_4_bits_at_borders():
    """Blocks whose largest value is 6 s exactly, or just above it, and values at the midpoints between two codes."""
    rng = np.random.default_rng(3)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1, 1.5, 2, 3, 4, 6, 0])
    rows = []
    for k in range(60):
        v = np.zeros((32, 16))
        for b in range(32):
            s = qc.SCALES[rng.integers(len(qc.SCALES))]
            v[b] = rng.choice(mids, 16) * rng.choice([-1, 1], 16) * s
            v[b, rng.integers(16)] = 6 * s
        v[0, 0] = 432
        rows.append(v.reshape(512))
    c = torch.from_numpy(np.array(rows)).to(torch.bfloat16)
    exact = c.double().numpy() == np.array(rows)
    assert exact.mean() > 0.9  # bf16 holds most of them, so that the borders are met
    _append_and_compare(c, torch.zeros((60, 64), dtype=torch.bfloat16), torch.arange(60), qc.FP4)


@pytest.mark.parametrize("row", FORMATS)
def test_zeros_large_and_small_rows(row):
    g = torch.Generator().manual_seed(row)
    c = torch.randn((9, 512), generator=g)
    c[0] = 0
    c[1] = 0
    c[1, 77] = 2.0 ** -133                       # less than the smallest scale can hold
    for i, e in enumerate((-80, -66, -59, 55, 62, 70, 110)):
        c[2 + i] *= 2.0 ** e                     # above 2^60 codes saturate
    c = c.to(torch.bfloat16)
    _append_and_compare(c, torch.randn((9, 64), generator=g).to(torch.bfloat16), torch.arange(9) * 3, row)
    # zeros stay zeros under a norm, with and without an epsilon
    z = torch.zeros((3, 512), dtype=torch.bfloat16)
    for eps in (0.0, 1e-6):
        cache = torch.full((1, 4, row), 255, dtype=torch.uint8, device="cuda")
        dsa.dsa_mla_quant_append(z.cuda(), z[:, :64].contiguous().cuda(), torch.arange(3).cuda(), cache,
                                 norm_weight=torch.ones(512, device="cuda"), norm_eps=eps)
        _ok()
        back = cache.cpu().numpy()[0]
        for t in range(3):
            v, rr, s = qc.decode_row(back[t])
            assert not v.any() and not rr.any() and s == 1
        assert (back[3] == 255).all()


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("n", [4099, 16390])
def test_the_number_of_tokens_does_not_matter(row, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    c = torch.randn((n, 512), generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn((n, 64), generator=g, device="cuda").to(torch.bfloat16)
    w = 1 + 0.1 * torch.randn(512, generator=g, device="cuda")
    ang = torch.rand((n, 32), generator=g, device="cuda") * 6.28
    kw = dict(norm_weight=w, rope_cos=ang.cos(), rope_sin=ang.sin())
    slots = torch.randperm(n, generator=g, device="cuda")
    caches = [torch.zeros((-(-n // 64), 64, row), dtype=torch.uint8, device="cuda") for _ in range(2)]
    dsa.dsa_mla_quant_append(c, r, slots, caches[0], **kw)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    for i in range(0, n, 1111):
        j = min(n, i + 1111)
        dsa.dsa_mla_quant_append(c[i:j], r[i:j], slots[i:j].contiguous(), caches[1], positions=pos[i:j].contiguous(), **kw)
    _ok()
    assert torch.equal(caches[0], caches[1])
    at = torch.randperm(n, generator=torch.Generator().manual_seed(1))[:40]
    lc, lr = qc.latent(c[at], r[at], norm_weight=w, rope_cos=kw["rope_cos"], rope_sin=kw["rope_sin"], positions=at)
    got = caches[0].view(-1, row)[slots[at.cuda()]].cpu().numpy()
    want = np.array([qc.encode_row(a, b, row) for a, b in zip(lc, lr)])
    assert np.array_equal(_split(got, row)[0], _split(want, row)[0])


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("what", ["slot", "position", "no pages"])
def test_what_is_outside_is_reported_and_skipped(row, what):
    c, r = torch.ones((6, 512), dtype=torch.bfloat16, device="cuda"), torch.ones((6, 64), dtype=torch.bfloat16, device="cuda")
    cache = torch.full((3, 8, row), 7, dtype=torch.uint8, device="cuda")
    slots = torch.tensor([3, -1, 9, 4, -1 << 40, 15], device="cuda")
    kw, left = {}, [4, 9]
    if what == "slot":
        slots[0], slots[5] = 16, 1 << 40
    else:
        table = torch.ones((10, 32), device="cuda")
        kw = dict(rope_cos=table, rope_sin=table, positions=torch.tensor([10, 0, 9, 0, 0, -1], dtype=torch.int32, device="cuda"))
    view = cache[:2] if what != "no pages" else cache[:0]
    if what == "no pages":
        left = []
    dsa.dsa_mla_quant_append(c, r, slots, view, **kw)
    assert dsa.dsa_check_device_status() == dsa.DSA_ERR_DEVICE_CHECK
    touched = (cache.view(-1, row) != 7).any(1).nonzero().flatten().tolist()
    assert touched == left


def _rows(n, row, seed=0):
    rng = np.random.default_rng(seed)
    return np.array([qc.encode_row(rng.standard_normal(512) * 2.0 ** rng.integers(-20, 20), rng.standard_normal(64), row)
                     for _ in range(n)])


@pytest.mark.parametrize("row", FORMATS)
@pytest.mark.parametrize("page,lens,starts,extra", [
    (1, [3, 0, 5, 1], None, 0), (16, [40, 1, 0, 16, 17], [0, 15, 9, 16, 31], 6), (24, [0, 0, 70], [2, 0, 1], 0), (64, [1], None, 0),
    (7, [21, 20, 22], [0, 7, 6], 3), (64, [0, 0], [5, 0], 4)])
def test_read(row, page, lens, starts, extra):
    B, first = len(lens), starts or [0] * len(lens)
    width = max(-(-(s + n) // page) for s, n in zip(first, lens)) + 1
    pages = B * width + 3
    cache = _rows(pages * page, row, seed=page).reshape(pages, page, row)
    bt = np.random.default_rng(1).permutation(pages)[: B * width].reshape(B, width)
    cu = np.concatenate([[0], np.cumsum(lens)])
    total = int(cu[-1]) + extra
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32).cuda()
    out = torch.full((total, 640), 3.0, dtype=torch.bfloat16, device="cuda")
    got = dsa.dsa_mla_quant_read(torch.from_numpy(cache).cuda(), i32(bt), i32(cu), total=total, starts=None if starts is None else i32(first),
                                 c_kv=out[:, :512], k_rope=out[:, 512:576])
    _ok()
    assert got[0].data_ptr() == out.data_ptr()
    res = out.double().cpu().numpy()
    assert (res[:, 576:] == 3).all() and (res[int(cu[-1]):] == 3).all()
    for b in range(B):
        for i in range(lens[b]):
            p = first[b] + i
            c, r, _ = qc.decode_row(cache[bt[b, p // page], p % page])
            assert np.array_equal(res[cu[b] + i, :512], c) and np.array_equal(res[cu[b] + i, 512:576], r)
    if total > 1:  # less room than rows: the rest is dropped
        short = torch.full((total + 1, 512), 3.0, dtype=torch.bfloat16, device="cuda")
        c, r = dsa.dsa_mla_quant_read(torch.from_numpy(cache).cuda(), i32(bt), i32(cu), total=1, starts=None if starts is None else i32(first),
                                      c_kv=short[:1])
        _ok()
        assert (short[1:] == 3).all() and r.shape == (1, 64)


@pytest.mark.parametrize("row", FORMATS)
def test_read_leaves_out_pages_that_are_not_there(row):
    cache = torch.from_numpy(_rows(32, row).reshape(2, 16, row)).cuda()
    bt = torch.tensor([[0, 2, 1], [-1, 1, -5], [1, 0, 0]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 48, 96, 150], dtype=torch.int32, device="cuda")  # the last request passes its table
    c, r = torch.full((150, 512), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((150, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_mla_quant_read(cache, bt, cu, total=150, c_kv=c, k_rope=r)
    assert dsa.dsa_check_device_status() == dsa.DSA_ERR_DEVICE_CHECK
    left = (c == 9).all(1).nonzero().flatten().tolist()
    assert left == list(range(16, 32)) + list(range(48, 64)) + list(range(80, 96)) + list(range(144, 150))
    start = torch.tensor([-1, 0, 0], dtype=torch.int32, device="cuda")
    c.fill_(9)
    dsa.dsa_mla_quant_read(cache, bt, torch.tensor([0, 2, 2, 2], dtype=torch.int32, device="cuda"), total=2, starts=start, c_kv=c[:2])
    assert dsa.dsa_check_device_status() == dsa.DSA_ERR_DEVICE_CHECK
    assert (c[0] == 9).all() and np.array_equal(c[1].double().cpu().numpy(), qc.decode_row(cache[0, 0].cpu().numpy())[0])


@pytest.mark.parametrize("row", FORMATS)
def test_rows_survive_a_second_writing(row):
    """What e4m3 rows stand for is written as itself; a page is moved as bytes."""
    g = torch.Generator(device="cuda").manual_seed(2)
    c, r = torch.randn((200, 512), generator=g, device="cuda").to(torch.bfloat16), torch.randn((200, 64), generator=g, device="cuda").to(torch.bfloat16)
    cache = torch.zeros((8, 32, row), dtype=torch.uint8, device="cuda")
    dsa.dsa_mla_quant_append(c, r, torch.arange(200, device="cuda"), cache)
    bt, cu = torch.arange(8, dtype=torch.int32, device="cuda")[None], torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    c1, r1 = dsa.dsa_mla_quant_read(cache, bt, cu, total=200)
    assert torch.equal(r1, r)
    moved = cache[torch.tensor([3, 1, 0, 2, 7, 6, 5, 4], device="cuda")].contiguous()
    c2, r2 = dsa.dsa_mla_quant_read(moved, torch.tensor([[2, 1, 3, 0, 7, 6, 5, 4]], dtype=torch.int32, device="cuda"), cu, total=200)
    assert torch.equal(c1, c2) and torch.equal(r1, r2)
    if row == qc.FP8:
        again = torch.zeros_like(cache)
        dsa.dsa_mla_quant_append(c1, r1, torch.arange(200, device="cuda"), again)
        c3, _ = dsa.dsa_mla_quant_read(again, bt, cu, total=200)
        assert torch.equal(c1, c3)
    _ok()
