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
