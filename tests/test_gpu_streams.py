"""Calls on a stream of their own while the current stream still has work queued: what they
allocate must not be memory that this work writes later."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("sparse_attention_token_gb300")

SLEEP = 200_000_000  # cycles: some 0.1 s, far longer than the calls below take


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def _queued_garbage(sizes):
    """Behind a long kernel on the current stream, fills of temporaries of these sizes (bytes),
    whose memory the allocator may hand out again at once."""
    torch.cuda._sleep(SLEEP)
    held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    for t in held:
        t.fill_(255)


def _step(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(q=rnd(5, 16, 576), cc=rnd(40, 64, 512), cr=rnd(40, 64, 64), q_lens=torch.tensor([1, 3, 1], **i32),
                lens=torch.tensor([700, 515, 640], **i32), prefix=torch.arange(8, **i32),
                free=torch.arange(20, 40, **i32),
                bt=torch.tensor([[-1] * 8 + [8, 9, 10, -1], [-1] * 8 + [11, -1, -1, -1], [-1] * 8 + [13, 14, -1, -1]], **i32))


def _plan(s, **kw):
    bt = s["bt"].clone() if "bt" not in kw else kw.pop("bt")
    return dsa.dsa_page_plan(s["q_lens"], s["lens"], bt, s["free"], page_size=64, total_q=5, prefix_pages=s["prefix"],
                             **kw)


def _attend(s, cu, bt, **kw):
    return dsa.dsa_prefix_mla(s["q"][..., :512], s["q"][..., 512:], s["cc"], s["cr"], bt, cu, s["lens"], s["prefix"],
                              prefix_len=512, scale=576 ** -0.5, **kw)


def test_a_planned_step_on_a_side_stream():
    s, side = _step(1), torch.cuda.Stream()
    bt = s["bt"].clone()
    ref = _plan(s, bt=bt)
    ref_out = _attend(s, ref[0], bt)
    need = dsa.dsa_prefix_mla_workspace_size(3, 5, 16, prefix_len=512)
    tables = s["bt"].clone()
    torch.cuda.synchronize()
    _queued_garbage([16, 20, 40, 4, 5 * 16 * 512 * 2, 5 * 16 * 4, need])
    got = _plan(s, bt=tables, stream=side)
    got_out = _attend(s, got[0], tables, stream=side)
    side.synchronize()
    early = [t.clone() for t in got + got_out]  # queued behind the fills as well
    torch.cuda.synchronize()
    assert dsa.dsa_check_device_status() == dsa.DSA_OK
    for a, b, c in zip(ref + ref_out, got + got_out, early):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_scores_and_top_k_on_a_side_stream():
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    q, k, w = rnd(64, 32, 128).to(torch.bfloat16), rnd(900, 128).to(torch.bfloat16), rnd(64, 32)
    ref = dsa.dsa_indexer_scores(q, k, w)
    top = dsa.dsa_indexer_topk(ref, T=64, S=900, q_pos0=836, topk_limit=256)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _queued_garbage([64 * 900 * 4, 64 * 256 * 4])
    got = dsa.dsa_indexer_scores(q, k, w, stream=side)
    got_top = dsa.dsa_indexer_topk(got, T=64, S=900, q_pos0=836, topk_limit=256, stream=side)
    torch.cuda.synchronize()
    assert dsa.dsa_check_device_status() == dsa.DSA_OK
    assert torch.equal(ref, got) and torch.equal(top, got_top)


def test_a_side_stream_inside_a_captured_graph():
    s, side = _step(3), torch.cuda.Stream()
    bt = s["bt"].clone()
    ref = _plan(s, bt=bt)
    ref_out = _attend(s, ref[0], bt)
    tables = s["bt"].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = _plan(s, bt=tables, stream=side)
        got_out = _attend(s, got[0], tables, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        doubled = got_out[1] * 2  # reads the result on the capturing stream
    for _ in range(3):
        for t in got + got_out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert dsa.dsa_check_device_status() == dsa.DSA_OK
        for a, b in zip(ref + ref_out, got + got_out):
            assert torch.equal(a, b)
        assert torch.equal(doubled, ref_out[1] * 2)
