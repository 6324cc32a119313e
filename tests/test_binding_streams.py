"""Where the bindings' memory comes from when a call is given a stream, and that every tensor of
a call lies on the current device, without a GPU.

The tensors are CPU tensors that answer as CUDA ones, the C entry points are stand-ins that
return DSA_OK (workspace sizes come from the real ones), and torch's allocation and stream calls
are watched: what a call allocates must come from the memory of the stream that its kernels run
on, its inputs must be held for that stream, and its results for the caller's current stream.
"""
import ctypes
import types

import pytest
import torch


class Cuda(torch.Tensor):
    """A CPU tensor that answers as one on cuda:0 (or the device set as `index`)."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    index = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index

    def record_stream(self, stream):
        LOG.setdefault(id(self), []).append(stream.name)


LOG = {}
AWAY = {}  # "left": tensors still to be made before the one that lies on cuda:1


def cuda(t):
    t = torch.Tensor._make_subclass(Cuda, t)
    if AWAY:
        t.index = 1 if AWAY["left"] == 0 else 0
        AWAY["left"] -= 1
    return t


class Stream:
    def __init__(self, name, raw):
        self.name, self.cuda_stream, self.device_index = name, raw, 0


@pytest.fixture
def box(monkeypatch):
    """(binding, current stream's name at every allocation, raw streams of the launches)."""
    import __graft_entry__ as g
    g.build()
    import sparse_attention_token_gb300 as dsa
    real, LOG_launch, made = dsa.lib(), [], []
    main, side = Stream("main", 0), Stream("side", 77)
    current = [main]

    class On:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            current.append(self.s)

        def __exit__(self, *exc):
            current.pop()

    class Lib:
        def __getattr__(self, name):
            if name.endswith("workspace_size") or name in ("dsa_status_string", "dsa_topk_width"):
                return getattr(real, name)

            def call(*args):
                raw = args[-1]
                LOG_launch.append((name, getattr(raw, "value", raw)))
                return dsa.DSA_OK
            return call

    def alloc(fn):
        def make(*a, device=None, pin_memory=False, **kw):
            t = fn(*a, **kw)
            if device is not None:
                t = cuda(t)
                made.append((t, current[-1].name))
            return t
        return make

    LOG.clear()
    AWAY.clear()
    fake = Lib()
    monkeypatch.setattr(dsa, "lib", lambda: fake)
    monkeypatch.setattr(torch, "empty", alloc(torch.empty))
    monkeypatch.setattr(torch, "full", alloc(torch.full))
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: current[-1].cuda_stream, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return types.SimpleNamespace(dsa=dsa, made=made, launches=LOG_launch, side=side, main=main)


i32 = lambda *s: cuda(torch.zeros(s, dtype=torch.int32))
i64 = lambda *s: cuda(torch.zeros(s, dtype=torch.int64))
f32 = lambda *s: cuda(torch.zeros(s, dtype=torch.float32))
b16 = lambda *s: cuda(torch.zeros(s, dtype=torch.bfloat16))


def _paged():
    return b16(2, 32, 128), f32(2, 32), b16(4, 64, 128), i32(3), i32(2), i32(2, 2)


CALLS = {
    "dsa_page_plan": lambda d, **kw: d.dsa_page_plan(i32(3), i32(3), i32(3, 4), i32(9), page_size=64, total_q=5, **kw),
    "dsa_mla_cache_append": lambda d, **kw: d.dsa_mla_cache_append(b16(5, 512), b16(5, 64), i64(5), b16(2, 16, 512),
                                                                   b16(2, 16, 64), **kw),
    "dsa_prefix_mla": lambda d, **kw: d.dsa_prefix_mla(b16(3, 16, 512), b16(3, 16, 64), b16(4, 64, 512), b16(4, 64, 64),
                                                       i32(2, 2), i32(3), i32(2), i32(1), prefix_len=60, scale=0.1, **kw),
    "dsa_indexer_scores": lambda d, **kw: d.dsa_indexer_scores(b16(4, 32, 128), b16(8, 128), f32(4, 32), **kw),
    "dsa_indexer_topk": lambda d, **kw: d.dsa_indexer_topk(f32(4, 8), T=4, S=8, q_pos0=4, topk_limit=4, **kw),
    "dsa_indexer": lambda d, **kw: d.dsa_indexer(*_paged(), max_seq_len=128, topk_limit=64, **kw),
    "dsa_indexer_static": lambda d, **kw: d.dsa_indexer_static(*_paged(), max_seq_len=128, topk_limit=64, **kw),
    "dsa_indexer_cache_append": lambda d, **kw: d.dsa_indexer_cache_append(b16(3, 128), i64(3), b16(2, 16, 128), **kw),
    "dsa_indexer_prepare": lambda d, **kw: d.dsa_indexer_prepare(
        b16(2, 256), b16(2, 128), f32(2, 32), f32(2, 32), b16(32 * 128, 128), b16(128, 256), b16(32, 256), f32(128),
        b16(2, 64, 128), i64(2), H=32, rope_dim=64, **kw),
    "dsa_indexer_shard_candidates": lambda d, **kw: d.dsa_indexer_shard_candidates(
        b16(4, 32, 128), b16(8, 128), f32(4, 32), q_pos0=4, key_offset=0, k_cand=4, **kw),
    "dsa_indexer_merge_candidates": lambda d, **kw: d.dsa_indexer_merge_candidates(f32(2, 4, 8), i32(2, 4, 8),
                                                                                  topk_limit=8, **kw),
    "dsa_sparse_mla": lambda d, **kw: d.dsa_sparse_mla(b16(3, 16, 512), b16(3, 16, 64), b16(4, 64, 512), b16(4, 64, 64),
                                                       i32(2, 2), i32(3), i32(2), i32(3, 64), scale=0.1, **kw),
    "dsa_clock_sample": lambda d, **kw: d.dsa_clock_sample(4, **kw),
}
RESULTS = {"dsa_mla_cache_append": 0, "dsa_indexer_cache_append": 0, "dsa_page_plan": 4, "dsa_prefix_mla": 2,
           "dsa_indexer_prepare": 2, "dsa_indexer_shard_candidates": 2}  # tensors a call returns (others 1)


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_a_stream_allocates_there(box, name):
    got = CALLS[name](box.dsa, stream=box.side)
    assert box.launches == [(name, 77)]
    assert [where for _, where in box.made] == ["side"] * len(box.made)
    results = [] if got is None else [t for t in (got if isinstance(got, tuple) else (got,)) if t is not None]
    assert len(results) == RESULTS.get(name, 1)
    for t in results:
        assert "main" in LOG[id(t)]              # the caller may use and drop it on its own stream
    inputs = [names for i, names in LOG.items() if all(i != id(t) for t in results)]
    assert all(names == ["side"] for names in inputs)
    assert inputs or name == "dsa_clock_sample"  # the caller's tensors may be dropped as well


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_the_current_stream_holds_nothing(box, name):
    CALLS[name](box.dsa)
    assert box.launches[0][1] in (0, None) and not LOG
    assert [where for _, where in box.made] == ["main"] * len(box.made)


def test_the_callers_outputs_are_used(box):
    out, lse, ws = b16(3, 16, 512), f32(3, 16), cuda(torch.zeros(1 << 16, dtype=torch.uint8))
    got = CALLS["dsa_prefix_mla"](box.dsa, stream=box.side, out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse and not box.made
    assert LOG[id(ws)] == ["side"] and sorted(LOG[id(out)]) == ["main", "side"]


def test_the_host_pipeline_allocates_its_workspace_there(box):
    h = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    box.dsa.dsa_indexer_dense_host(h(4, 32, 128), h(8, 128), h(4, 32, dtype=torch.float32), topk_limit=4, stream=box.side)
    assert [where for _, where in box.made] == ["side"] and box.launches == [("dsa_indexer_dense_host", 77)]


@pytest.mark.parametrize("name", [n for n in CALLS if n != "dsa_clock_sample"])
def test_tensors_of_another_device_are_refused(box, name):
    CALLS[name](box.dsa)                       # all of them on the current device
    box.launches.clear()
    n = 0
    while True:                                # the n-th tensor that is made lies on the other device
        AWAY["left"] = n
        box.made.clear()
        try:
            CALLS[name](box.dsa)
            refused = False
        except ValueError as e:
            refused = "cuda:1" in str(e) and "current device" in str(e) and not box.launches
        if AWAY["left"] >= 0 or any(t.index for t, _ in box.made):
            break                              # past the caller's tensors
        assert refused, f"tensor {n}"
        n += 1
    assert n >= 1


def test_a_stream_of_another_device_is_refused(box):
    other = Stream("other", 99)
    other.device_index = 1
    for name in CALLS:
        with pytest.raises(ValueError, match="stream"):
            CALLS[name](box.dsa, stream=other)
    assert not box.launches
