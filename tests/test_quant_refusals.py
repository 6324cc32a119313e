"""The quantised latent cache without a GPU: refusals of its entry points, workspace sizes, streams and devices."""
import ctypes

import pytest
import torch

from test_binding_streams import AWAY, LOG, box, cuda, f32, i32, i64, b16  # noqa: F401 (box is a fixture)

FAKE = 1 << 20  # never dereferenced: every call here fails (or has nothing to do) before a launch
u8 = lambda *s: cuda(torch.zeros(s, dtype=torch.uint8))


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__ as g
    g.build()
    import sparse_attention_token_gb300 as m
    return m


def _call(dsa, entry, defaults, kw, *more):
    args = getattr(dsa, entry + "_args")()
    for k, v in {**defaults, **kw}.items():
        setattr(args, k, v)
    return getattr(dsa.lib(), entry)(ctypes.byref(args), None)


APPEND = dict(format=1, n=4, kv_rank=512, rope_dim=64, page_size=64, num_pages=8, rope_interleaved=0, rope_rows=100,
              norm_eps=1e-6, c_kv=FAKE, k_rope=FAKE, c_stride=576, r_stride=576, slot_mapping=FAKE, norm_weight=FAKE,
              rope_cos=FAKE, rope_sin=FAKE, positions=FAKE, cache=FAKE)
READ = dict(format=2, B=3, total=40, kv_rank=512, rope_dim=64, page_size=64, num_pages=8, max_pages_per_seq=4, cache=FAKE,
            block_tables=FAKE, cu_lens=FAKE, starts=FAKE, c_kv=FAKE, k_rope=FAKE, c_stride=512, r_stride=64)
MLA = dict(format=1, B=3, total_q=5, H=20, kv_rank=512, rope_dim=64, page_size=64, num_pages=8, max_pages_per_seq=4,
           topk_width=100, scale=0.1, q_nope=FAKE, q_rope=FAKE, qn_stride_t=20 * 576, qn_stride_h=576, qr_stride_t=20 * 64,
           qr_stride_h=64, cache=FAKE, block_tables=FAKE, cu_q_lens=FAKE, seq_lens=FAKE, topk=FAKE, out=FAKE, lse=FAKE,
           workspace=FAKE, workspace_bytes=1 << 40)


@pytest.mark.parametrize("bad", [dict(n=-1), dict(page_size=0), dict(num_pages=-1), dict(kv_rank=0), dict(rope_dim=-1),
                                 dict(c_kv=None), dict(k_rope=None), dict(slot_mapping=None), dict(cache=None),
                                 dict(rope_cos=None), dict(rope_sin=None), dict(rope_rows=0),
                                 dict(positions=None, rope_rows=3), dict(norm_eps=-1e-6), dict(norm_eps=float("nan")),
                                 dict(c_stride=577), dict(r_stride=68), dict(c_stride=-576), dict(c_kv=FAKE + 8),
                                 dict(k_rope=FAKE + 8), dict(cache=FAKE + 8), dict(slot_mapping=FAKE + 4),
                                 dict(norm_weight=FAKE + 4), dict(rope_cos=FAKE + 4), dict(rope_sin=FAKE + 8),
                                 dict(positions=FAKE + 2)], ids=str)
def test_append_refuses(dsa, bad):
    assert _call(dsa, "dsa_mla_quant_append", APPEND, bad) == dsa.DSA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("bad", [dict(B=-1), dict(total=-1), dict(page_size=0), dict(num_pages=-1), dict(max_pages_per_seq=-1),
                                 dict(kv_rank=0), dict(cache=None), dict(cu_lens=None), dict(c_kv=None), dict(k_rope=None),
                                 dict(block_tables=None), dict(c_stride=516), dict(r_stride=-64), dict(cache=FAKE + 4),
                                 dict(c_kv=FAKE + 2), dict(k_rope=FAKE + 8), dict(block_tables=FAKE + 2),
                                 dict(cu_lens=FAKE + 1), dict(starts=FAKE + 2)], ids=str)
def test_read_refuses(dsa, bad):
    assert _call(dsa, "dsa_mla_quant_read", READ, bad) == dsa.DSA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("bad", [dict(B=-1), dict(total_q=-1), dict(H=0), dict(topk_width=-1), dict(page_size=0),
                                 dict(num_pages=-1), dict(max_pages_per_seq=-1), dict(scale=0.0), dict(scale=-1.0),
                                 dict(scale=float("nan")), dict(q_nope=None), dict(q_rope=None), dict(cache=None),
                                 dict(block_tables=None), dict(cu_q_lens=None), dict(seq_lens=None), dict(topk=None),
                                 dict(out=None), dict(qn_stride_t=20 * 576 + 1), dict(qn_stride_h=580), dict(qr_stride_t=4),
                                 dict(qr_stride_h=-64), dict(q_nope=FAKE + 8), dict(q_rope=FAKE + 2), dict(cache=FAKE + 8),
                                 dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(block_tables=FAKE + 2), dict(cu_q_lens=FAKE + 2),
                                 dict(seq_lens=FAKE + 1), dict(topk=FAKE + 2)], ids=str)
def test_attention_refuses(dsa, bad):
    assert _call(dsa, "dsa_quant_mla", MLA, bad) == dsa.DSA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("entry,base", [("dsa_mla_quant_append", APPEND), ("dsa_mla_quant_read", READ), ("dsa_quant_mla", MLA)])
def test_what_there_is_no_kernel_for(dsa, entry, base):
    for bad in (dict(format=0), dict(format=3), dict(format=-1), dict(kv_rank=256), dict(rope_dim=32)):
        assert _call(dsa, entry, base, bad) == dsa.DSA_ERR_UNSUPPORTED
    if entry == "dsa_quant_mla":
        for bad in (dict(H=129), dict(total_q=1 << 25, H=128), dict(num_pages=1 << 25, page_size=64)):
            assert _call(dsa, entry, base, bad) == dsa.DSA_ERR_UNSUPPORTED
    assert getattr(dsa.lib(), entry)(None, None) == dsa.DSA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("entry,base,nothing", [
    ("dsa_mla_quant_append", APPEND, dict(n=0, c_kv=None, cache=None)), ("dsa_mla_quant_read", READ, dict(total=0, cache=None)),
    ("dsa_mla_quant_read", READ, dict(B=0, cache=None)), ("dsa_quant_mla", MLA, dict(total_q=0, q_nope=None, workspace=None))])
def test_nothing_to_do(dsa, entry, base, nothing):
    assert _call(dsa, entry, base, nothing) == dsa.DSA_OK


def _size(dsa, **kw):
    args, n = dsa.dsa_quant_mla_args(), ctypes.c_size_t(0)
    for k, v in {**MLA, **kw}.items():
        setattr(args, k, v)
    assert dsa.lib().dsa_quant_mla_workspace_size(ctypes.byref(args), ctypes.byref(n)) == dsa.DSA_OK
    return n.value


@pytest.mark.parametrize("kw", [dict(topk_width=0, topk=None), dict(topk_width=0, topk=None, total_q=900), dict(total_q=151, H=64, topk_width=1000),
                                dict(total_q=160, H=64, topk_width=1000), dict(topk_width=64)])
def test_workspace(dsa, kw):
    need = _size(dsa, **kw)
    t, h = kw.get("total_q", 5), kw.get("H", 20)
    assert dsa.dsa_quant_mla_workspace_size(t, h, k=kw.get("topk_width", 100)) == need
    if need == 0:  # tiles that are not cut, or whose pieces stay in a cluster
        assert kw["topk_width"] > 0
        return
    for bad in (dict(workspace_bytes=need - 1), dict(workspace=None), dict(workspace=FAKE + 8)):
        assert _call(dsa, "dsa_quant_mla", MLA, {**kw, "workspace_bytes": need, **bad}) == dsa.DSA_ERR_WORKSPACE
    # two pieces of 64 x 512 fp32 and their sums for each SM, and 8 bytes a query: not by the cache or the keys
    assert need <= 160 * 2 * 64 * 514 * 4 + 160 * 8 + 8 * (t + 1)
    n = ctypes.c_size_t(0)
    assert dsa.lib().dsa_quant_mla_workspace_size(None, ctypes.byref(n)) == dsa.DSA_ERR_INVALID_ARGUMENT
    assert dsa.lib().dsa_quant_mla_workspace_size(ctypes.byref(dsa.dsa_quant_mla_args()), None) == dsa.DSA_ERR_INVALID_ARGUMENT
    with pytest.raises(dsa.DsaError):
        dsa.dsa_quant_mla_workspace_size(3, 129)


def test_strides_of_dimensions_of_size_one_do_not_count(dsa):
    call = lambda **kw: _call(dsa, "dsa_quant_mla", MLA, dict(workspace_bytes=0, topk_width=0, **kw))
    odd = dict(qn_stride_t=577, qr_stride_t=-3)
    assert call(total_q=1, **odd) == dsa.DSA_ERR_WORKSPACE and call(**odd) == dsa.DSA_ERR_INVALID_ARGUMENT
    odd = dict(qn_stride_h=577, qr_stride_h=65)
    assert call(H=1, **odd) == dsa.DSA_ERR_WORKSPACE and call(**odd) == dsa.DSA_ERR_INVALID_ARGUMENT


def test_row_bytes(dsa):
    assert (dsa.dsa_mla_quant_row_bytes(dsa.DSA_FP8_E4M3), dsa.dsa_mla_quant_row_bytes(dsa.DSA_FP4_E2M1)) == (656, 416)
    for other in (dsa.DSA_BF16, 3, -1):
        with pytest.raises(ValueError, match="format"):
            dsa.dsa_mla_quant_row_bytes(other)


CALLS = {
    "dsa_mla_quant_append": lambda d, **kw: d.dsa_mla_quant_append(b16(5, 512), b16(5, 64), i64(5), u8(2, 16, 656), **kw),
    "dsa_mla_quant_read": lambda d, **kw: d.dsa_mla_quant_read(u8(4, 64, 416), i32(2, 2), i32(3), total=7, **kw),
    "dsa_quant_mla": lambda d, **kw: d.dsa_quant_mla(b16(3, 16, 512), b16(3, 16, 64), u8(4, 64, 656), i32(2, 2), i32(3), i32(2),
                                                     i32(3, 64), scale=0.1, **kw),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_a_stream(box, name):  # noqa: F811
    got = CALLS[name](box.dsa, stream=box.side)
    assert box.launches == [(name, 77)] and {where for _, where in box.made} <= {"side"}
    results = [] if got is None else list(got)
    assert len(results) == (0 if name == "dsa_mla_quant_append" else 2)
    assert all("main" in LOG[id(t)] for t in results)
    inputs = [names for i, names in LOG.items() if all(i != id(t) for t in results)]
    assert inputs and all(names == ["side"] for names in inputs)


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_the_current_stream_holds_nothing(box, name):  # noqa: F811
    CALLS[name](box.dsa)
    assert box.launches[0][1] in (0, None) and not LOG and {where for _, where in box.made} <= {"main"}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_are_refused(box, name):  # noqa: F811
    n = 0
    while True:
        AWAY["left"] = n
        box.made.clear()
        try:
            CALLS[name](box.dsa)
            refused = False
        except ValueError as e:
            refused = "cuda:1" in str(e) and "current device" in str(e) and not box.launches
        if AWAY["left"] >= 0 or any(t.index for t, _ in box.made):
            break
        assert refused, f"tensor {n}"
        n += 1
    assert n >= 3


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(box, name):  # noqa: F811
    other = type(box.side)("other", 99)
    other.device_index = 1
    with pytest.raises(ValueError, match="stream"):
        CALLS[name](box.dsa, stream=other)
    assert not box.launches


def _bad(d, **kw):
    a = dict(q_nope=b16(3, 16, 512), q_rope=b16(3, 16, 64), cache=u8(4, 64, 656), block_tables=i32(2, 2), cu_q_lens=i32(3),
             seq_lens=i32(2), topk=i32(3, 64), scale=0.1)
    a.update(kw)
    return d.dsa_quant_mla(**a)


def test_shapes_and_types(box):  # noqa: F811
    d = box.dsa
    for kw in (dict(q_rope=b16(3, 15, 64)), dict(q_nope=b16(3, 512)), dict(cache=u8(4, 64, 576)), dict(cache=u8(4, 656)),
               dict(cache=b16(4, 64, 656)), dict(block_tables=i32(3, 2)), dict(cu_q_lens=i32(2)), dict(topk=i32(2, 64)),
               dict(topk=i32(3)), dict(topk=i32(3, 0)), dict(topk=i64(3, 64)), dict(seq_lens=i64(2)), dict(q_nope=f32(3, 16, 512)),
               dict(out=b16(3, 16, 500)), dict(lse=f32(3, 15)), dict(cache=u8(4, 64, 700)[:, :, :656])):
        with pytest.raises((ValueError, TypeError)):
            _bad(d, **kw)
    for kw in (dict(slot_mapping=i32(5)), dict(k_rope=b16(4, 64)), dict(cache=u8(2, 16, 576)), dict(norm_weight=f32(64)),
               dict(rope_cos=f32(9, 32)), dict(rope_cos=f32(9, 32), rope_sin=f32(8, 32)), dict(positions=i32(4)),
               dict(cache=u8(2, 16, 672)[:, :, :656])):
        a = dict(c_kv=b16(5, 512), k_rope=b16(5, 64), slot_mapping=i64(5), cache=u8(2, 16, 656))
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            d.dsa_mla_quant_append(**a)
    for kw in (dict(cu_lens=i32(2)), dict(starts=i32(3)), dict(c_kv=b16(6, 512)), dict(k_rope=b16(7, 32)), dict(block_tables=i32(2)),
               dict(c_kv=f32(7, 512)), dict(cache=u8(4, 64, 415))):
        a = dict(cache=u8(4, 64, 416), block_tables=i32(2, 2), cu_lens=i32(3), total=7)
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            d.dsa_mla_quant_read(**a)
    assert not box.launches
