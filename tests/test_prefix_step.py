"""The shared-prefix step without a GPU: refusals of its entry points, and pins of its oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import prefix_step

FAKE = 1 << 20  # never dereferenced: every call here fails (or has nothing to do) before a launch


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__ as g
    g.build()
    import sparse_attention_token_gb300 as m
    return m


def _fill(args, **kw):
    for k, v in kw.items():
        setattr(args, k, v)
    return args


# ---------------------------------------------------------------- refusals

def _plan(dsa, **kw):
    a = dict(B=4, total_q=8, page_size=64, max_pages_per_seq=16, num_prefix_pages=2, num_free=10, q_lens=FAKE,
             seq_lens=FAKE, prefix_pages=FAKE, free_pages=FAKE, block_tables=FAKE, cu_q_lens=FAKE, slot_mapping=FAKE,
             positions=FAKE, used=FAKE)
    a.update(kw)
    return dsa.lib().dsa_page_plan(ctypes.byref(_fill(dsa.dsa_page_plan_args(), **a)), None)


@pytest.mark.parametrize("bad", [dict(B=-1), dict(total_q=-1), dict(page_size=0), dict(max_pages_per_seq=-1),
                                 dict(num_prefix_pages=-1), dict(num_prefix_pages=17), dict(num_free=-1),
                                 dict(q_lens=None), dict(seq_lens=None), dict(prefix_pages=None),
                                 dict(free_pages=None), dict(block_tables=None), dict(cu_q_lens=None),
                                 dict(slot_mapping=None), dict(positions=None), dict(used=None),
                                 dict(slot_mapping=FAKE + 4), dict(q_lens=FAKE + 2), dict(block_tables=FAKE + 1)])
def test_page_plan_refuses(dsa, bad):
    assert _plan(dsa, **bad) == dsa.DSA_ERR_INVALID_ARGUMENT


def test_page_plan_refuses_null(dsa):
    assert dsa.lib().dsa_page_plan(None, None) == dsa.DSA_ERR_INVALID_ARGUMENT


def _append(dsa, **kw):
    a = dict(n=4, kv_rank=512, rope_dim=64, page_size=64, num_pages=8, rope_interleaved=0, rope_rows=100,
             norm_eps=1e-6, c_kv=FAKE, k_rope=FAKE, c_stride=576, r_stride=576, slot_mapping=FAKE, norm_weight=FAKE,
             rope_cos=FAKE, rope_sin=FAKE, positions=FAKE, cache_c=FAKE, cache_r=FAKE)
    a.update(kw)
    return dsa.lib().dsa_mla_cache_append(ctypes.byref(_fill(dsa.dsa_mla_cache_append_args(), **a)), None)


@pytest.mark.parametrize("bad", [dict(n=-1), dict(page_size=0), dict(num_pages=-1), dict(kv_rank=0), dict(c_kv=None),
                                 dict(k_rope=None), dict(slot_mapping=None), dict(cache_c=None), dict(cache_r=None),
                                 dict(rope_cos=None), dict(rope_sin=None), dict(rope_rows=0),
                                 dict(positions=None, rope_rows=3), dict(norm_eps=-1.0), dict(norm_eps=math.nan),
                                 dict(c_stride=577), dict(r_stride=-8), dict(c_kv=FAKE + 2), dict(cache_r=FAKE + 8),
                                 dict(slot_mapping=FAKE + 4), dict(norm_weight=FAKE + 4)])
def test_latent_append_refuses(dsa, bad):
    assert _append(dsa, **bad) == dsa.DSA_ERR_INVALID_ARGUMENT


def test_latent_append_other_widths_and_nothing_to_do(dsa):
    assert _append(dsa, kv_rank=256) == dsa.DSA_ERR_UNSUPPORTED
    assert _append(dsa, rope_dim=32) == dsa.DSA_ERR_UNSUPPORTED
    assert _append(dsa, n=0) == dsa.DSA_OK


def _attend_args(dsa, **kw):
    a = dict(B=2, total_q=4, H=64, kv_rank=512, rope_dim=64, page_size=64, num_pages=100, max_pages_per_seq=10,
             prefix_len=100, num_prefix_pages=2, scale=0.05, q_nope=FAKE, q_rope=FAKE, qn_stride_t=64 * 512,
             qn_stride_h=512, qr_stride_t=64 * 64, qr_stride_h=64, cache_c=FAKE, cache_r=FAKE, prefix_pages=FAKE,
             block_tables=FAKE, cu_q_lens=FAKE, seq_lens=FAKE, out=FAKE, lse=FAKE, workspace=FAKE,
             workspace_bytes=1 << 40)
    a.update(kw)
    return _fill(dsa.dsa_prefix_mla_args(), **a)


@pytest.mark.parametrize("bad", [dict(B=-1), dict(B=0), dict(total_q=-1), dict(H=0), dict(page_size=0),
                                 dict(num_pages=-1), dict(prefix_len=-1), dict(prefix_len=129), dict(scale=0.0),
                                 dict(scale=math.nan), dict(scale=math.inf), dict(q_nope=None), dict(q_rope=None),
                                 dict(cache_c=None), dict(cache_r=None), dict(prefix_pages=None),
                                 dict(block_tables=None), dict(cu_q_lens=None), dict(seq_lens=None), dict(out=None),
                                 dict(qn_stride_h=516), dict(qr_stride_t=4), dict(q_nope=FAKE + 8),
                                 dict(cache_c=FAKE + 2), dict(out=FAKE + 4), dict(lse=FAKE + 2)])
def test_prefix_mla_refuses(dsa, bad):
    a = _attend_args(dsa, **bad)
    assert dsa.lib().dsa_prefix_mla(ctypes.byref(a), None) == dsa.DSA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("bad", [dict(kv_rank=256), dict(rope_dim=32), dict(H=129), dict(page_size=48, num_prefix_pages=3),
                                 dict(page_size=256)])
def test_prefix_mla_unsupported(dsa, bad):
    a = _attend_args(dsa, **bad)
    assert dsa.lib().dsa_prefix_mla(ctypes.byref(a), None) == dsa.DSA_ERR_UNSUPPORTED


def test_prefix_mla_no_queries(dsa):
    a = _attend_args(dsa, total_q=0)
    assert dsa.lib().dsa_prefix_mla(ctypes.byref(a), None) == dsa.DSA_OK
    n = ctypes.c_size_t(0)
    assert dsa.lib().dsa_prefix_mla_workspace_size(ctypes.byref(a), None) == dsa.DSA_ERR_INVALID_ARGUMENT
    assert dsa.lib().dsa_prefix_mla_workspace_size(ctypes.byref(a), ctypes.byref(n)) == dsa.DSA_OK


def test_bindings_check_shapes_and_devices(dsa):
    i32, bf = torch.int32, torch.bfloat16
    q, s, bt, free = torch.ones(3, dtype=i32), torch.ones(3, dtype=i32), torch.zeros((3, 4), dtype=i32), torch.zeros(9, dtype=i32)
    with pytest.raises(ValueError, match="seq_lens must have shape"):
        dsa.dsa_page_plan(q, s[:2], bt, free, page_size=64, total_q=3)
    with pytest.raises(ValueError, match="block_tables must have shape"):
        dsa.dsa_page_plan(q, s, bt[:2], free, page_size=64, total_q=3)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_page_plan(q, s, bt, free, page_size=64, total_q=3)
    kv = torch.zeros((5, 576), dtype=bf)
    cc, cr = torch.zeros((2, 16, 512), dtype=bf), torch.zeros((2, 16, 64), dtype=bf)
    slots = torch.zeros(5, dtype=torch.int64)
    with pytest.raises(ValueError, match="slot_mapping must have shape"):
        dsa.dsa_mla_cache_append(kv[:, :512], kv[:, 512:], slots[:4], cc, cr)
    with pytest.raises(ValueError, match="go together"):
        dsa.dsa_mla_cache_append(kv[:, :512], kv[:, 512:], slots, cc, cr, rope_cos=torch.zeros((5, 32)))
    with pytest.raises(ValueError, match="cache_r must have shape"):
        dsa.dsa_mla_cache_append(kv[:, :512], kv[:, 512:], slots, cc, cr[:1])
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_mla_cache_append(kv[:, :512], kv[:, 512:], slots, cc, cr)
    qq = torch.zeros((3, 16, 576), dtype=bf)
    cu = torch.zeros(4, dtype=i32)
    with pytest.raises(ValueError, match="cu_q_lens must have shape"):
        dsa.dsa_prefix_mla(qq[..., :512], qq[..., 512:], cc, cr, bt, cu[:3], s, prefix_len=0, scale=0.1)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_prefix_mla(qq[..., :512], qq[..., 512:], cc, cr, bt, cu, s, prefix_len=0, scale=0.1)


# ---------------------------------------------------------------- oracle pins

def test_oracle_page_plan_hand_worked():
    # pages of 4; prefix pages [7, 8]; request 0: 9 tokens cached (pages 7, 8, 3), 4 new -> fills
    # page 3 and takes page 20; request 1: new, 3 tokens after the prefix -> takes 21;
    # request 2: idle; request 3: no new token; request 4: 8 new tokens right on a border
    bt = [[-9, -9, 3, -9, -9], [-9] * 5, [5] * 5, [-9, -9, 6, -9, -9], [-9] * 5]
    table, cu, slots, pos, used = prefix_step.page_plan(
        [4, 3, 0, 0, 8], [13, 11, 0, 12, 16], bt, [20, 21, 22, 23, 24], page_size=4, total_q=17, prefix_pages=[7, 8])
    assert table == [[7, 8, 3, 20, -1], [7, 8, 21, -1, -1], [-1] * 5, [7, 8, 6, -1, -1], [7, 8, 22, 23, -1]]
    assert cu == [0, 4, 7, 7, 7, 15] and used == 4
    assert pos == [9, 10, 11, 12, 8, 9, 10, 8, 9, 10, 11, 12, 13, 14, 15, -1, -1]
    assert slots == [13, 14, 15, 80, 84, 85, 86, 88, 89, 90, 91, 92, 93, 94, 95, -1, -1]


def test_oracle_latent_append_hand_worked():
    c = torch.tensor([[3.0, 4.0]])
    r = torch.tensor([[1.0, 2.0, 3.0, 4.0]])
    cc, cr = torch.zeros((1, 2, 2)), torch.zeros((1, 2, 4))
    cos, sin = torch.tensor([[0.0, 1.0]]), torch.tensor([[1.0, 0.0]])
    kw = dict(norm_weight=torch.tensor([1.0, 2.0]), norm_eps=0.0, rope_cos=cos, rope_sin=sin)
    a, b = prefix_step.latent_append(c, r, torch.tensor([1]), cc, cr, **kw)
    rms = math.sqrt(12.5)
    assert np.allclose(a[0, 1], [3 / rms, 8 / rms]) and np.all(a[0, 0] == 0)
    assert np.allclose(b[0, 1], [-3, 2, 1, 4])                  # pair (1, 3) by 90 degrees, (2, 4) by none
    _, b = prefix_step.latent_append(c, r, torch.tensor([0]), cc, cr, rope_interleaved=True, **kw)
    assert np.allclose(b[0, 0], [-2, 1, 3, 4])                  # pair (1, 2) by 90 degrees, (3, 4) by none


def test_oracle_prefix_mla_equals_dense_attention():
    g = torch.Generator().manual_seed(3)
    H, R, P, page, prefix = 3, 8, 4, 4, 6
    lens, qs = [9, 7], [2, 1]
    cc, cr = torch.randn((9, page, R), generator=g), torch.randn((9, page, P), generator=g)
    qn, qr = torch.randn((3, H, R), generator=g), torch.randn((3, H, P), generator=g)
    pp = torch.tensor([4, 2])
    bt = torch.tensor([[4, 7, 1], [4, 5, -1]])
    got = prefix_step.prefix_mla(qn, qr, cc, cr, bt, torch.tensor([0, 2, 3]), torch.tensor(lens), pp,
                                 prefix_len=prefix, scale=0.3)
    # the sequences written out: positions 0..5 from pages 4 and 2, the rest from the own table
    for b, t0 in ((0, 0), (1, 2)):
        where = [(4, 0), (4, 1), (4, 2), (4, 3), (2, 0), (2, 1)]
        own = int(bt[b, 1])
        where += [(own, 2), (own, 3)] + ([(1, 0)] if b == 0 else [])
        where = where[: lens[b]]
        k = torch.stack([torch.cat([cc[p, i], cr[p, i]]) for p, i in where]).double()
        q = torch.cat([qn, qr], 2)[t0: t0 + qs[b]].double()
        mask = torch.ones((qs[b], lens[b]), dtype=torch.bool).tril(lens[b] - qs[b])
        ref = torch.nn.functional.scaled_dot_product_attention(
            q.transpose(0, 1), k.expand(H, -1, -1), k[:, :R].expand(H, -1, -1), attn_mask=mask, scale=0.3)
        assert np.allclose(got["out"][t0: t0 + qs[b]], ref.transpose(0, 1).numpy(), atol=1e-12)
        x = (q @ k.T * 0.3).masked_fill(~mask[:, None, :], -math.inf)
        assert np.allclose(got["lse"][t0: t0 + qs[b]], torch.logsumexp(x, 2).numpy(), atol=1e-12)


def test_oracle_prefix_mla_sees_nothing():
    cc, cr = torch.ones((2, 4, 8)), torch.ones((2, 4, 4))
    got = prefix_step.prefix_mla(torch.ones((2, 1, 8)), torch.ones((2, 1, 4)), cc, cr, torch.zeros((1, 1), dtype=torch.int64),
                                 torch.tensor([0, 1]), torch.tensor([0]), torch.tensor([0]), prefix_len=2, scale=1.0)
    assert np.all(got["out"] == 0) and np.all(np.isneginf(got["lse"]))
