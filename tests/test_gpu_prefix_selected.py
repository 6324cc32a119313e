"""The indexer and the sparse attention on the tables, slots and latent rows of a shared-prefix step.

dsa_page_plan makes tables and slots, dsa_mla_cache_append and the indexer's key append write
through them, dsa_indexer selects keys and dsa_sparse_mla attends over them.  Index keys, queries
and weights are small whole numbers, so the selection is exact.  The sparse attention is compared
within its own bound (2^-7 of the row's largest latent, see test_gpu_sparse_mla.py); where every
visible key is selected, dsa_prefix_mla is compared on the same caches within its bound.
"""
import types

import numpy as np
import pytest
import torch

import oracle
from oracle import sparse_mla as smla
from test_gpu_prefix_step import Case, dsa

pytestmark = pytest.mark.gpu

INDEX_HEADS, D = 32, 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("page,H", [(64, 64), (16, 16)])
@pytest.mark.parametrize("fp8", [False, True])
def test_selected_keys_of_planned_steps(page, H, fp8):
    g = torch.Generator().manual_seed(page + fp8)
    whole = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g).float()
    prompt, B, topk = 5 * 64 + 9, 3, 256
    shared = prompt // page
    pages = shared + B * (400 // page + 1) + 4
    order = torch.randperm(pages, generator=g).to(torch.int32).cuda()
    prefix, free = order[:shared].contiguous(), order[shared:].contiguous()
    cc, cr = torch.zeros((pages, page, 512), dtype=torch.bfloat16).cuda(), torch.zeros((pages, page, 64), dtype=torch.bfloat16).cuda()
    ck = torch.zeros((pages, page, D)).to(torch.float8_e4m3fn if fp8 else torch.bfloat16).cuda()
    scales = torch.zeros((pages, page), device="cuda") if fp8 else None
    bt = torch.full((B, (prompt + 400) // page + 1), -1, dtype=torch.int32, device="cuda")

    def append(slots):
        n = slots.shape[0]
        kv = torch.randn((n, 576), generator=g).to(torch.bfloat16).cuda()
        dsa.dsa_mla_cache_append(kv[:, :512], kv[:, 512:], slots, cc, cr, norm_weight=torch.ones(512, device="cuda"))
        keys = whole(-3, 3, n, D)
        keys[:, 0] = 7  # amax 7 = 448 / 64: the e4m3 scale is a power of two and the values stay exact
        dsa.dsa_indexer_cache_append(keys.to(torch.bfloat16).cuda(), slots, ck, scales)

    one = torch.tensor([shared * page], dtype=torch.int32, device="cuda")
    _, slots, _, _ = dsa.dsa_page_plan(one, one, torch.full((1, shared), -1, dtype=torch.int32, device="cuda"), prefix,
                                       page_size=page, total_q=shared * page)
    append(slots)
    lens = torch.full((B,), shared * page, dtype=torch.int32, device="cuda")
    for new in ([60, 9, 100], [1, 1, 1], [2, 0, 3]):
        q_lens = torch.tensor(new, dtype=torch.int32, device="cuda")
        lens = lens + q_lens
        T = sum(new)
        cu, slots, pos, used = dsa.dsa_page_plan(q_lens, lens, bt, free, page_size=page, total_q=T, prefix_pages=prefix)
        free = free[used.item():].contiguous()
        append(slots)
        q = torch.randn((T, H, 576), generator=g).to(torch.bfloat16).cuda()
        qn, qr = q[..., :512].contiguous(), q[..., 512:].contiguous()
        iq, w = whole(-3, 3, T, INDEX_HEADS, D), whole(-2, 2, T, INDEX_HEADS)
        iq = iq.to(torch.float8_e4m3fn if fp8 else torch.bfloat16).cuda()
        q_scale = torch.ones((T, INDEX_HEADS), device="cuda") if fp8 else None
        longest = int(lens.max())
        case = types.SimpleNamespace(q=iq.cpu(), q_scale=None if q_scale is None else q_scale.cpu(), w=w, k_cache=ck.cpu(),
                                     k_scale_cache=None if scales is None else scales.cpu(), cu_q_lens=cu.cpu(),
                                     seq_lens=lens.cpu(), block_tables=bt.cpu())
        scale = 576 ** -0.5
        for limit in (topk, longest):  # some of the keys, all of them
            sel = dsa.dsa_indexer(iq, w.cuda(), ck, cu, lens, bt, max_seq_len=longest, topk_limit=limit, q_scale=q_scale,
                                  k_scale_cache=scales)
            out = dsa.dsa_sparse_mla(qn, qr, cc, cr, bt, cu, lens, sel, scale=scale)
            assert dsa.dsa_check_device_status() == dsa.DSA_OK
            ref_sel, _, _ = oracle.paged(case, topk_limit=limit, k_out=limit)
            assert np.array_equal(sel.cpu().numpy(), ref_sel)
            ref = smla.sparse_mla(qn, qr, cc, cr, bt, cu, sel, page_size=page, scale=scale)
            assert np.all(np.abs(out.double().cpu().numpy() - ref) <= 2.0 ** -7 * cc.abs().max().item() + 1e-6)
        c = Case.__new__(Case)
        c.prefix, c.scale, c.page = shared * page, scale, page
        c.qn, c.qr, c.cc, c.cr, c.bt, c.cu, c.lens, c.pp = (t.cpu() for t in (qn, qr, cc, cr, bt, cu, lens, prefix))
        dense = dsa.dsa_prefix_mla(qn, qr, cc, cr, bt, cu, lens, prefix, prefix_len=shared * page, scale=scale)
        c.check(dense)
        # every key selected: the same attention, each within its bound of it
        got = out.double().cpu().numpy()
        exact = c.oracle()["out"]
        assert np.all(np.abs(got - exact) <= 2.0 ** -7 * cc.abs().max().item() + 1e-6)
    assert dsa.dsa_check_device_status() == dsa.DSA_OK
