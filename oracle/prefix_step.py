"""CPU oracle of the shared-prefix serving step -- TEST INFRASTRUCTURE ONLY (Python integers, numpy fp64).

page_plan      block tables, slots, positions and offsets by walking the requests one by one
latent_append  c / sqrt(mean(c^2) + eps) * weight and RoPE rows into copies of the cache
prefix_mla     softmax attention of every (query, head) row over the positions it sees, each
               read from the page that the prefix or the request's own table names; also the
               sums that error bounds are made of
"""
from __future__ import annotations

import numpy as np
import torch


def _f64(t) -> np.ndarray:
    return t.detach().to(torch.float64).cpu().numpy()


def page_plan(q_lens, seq_lens, block_tables, free_pages, *, page_size, total_q, prefix_pages=()):
    """(block_tables, cu_q_lens, slot_mapping, positions, used) as lists; -1 where there is none."""
    table = [list(map(int, row)) for row in block_tables]
    prefix, free = [int(p) for p in prefix_pages], [int(p) for p in free_pages]
    cu, slots, positions, used = [0], [], [], 0
    for b, (q, n) in enumerate(zip(map(int, q_lens), map(int, seq_lens))):
        if n == 0:
            table[b] = [-1] * len(table[b])
        else:
            pages = list(prefix)
            held = -(-(n - q) // page_size)
            pages += table[b][len(prefix):held]
            while len(pages) * page_size < n:
                pages.append(free[used] if used < len(free) else -1)
                used += 1
            table[b] = pages + [-1] * (len(table[b]) - len(pages))
        for p in range(n - q, n):
            positions.append(p)
            page = table[b][p // page_size]
            slots.append(page * page_size + p % page_size if page >= 0 else -1)
        cu.append(cu[-1] + q)
    pad = [-1] * (total_q - len(slots))
    return table, cu, slots + pad, positions + pad, used


def latent_append(c_kv, k_rope, slot_mapping, cache_c, cache_r, *, norm_weight=None, norm_eps=1e-6, rope_cos=None,
                  rope_sin=None, positions=None, rope_interleaved=False):
    """(cache_c, cache_r) after the append, in fp64 (written rows unrounded)."""
    c, r = _f64(c_kv), _f64(k_rope)
    cc, cr = _f64(cache_c), _f64(cache_r)
    flat_c, flat_r = cc.reshape(-1, cc.shape[-1]), cr.reshape(-1, cr.shape[-1])
    for t, slot in enumerate(slot_mapping.tolist()):
        if slot < 0:
            continue
        x, y = c[t], r[t].copy()
        if norm_weight is not None:
            x = x / np.sqrt(np.mean(x * x) + norm_eps) * _f64(norm_weight)
        if rope_cos is not None:
            p = t if positions is None else int(positions[t])
            cos, sin = _f64(rope_cos[p]), _f64(rope_sin[p])
            half = len(y) // 2
            i = np.arange(half)
            ia, ib = (2 * i, 2 * i + 1) if rope_interleaved else (i, i + half)
            a, b = r[t][ia], r[t][ib]
            y[ia], y[ib] = a * cos - b * sin, a * sin + b * cos
        flat_c[slot], flat_r[slot] = x, y
    return cc, cr


def prefix_mla(q_nope, q_rope, cache_c, cache_r, block_tables, cu_q_lens, seq_lens, prefix_pages, *, prefix_len,
               scale):
    """dict of out [T, H, R], lse [T, H], cond [T, H, R] = sum_s p_s |c_s| and reach [T, H] =
    max_s scale * sum_d |q_d k_d| (what the logits' rounding is relative to), n [T] keys seen.
    Positions that no table entry covers, or whose page is outside the cache, are left out."""
    qn, qr, cc, cr = _f64(q_nope), _f64(q_rope), _f64(cache_c), _f64(cache_r)
    page = cc.shape[1]
    bt, cu, lens = block_tables.cpu().numpy(), cu_q_lens.cpu().numpy(), seq_lens.cpu().numpy()
    pp = prefix_pages.cpu().numpy() if prefix_pages is not None else np.zeros(0, dtype=np.int64)
    T, H, R = qn.shape
    res = {"out": np.zeros((T, H, R)), "lse": np.full((T, H), -np.inf), "cond": np.zeros((T, H, R)),
           "reach": np.zeros((T, H)), "n": np.zeros(T, dtype=np.int64)}
    for b in range(len(lens)):
        q = int(cu[b + 1] - cu[b])
        for i in range(q):
            t, n = int(cu[b]) + i, int(lens[b]) - q + i + 1
            if n <= 0:
                continue
            pos = np.arange(n)
            tables = [pp if s < prefix_len else bt[b] for s in pos]
            pg = np.array([tab[s // page] if s // page < len(tab) else -1 for s, tab in zip(pos, tables)])
            there = (pg >= 0) & (pg < len(cc))
            if not there.any():
                continue
            pos, pg, n = pos[there], pg[there], int(there.sum())
            c, r = cc[pg, pos % page], cr[pg, pos % page]
            x = scale * (qn[t] @ c.T + qr[t] @ r.T)
            m = x.max(axis=1, keepdims=True)
            e = np.exp(x - m)
            total = e.sum(axis=1, keepdims=True)
            p = e / total
            res["out"][t], res["cond"][t] = p @ c, p @ np.abs(c)
            res["lse"][t] = (m + np.log(total))[:, 0]
            res["reach"][t] = (scale * (np.abs(qn[t]) @ np.abs(c).T + np.abs(qr[t]) @ np.abs(r).T)).max(axis=1)
            res["n"][t] = n
    return res
