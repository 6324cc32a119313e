"""CPU oracle of the quantised latent cache -- TEST INFRASTRUCTURE ONLY (numpy fp64, one row at a time).

encode_row  a row's bytes from its latent values (fp64) and its rotary values: the nearest code of every value,
            found by comparing with every value of the grid
decode_row  what the bytes stand for
quant_mla   softmax attention of every (query, head) row over its keys; also the sums that error bounds are made of
"""
from __future__ import annotations

import numpy as np
import torch

FP8, FP4 = 656, 416  # bytes of a row
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127])
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
SCALES = np.array([(1 + m / 8) * 2.0 ** k for k in range(-5, 7) for m in range(8)][:90])


def f64(t) -> np.ndarray:
    return t.detach().to(torch.float64).cpu().numpy()


def nearest(x, grid):
    """The place in `grid` nearest to each |x|, an even one where two are as near."""
    a = np.abs(np.asarray(x, dtype=np.float64))[..., None]
    d = np.abs(a - grid)
    i = d.argmin(-1)
    tie = (np.take_along_axis(d, np.minimum(i + 1, len(grid) - 1)[..., None], -1)[..., 0] == d.min(-1)) & (i + 1 < len(grid)) & (i % 2 == 1)
    return np.where(tie, i + 1, i)


def row_exponent(c, row):
    amax, top = np.abs(c).max(), 448.0 if row == FP8 else 432.0
    if amax == 0:
        return 0
    e = -60
    while e < 60 and amax > top * 2.0 ** e:
        e += 1
    return e


def bf16_bytes(v) -> np.ndarray:
    t = torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(torch.bfloat16)
    return t.view(torch.uint8).numpy()


def encode_row(c, r, row) -> np.ndarray:
    """The row's bytes; r fp64, rounded to bf16 before it is divided by the row's scale."""
    E = row_exponent(c, row)
    y = c / 2.0 ** E
    rope = bf16_bytes(torch.from_numpy(np.asarray(r)).to(torch.bfloat16).double().numpy() / 2.0 ** E)
    out = np.zeros(row, dtype=np.uint8)
    if row == FP8:
        out[:512] = nearest(y, E4M3) + np.where(np.signbit(y), 128, 0)
        out[512:640] = rope
        out[640:644] = np.frombuffer(np.float32(2.0 ** E).tobytes(), dtype=np.uint8)
        return out
    for b in range(32):
        v = y[16 * b: 16 * b + 16]
        code = min(int(np.searchsorted(6 * SCALES, np.abs(v).max())), len(SCALES) - 1)  # (rows above 2^60 saturate)
        q = nearest(v / SCALES[code], E2M1)
        out[384 + b] = code
        for j in range(16):
            word, i = 2 * b + j // 8, j % 8
            out[4 * word + i // 2] |= int(q[j]) << (4 * (i % 2))
            if np.signbit(v[j]):
                out[4 * word + i % 4] |= 0x80 if i < 4 else 0x08
    out[256:384] = rope
    for i in range(8):
        out[384 + i] |= ((E + 128) >> i & 1) << 7
    return out


def decode_row(b):
    """(c [512], r [64], the row's scale) of a row's bytes."""
    if len(b) == FP8:
        s = float(np.frombuffer(b[640:644].tobytes(), dtype=np.float32)[0])
        code = b[:512].astype(int)
        c = np.append(E4M3, np.nan)[code & 127] * np.where(code > 127, -1.0, 1.0)
        rope = b[512:640]
    else:
        s = 2.0 ** (sum((int(b[384 + i]) >> 7) << i for i in range(8)) - 128)
        c = np.zeros(512)
        for j in range(512):
            word, i = j // 8, j % 8
            mag = int(b[4 * word + i // 2]) >> (4 * (i % 2)) & 7
            neg = int(b[4 * word + i % 4]) >> (7 if i < 4 else 3) & 1
            v = E2M1[mag] * SCALES[b[384 + j // 16] & 127]
            c[j] = E4M3[nearest(v, E4M3)] * (-1.0 if neg else 1.0)
        rope = b[256:384]
    r = torch.from_numpy(rope.copy()).view(torch.bfloat16).double().numpy()
    return c * s, r * s, s


def decode_rows(cache: np.ndarray):
    """decode_row of every row of cache [n, row]: (c [n, 512], r [n, 64], scale [n])."""
    rows = [decode_row(b) for b in cache]
    return np.array([x[0] for x in rows]), np.array([x[1] for x in rows]), np.array([x[2] for x in rows])


def latent(c_kv, k_rope, *, norm_weight=None, norm_eps=1e-6, rope_cos=None, rope_sin=None, positions=None,
           rope_interleaved=False):
    """The rows that are to be quantised, in fp64."""
    c, r = f64(c_kv), f64(k_rope)
    if norm_weight is not None:
        c = f64(norm_weight) * c / np.sqrt((c * c).mean(1, keepdims=True) + float(np.float32(norm_eps)))
    if rope_cos is not None:
        p = np.arange(len(r)) if positions is None else positions.cpu().numpy()
        cos, sin = f64(rope_cos)[p], f64(rope_sin)[p]
        i = np.arange(32)
        ia, ib = (2 * i, 2 * i + 1) if rope_interleaved else (i, i + 32)
        a, b = r[:, ia].copy(), r[:, ib].copy()
        r = r.copy()
        r[:, ia], r[:, ib] = a * cos - b * sin, a * sin + b * cos
    return c, r


def quant_mla(q_nope, q_rope, rows, block_tables, cu_q_lens, seq_lens, topk=None, *, scale, page_size, num_pages):
    """dict of out [T, H, 512], lse [T, H] and what their error bounds are made of: cond [T, H, 512] = sum_s p_s |c_s|,
    square [T, H, 512] = sum_s p_s^2 c_s^2,
    tail [T, H, 512] = max_s(p_s S_s) sum_s |c_s| / S_s (S the rows' scales), tail2 = max_s(p_s S_s)^2 sum_s (c_s / S_s)^2,
    reach [T, H] = max_s scale sum_d |q_d k_d|,
    small [T, H] = max_s scale max_d |q_d| sum_d |k_d|, n [T] keys.  rows: (c, r, S) of every row of the cache.  A
    position that the table does not cover, or whose page is not in the cache, is left out."""
    qn, qr = f64(q_nope), f64(q_rope)
    c_all, r_all, s_all = rows
    bt, cu, lens = block_tables.cpu().numpy(), cu_q_lens.cpu().numpy(), seq_lens.cpu().numpy()
    tk = None if topk is None else topk.cpu().numpy()
    T, H, R = qn.shape
    res = {"out": np.zeros((T, H, R)), "lse": np.full((T, H), -np.inf), "cond": np.zeros((T, H, R)), "tail": np.zeros((T, H, R)),
           "reach": np.zeros((T, H)), "small": np.zeros((T, H)), "square": np.zeros((T, H, R)),
           "tail2": np.zeros((T, H, R)), "n": np.zeros(T, dtype=np.int64)}
    for b in range(len(lens)):
        q = int(cu[b + 1] - cu[b])
        for i in range(q):
            t = int(cu[b]) + i
            pos = np.arange(max(0, int(lens[b]) - q + i + 1)) if tk is None else tk[t][(tk[t] >= 0) & (tk[t] < lens[b])]
            lp = pos // page_size
            pg = np.where(lp < bt.shape[1], bt[b][np.minimum(lp, bt.shape[1] - 1)], -1) if bt.shape[1] else np.full(len(pos), -1)
            there = (pg >= 0) & (pg < num_pages)
            if not there.any():
                continue
            at = pg[there] * page_size + pos[there] % page_size
            c, r, S = c_all[at], r_all[at], s_all[at]
            x = scale * (qn[t] @ c.T + qr[t] @ r.T)
            m = x.max(1, keepdims=True)
            e = np.exp(x - m)
            p = e / e.sum(1, keepdims=True)
            res["out"][t], res["cond"][t] = p @ c, p @ np.abs(c)
            res["square"][t] = (p * p) @ (c * c)
            res["tail"][t] = (p * S).max(1, keepdims=True) * (np.abs(c) / S[:, None]).sum(0)
            res["tail2"][t] = (p * S).max(1, keepdims=True) ** 2 * ((c / S[:, None]) ** 2).sum(0)
            res["lse"][t] = (m + np.log(e.sum(1, keepdims=True)))[:, 0]
            ka = np.abs(c).sum(1) + np.abs(r).sum(1)
            res["reach"][t] = (scale * (np.abs(qn[t]) @ np.abs(c).T + np.abs(qr[t]) @ np.abs(r).T)).max(1)
            res["small"][t] = scale * np.maximum(np.abs(qn[t]).max(1), np.abs(qr[t]).max(1)) * ka.max()
            res["n"][t] = len(at)
    return res
