"""Cases, plain forms and work of the shared-prefix serving operators.

Three operators make one step of a batch of requests that begin with the same prompt:

  plan    dsa_page_plan         block tables, slot mapping, positions and query offsets from request lengths
  append  dsa_mla_cache_append  the step's latent rows (norm, RoPE) through the slot mapping into the paged cache
  attend  dsa_prefix_mla        latent attention, the prefix computed once for the whole batch

Where `own` is false, run() computes them with elementary torch operations in fp32; where it is
true, it calls the package.
"""
import math
import random

import torch

own = False

R, P = 512, 64  # latent and rotary widths of the cache rows


# ---- lengths: part of the case, drawn from its own "lens" number ------------------------------

def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(max(hi, 1))))))))


def _lengths(case):
    """(new tokens, total length) of every request."""
    rng = random.Random(case["lens"])
    out = []
    for _ in range(case["B"]):
        q = rng.randint(case["q_lo"], case["q_hi"])
        own_len = rng.randint(case["own_lo"], case["own_hi"])
        out.append((q, case["prefix"] + max(q, own_len)))
    return out


def _cdiv(a, b):
    return -(-a // b)


# ---- the cases ---------------------------------------------------------------------------------

def _plan(name, B, q_lo, q_hi, own_lo, own_hi, prefix, page, max_pages, lens):
    c = {"op": "plan", "B": B, "q_lo": q_lo, "q_hi": q_hi, "own_lo": own_lo, "own_hi": own_hi, "prefix": prefix,
         "page": page, "max_pages": max_pages, "lens": lens}
    return dict(c, name=name) if name else c


def _append(name, T, page, pages, norm, rope, interleaved):
    c = {"op": "append", "T": T, "page": page, "pages": pages, "norm": norm, "rope": rope, "interleaved": interleaved}
    return dict(c, name=name) if name else c


def _attend(name, B, H, prefix, q_lo, q_hi, own_lo, own_hi, page, packed, lens):
    c = {"op": "attend", "B": B, "H": H, "prefix": prefix, "q_lo": q_lo, "q_hi": q_hi, "own_lo": own_lo,
         "own_hi": own_hi, "page": page, "packed": packed, "lens": lens}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of 64 requests behind an 8K system prompt: the table and slots of one new token each
        _plan("plan_decode_b64", 64, 1, 1, 1, 57344, 8192, 64, 1024, 1),
        # sixteen new requests admitted with their whole prompts
        _plan("plan_prefill_b16", 16, 1, 8192, 1, 8192, 2048, 64, 256, 2),
        # a large decode batch with one to three speculated tokens, small pages, long tables
        _plan("plan_speculative_b1024", 1024, 1, 3, 1, 65536, 4096, 16, 4352, 3),
        # the decode step's 64 new latent rows
        _append("append_decode_t64", 64, 64, 4096, True, True, False),
        # a prefill chunk of 8192 tokens
        _append("append_chunk_t8192", 8192, 64, 4096, True, True, True),
        # many requests' prompts at once, ragged count
        _append("append_t65537", 65537, 32, 8192, True, True, False),
        # a few requests on a tensor-parallel rank: latency counts
        _attend("attend_b4_h16_p1000", 4, 16, 1000, 1, 1, 1, 200, 64, False, 4),
        # one request alone, a long prompt: the long axis is all there is to share out
        _attend("attend_b1_h64_p65536", 1, 64, 65536, 1, 1, 17, 17, 64, False, 5),
        # the decode batch of 64 behind an 8K prompt
        _attend("attend_b64_h64_p8192", 64, 64, 8192, 1, 1, 1, 1024, 64, False, 6),
        # many requests on a tensor-parallel rank, long prompt, long own parts
        _attend("attend_b128_h16_p32768", 128, 16, 32768, 1, 1, 64, 4096, 64, False, 7),
        # speculated tokens with all heads, queries as views of one tensor, pages of 32, odd lengths
        _attend("attend_mtp_b32_h128_p4001", 32, 128, 4001, 1, 3, 3, 2000, 32, True, 8),
        # the requests' own prompts prefilled behind the shared one
        _attend("attend_prefill_b8_h64_p6000", 8, 64, 6000, 1, 512, 1, 700, 64, False, 9),
    ]


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend"])
    lens = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _spread(rng, 1, 1024)
        own_hi = _spread(rng, 1, 65536)
        prefix = rng.choice([0, page * _spread(rng, 1, 8192 // page)])
        q_hi = _spread(rng, 1, min(own_hi, max(1, 131072 // B)))
        max_pages = _cdiv(prefix + max(own_hi, q_hi), page) + rng.randint(0, 64)
        if B * max_pages > 4 << 20:
            B = max(1, (4 << 20) // max_pages)
        return _plan("", B, rng.choice([0, 1]), q_hi, rng.choice([1, own_hi]), own_hi, prefix, page, max_pages, lens)
    if op == "append":
        T = _spread(rng, 1, 65536)
        pages = _cdiv(T, page) + _spread(rng, 1, 2048)
        return _append("", T, page, pages, rng.random() < 0.8, rng.random() < 0.8, rng.random() < 0.5)
    H = rng.choice([8, 16, 20, 32, 64, 128])
    q_hi = rng.choice([1, 1, 1, rng.randint(1, 4), _spread(rng, 1, 512)])
    B = _spread(rng, 1, max(1, 128 if q_hi <= 4 else 8))
    prefix = rng.choice([0, _spread(rng, 1, 65536), _spread(rng, 1, 65536), _spread(rng, 1, 65536)])
    own_hi = max(q_hi, _spread(rng, 1, 4096))
    rows = B * q_hi * H
    # the plain form's products and score tensors stay within those of the listed cases
    prefix = min(prefix, (1 << 29) // rows, int(8e11 / 2176 / rows))
    own_hi = min(own_hi, max(q_hi, (1 << 29) // rows))
    return _attend("", B, H, prefix, rng.choice([min(1, q_hi), q_hi]), q_hi, rng.choice([1, own_hi]), own_hi, page,
                   rng.random() < 0.3, lens)


# ---- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _tables(case, lengths, g, held):
    """Pages in a seeded permutation: block tables with the pages that hold `held` tokens of every
    request, the shared prefix's pages, and the pages left over."""
    page, B = case["page"], case["B"]
    shared = case["prefix"] // page
    need = [_cdiv(h, page) - shared if h > shared * page else 0 for h in held]
    total = _cdiv(case["prefix"], page) + sum(need) + sum(_cdiv(s, page) + 1 for _, s in lengths)
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    n_prefix = _cdiv(case["prefix"], page)
    prefix_pages = perm[:n_prefix].contiguous()
    width = case.get("max_pages") or max(1, max(_cdiv(s, page) for _, s in lengths))
    n = torch.tensor(need, device="cuda")
    first = n_prefix + torch.cumsum(n, 0) - n
    j = torch.arange(width, device="cuda")[None, :] - shared
    own_page = perm[(first[:, None] + j).clamp(0, total - 1)]
    bt = torch.where((j >= 0) & (j < n[:, None]), own_page, -1)
    if shared:
        bt[:, :shared] = prefix_pages[:shared]
    used = n_prefix + sum(need)
    return bt.to(torch.int32).contiguous(), prefix_pages, perm[used:].contiguous(), total


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "plan":
        lengths = _lengths(case)
        page = case["page"]
        bt, prefix_pages, free, _ = _tables(case, lengths, g, [s - q for q, s in lengths])
        return {"op": "plan", "page": page, "bt": bt, "free": free,
                "prefix_pages": prefix_pages[: case["prefix"] // page],
                "q_lens": torch.tensor([q for q, _ in lengths], dtype=torch.int32, device="cuda"),
                "seq_lens": torch.tensor([s for _, s in lengths], dtype=torch.int32, device="cuda"),
                "total_q": sum(q for q, _ in lengths)}
    if case["op"] == "append":
        T, page, pages = case["T"], case["page"], case["pages"]
        slots = torch.randperm(page * pages, generator=g, device="cuda")[:T]
        # a step padded to its graph's size: the last few tokens may have no slot
        if T > 8:
            slots[T - T // 64 - 1:] = -1
        far = 65536
        pos = torch.randint(0, far, (T,), generator=g, device="cuda", dtype=torch.int32)
        freq = 10000.0 ** (-torch.arange(0, P, 2, device="cuda", dtype=torch.float64) / P)
        ang = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * freq
        kv = _normal((T, R + P), g)  # the projection's output: both parts are views of its rows
        return {"op": "append", "c": kv[:, :R], "r": kv[:, R:], "slots": slots, "pos": pos if case["rope"] else None,
                "weight": 1 + 0.1 * _normal((R,), g, torch.float32) if case["norm"] else None,
                "cos": ang.cos().float() if case["rope"] else None, "sin": ang.sin().float() if case["rope"] else None,
                "interleaved": case["interleaved"], "cache_c": _normal((pages, page, R), g),
                "cache_r": _normal((pages, page, P), g)}
    lengths = _lengths(case)
    page, H = case["page"], case["H"]
    bt, prefix_pages, _, total = _tables(case, lengths, g, [s for _, s in lengths])
    T = sum(q for q, _ in lengths)
    cu = [0]
    for q, _ in lengths:
        cu.append(cu[-1] + q)
    if case["packed"]:
        q = _normal((T, H, R + P), g)
        qn, qr = q[:, :, :R], q[:, :, R:]
    else:
        qn, qr = _normal((T, H, R), g), _normal((T, H, P), g)
    return {"op": "attend", "qn": qn, "qr": qr, "cache_c": _normal((total, page, R), g),
            "cache_r": _normal((total, page, P), g), "bt": bt, "prefix_pages": prefix_pages,
            "prefix": case["prefix"], "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"),
            "seq_lens": torch.tensor([s for _, s in lengths], dtype=torch.int32, device="cuda"),
            "scale": (R + P) ** -0.5, "q_max": max(q for q, _ in lengths),
            "own_max": max(s for _, s in lengths) - case["prefix"]}


# ---- plain forms -------------------------------------------------------------------------------

def _plain_plan(s):
    page, bt = s["page"], s["bt"]
    q, n = s["q_lens"].long(), s["seq_lens"].long()
    B, width = bt.shape
    cu = torch.zeros(B + 1, dtype=torch.int64, device=bt.device)
    cu[1:] = torch.cumsum(q, 0)
    shared = s["prefix_pages"].numel()
    held = torch.maximum((n - q + page - 1) // page, torch.full_like(n, shared))
    have = torch.maximum((n + page - 1) // page, torch.full_like(n, shared))
    new = have - held
    first = torch.cumsum(new, 0) - new
    j = torch.arange(width, device=bt.device)[None, :]
    fresh = s["free"][(first[:, None] + j - held[:, None]).clamp(0, s["free"].numel() - 1)]
    table = torch.where(j < held[:, None], bt, torch.where(j < have[:, None], fresh, -1))
    if shared:
        table[:, :shared] = s["prefix_pages"]
    table = torch.where((n > 0)[:, None], table, -1).to(torch.int32)
    t = torch.arange(s["total_q"], device=bt.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    pos = n[b] - q[b] + t - cu[b]
    slot = table[b, pos // page].long() * page + pos % page
    return {"block_tables": table, "cu_q_lens": cu.to(torch.int32), "slot_mapping": slot,
            "positions": pos.to(torch.int32), "used": new.sum().to(torch.int32).reshape(1)}


def _plain_append(s):
    c, r = s["c"].float(), s["r"].float()
    if s["weight"] is not None:
        c = c * torch.rsqrt((c * c).mean(1, keepdim=True) + 1e-6) * s["weight"]
    if s["cos"] is not None:
        cos, sin = s["cos"][s["pos"].long()], s["sin"][s["pos"].long()]
        if s["interleaved"]:
            a, b = r[:, 0::2], r[:, 1::2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], 2).reshape(r.shape)
        else:
            a, b = r[:, : P // 2], r[:, P // 2:]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], 1)
    keep = s["slots"] >= 0
    s["cache_c"].view(-1, R)[s["slots"][keep]] = c[keep].to(torch.bfloat16)
    s["cache_r"].view(-1, P)[s["slots"][keep]] = r[keep].to(torch.bfloat16)
    return {"cache_c": s["cache_c"], "cache_r": s["cache_r"]}


def _plain_attend(s):
    qn, qr = s["qn"].float(), s["qr"].float()
    T, H = qn.shape[:2]
    page, prefix, dev = s["cache_c"].shape[1], s["prefix"], qn.device
    cu, n = s["cu"].long(), s["seq_lens"].long()
    B = n.numel()
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    sees = n[b] - (cu[b + 1] - cu[b]) + t - cu[b] + 1  # keys that each query sees, its own among them
    # the prefix, for all queries at once
    kc = s["cache_c"][s["prefix_pages"].long()].reshape(-1, R)[:prefix].float()
    kr = s["cache_r"][s["prefix_pages"].long()].reshape(-1, P)[:prefix].float()
    one = (qn.reshape(-1, R) @ kc.T + qr.reshape(-1, P) @ kr.T).view(T, H, prefix) * s["scale"]
    # each request's own keys, padded to the longest, against its padded queries
    j = torch.arange(s["q_max"], device=dev)
    row = (cu[:-1, None] + j).clamp(max=T - 1)
    p = prefix + torch.arange(s["own_max"], device=dev)
    slot = s["bt"].long()[:, p // page].clamp(min=0) * page + p % page
    oc, orr = s["cache_c"].view(-1, R)[slot].float(), s["cache_r"].view(-1, P)[slot].float()
    two = (qn[row].reshape(B, -1, R) @ oc.transpose(1, 2) + qr[row].reshape(B, -1, P) @ orr.transpose(1, 2)) * s["scale"]
    seen = p[None, None, None, :] < sees[row][:, :, None, None]
    two = torch.where(seen, two.view(B, s["q_max"], H, -1), -math.inf)
    # back from the padded rows to the queries, then one softmax over both parts
    at = (b, t - cu[b])
    two_t = two[at]
    m = torch.maximum(two_t.amax(2), one.amax(2)) if prefix else two_t.amax(2)
    e1, e2 = torch.exp(one - m[:, :, None]), torch.exp(two - m[row][:, :, :, None])
    total = e1.sum(2) + e2.sum(3)[at]
    out = (e1.view(T * H, prefix) @ kc).view(T, H, R) + (e2.view(B, -1, s["own_max"]) @ oc).view(B, -1, H, R)[at]
    return {"out": (out / total[:, :, None]).to(torch.bfloat16), "lse": m + torch.log(total)}


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)
    import sparse_attention_token_gb300 as dsa
    if s["op"] == "plan":
        cu, slots, pos, used = dsa.dsa_page_plan(s["q_lens"], s["seq_lens"], s["bt"], s["free"], page_size=s["page"],
                                                 total_q=s["total_q"], prefix_pages=s["prefix_pages"])
        return {"block_tables": s["bt"], "cu_q_lens": cu, "slot_mapping": slots, "positions": pos, "used": used}
    if s["op"] == "append":
        dsa.dsa_mla_cache_append(s["c"], s["r"], s["slots"], s["cache_c"], s["cache_r"], norm_weight=s["weight"],
                                 rope_cos=s["cos"], rope_sin=s["sin"], positions=s["pos"],
                                 rope_interleaved=s["interleaved"])
        return {"cache_c": s["cache_c"], "cache_r": s["cache_r"]}
    out, lse = dsa.dsa_prefix_mla(s["qn"], s["qr"], s["cache_c"], s["cache_r"], s["bt"], s["cu"], s["seq_lens"],
                                  s["prefix_pages"], prefix_len=s["prefix"], scale=s["scale"])
    return {"out": out, "lse": lse}


def work(case):
    if case["op"] == "plan":
        lengths, page = _lengths(case), case["page"]
        T, shared = sum(q for q, _ in lengths), case["prefix"] // page
        new = sum(_cdiv(s, page) - max(_cdiv(s - q, page), shared) for q, s in lengths)
        tail = sum(case["max_pages"] - max(_cdiv(s - q, page), shared) for q, s in lengths)  # entries that change
        return {"bytes": 12 * case["B"] + 4 + 4 * new + 4 * shared * (1 + case["B"]) + 4 * tail + 12 * T, "flops": 0}
    if case["op"] == "append":
        T = case["T"]
        kept = T - (T // 64 + 1 if T > 8 else 0)
        extra = 8 * T + (4 * R if case["norm"] else 0) + (kept * (4 + 4 * P) if case["rope"] else 0)
        return {"bytes": 2 * 2 * kept * (R + P) + extra, "flops": kept * (4 * R * case["norm"] + 3 * P * case["rope"])}
    lengths, H = _lengths(case), case["H"]
    T = sum(q for q, _ in lengths)
    keys = case["prefix"] + sum(s - case["prefix"] for _, s in lengths)
    pairs = sum(q * s - q * (q - 1) // 2 for q, s in lengths)  # (query, key) pairs, causal among the new tokens
    return {"bytes": 2 * keys * (R + P) + T * H * (2 * (R + P) + 2 * R + 4),
            "flops": 2 * pairs * H * (R + P + R)}


# ---- the definition in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "append":
        out_c, out_r = s["cache_c"].double(), s["cache_r"].double()
        live = [i for i, x in enumerate((s["slots"] >= 0).tolist()) if x]
        c, r, slot = s["c"][live].double(), s["r"][live].double(), s["slots"][live]
        if case["norm"]:
            c = s["weight"].double() * c / (torch.linalg.vector_norm(c, dim=1, keepdim=True) ** 2 / R + 1e-6).sqrt()
        if case["rope"]:
            z = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"][live].long()]
            a, b = (r[:, 0::2], r[:, 1::2]) if case["interleaved"] else (r[:, : P // 2], r[:, P // 2:])
            y = torch.complex(a, b) * z
            first, second = torch.arange(0, P // 2, device="cuda"), torch.arange(P // 2, P, device="cuda")
            if case["interleaved"]:
                first, second = 2 * first, 2 * first + 1
            r = r.clone()
            r[:, first], r[:, second] = y.real, y.imag
        out_c.view(-1, R)[slot], out_r.view(-1, P)[slot] = c, r
        return {"cache_c": out_c, "cache_r": out_r}
    lengths, H, page = _lengths(case), case["H"], case["page"]
    pairs = sum(q * n for q, n in lengths) * H
    if pairs * 2176 > 2.5e12:
        return None
    T = s["qn"].shape[0]
    out = torch.zeros((T, H, R), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for b, (q, n) in enumerate(lengths):
        # the sequence's latent rows in order: the prefix's, then its own
        where = torch.arange(n, device="cuda")
        pages = s["bt"][b].long()[where // page]
        pre = where[: case["prefix"]]
        if case["prefix"]:
            pages[: case["prefix"]] = s["prefix_pages"].long()[pre // page]
        key = torch.cat([s["cache_c"][pages, where % page], s["cache_r"][pages, where % page]], 1).double()
        for i in range(0, q, 64):
            k = min(q, i + 64)
            query = torch.cat([s["qn"][t + i: t + k], s["qr"][t + i: t + k]], 2).double()
            x = torch.einsum("qhd,sd->qhs", query, key) * s["scale"]
            last = n - q + torch.arange(i, k, device="cuda")
            x = x.masked_fill(where[None, None, :] > last[:, None, None], -math.inf)
            lse[t + i: t + k] = torch.logsumexp(x, 2)
            out[t + i: t + k] = torch.einsum("qhs,sd->qhd", torch.exp(x - lse[t + i: t + k, :, None]), key[:, :R])
        t += q
    return {"out": out, "lse": lse}
