"""Cases, plain forms and work of the quantised latent cache.

Three operators keep the latent cache in 8 or 4 bits and attend over it:

  store   dsa_mla_quant_append  a step's latent rows (norm, RoPE), quantised into the paged cache, and
          dsa_mla_quant_read    the new rows read back
  read    dsa_mla_quant_read    rows of requests' contexts read back as bf16
  attend  dsa_quant_mla         latent attention over the codes: the selected keys, or all of them

Where `own` is false, run() computes them with elementary torch operations; where it is true, it calls
the package.  A cache row holds 512 latent and 64 rotary values:

  fp8 (656 bytes)  512 e4m3 codes | 64 bf16 | scale 2^E (fp32) | 12 bytes
  fp4 (416 bytes)  512 4-bit codes | 64 bf16 | 32 bytes: the scales of blocks of 16

The rotary values are held divided by 2^E.  A 4-bit code is an e2m1 magnitude and a sign; the eight
magnitudes of a 32-bit word are its nibbles' low three bits, the signs of values 0..3 are bits 7, 15, 23
and 31, those of values 4..7 bits 3, 11, 19 and 27.  A scale byte's low seven bits are 8 (k + 5) + m for
s = 2^k (1 + m / 8); bit 7 of scale byte i is bit i of E + 128.  A code q stands for 2^E e4m3(q s).
"""
import math
import random

import torch

own = False

R, P = 512, 64  # latent and rotary widths of a row
ROW = {"fp8": 656, "fp4": 416}
FAR = 65536     # positions of the rotary table


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
        out.append((q, max(q, rng.randint(case["len_lo"], case["len_hi"]))))
    return out


def _cdiv(a, b):
    return -(-a // b)


# ---- the cases ---------------------------------------------------------------------------------

def _store(name, fmt, B, q_lo, q_hi, len_lo, len_hi, page, norm, rope, interleaved, lens):
    c = {"op": "store", "fmt": fmt, "B": B, "q_lo": q_lo, "q_hi": q_hi, "len_lo": len_lo, "len_hi": len_hi, "page": page,
         "norm": norm, "rope": rope, "interleaved": interleaved, "lens": lens}
    return dict(c, name=name) if name else c


def _read(name, fmt, B, len_lo, len_hi, page, lens):
    c = {"op": "read", "fmt": fmt, "B": B, "q_lo": 0, "q_hi": 0, "len_lo": len_lo, "len_hi": len_hi, "page": page,
         "lens": lens}
    return dict(c, name=name) if name else c


def _attend(name, fmt, B, H, topk, q_lo, q_hi, len_lo, len_hi, page, packed, lens):
    c = {"op": "attend", "fmt": fmt, "B": B, "H": H, "topk": topk, "q_lo": q_lo, "q_hi": q_hi, "len_lo": len_lo,
         "len_hi": len_hi, "page": page, "packed": packed, "lens": lens}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of 64 requests: latency counts
        _store("store_decode_b64_fp8", "fp8", 64, 1, 1, 1, 65536, 64, True, True, False, 1),
        # a prefill chunk: four requests' next tokens
        _store("store_chunk_b4_fp8", "fp8", 4, 1500, 2500, 8192, 32768, 64, True, True, True, 2),
        # many prompts at once, ragged lengths, small pages, 4 bits
        _store("store_b64_fp4", "fp4", 64, 1, 2047, 1, 2047, 16, True, True, False, 3),
        # one short context, 4 bits
        _read("read_b1_fp4", "fp4", 1, 1001, 1001, 64, 4),
        # eight contexts before their next chunk's attention
        _read("read_b8_fp8", "fp8", 8, 4096, 32768, 64, 5),
        # a few requests on a tensor-parallel rank, some shorter than the selection: latency counts
        _attend("attend_b4_h16_k2048_fp8", "fp8", 4, 16, 2048, 1, 1, 1, 4000, 64, False, 6),
        # the decode batch of 64 behind the indexer
        _attend("attend_b64_h64_k2048_fp8", "fp8", 64, 64, 2048, 1, 1, 4096, 65536, 64, False, 7),
        # the same over 4 bits
        _attend("attend_b64_h64_k2048_fp4", "fp4", 64, 64, 2048, 1, 1, 4096, 65536, 64, False, 8),
        # speculated tokens with all heads, queries as views of one tensor, an odd selection
        _attend("attend_mtp_b32_h128_k1001_fp4", "fp4", 32, 128, 1001, 1, 3, 500, 8000, 32, True, 9),
        # a prefill chunk's tokens, each with its own selection
        _attend("attend_chunk_b2_h64_k2048_fp8", "fp8", 2, 64, 2048, 500, 600, 4000, 16384, 64, False, 10),
        # every position of ragged contexts, 4 bits
        _attend("attend_all_b16_h64_fp4", "fp4", 16, 64, 0, 1, 1, 1, 65536, 64, False, 11),
        # one long request with all heads, every position
        _attend("attend_all_b1_h128_fp8", "fp8", 1, 128, 0, 1, 1, 40001, 40001, 128, False, 12),
    ]


def draw(rng):
    op = rng.choice(["store", "store", "read", "attend", "attend", "attend", "attend"])
    fmt = rng.choice(["fp8", "fp4"])
    lens = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128])
    if op == "store":
        B = _spread(rng, 1, 64)
        q_hi = _spread(rng, 1, 65536 // B)
        return _store("", fmt, B, rng.choice([0, min(1, q_hi), q_hi]) if B > 1 else q_hi, q_hi, 1, max(q_hi, _spread(rng, 1, 65536 // B)),
                      page, rng.random() < 0.8, rng.random() < 0.8, rng.random() < 0.5, lens)
    if op == "read":
        B = _spread(rng, 1, 64)
        hi = _spread(rng, 1, min(65536, 131072 // B))
        return _read("", fmt, B, rng.choice([1, hi]), hi, page, lens)
    H = rng.choice([8, 16, 20, 32, 64, 96, 128])
    if rng.random() < 0.3:  # every position
        B, q_hi = _spread(rng, 1, 16), rng.choice([1, 1, rng.randint(1, 4)])
        hi = max(q_hi, min(_spread(rng, 1, 65536), (1 << 20) // (B * q_hi)))
        return _attend("", fmt, B, H, 0, rng.choice([min(1, q_hi), q_hi]), q_hi, rng.choice([1, hi]), hi, page,
                       rng.random() < 0.3, lens)
    q_hi = rng.choice([1, 1, 1, rng.randint(1, 4), _spread(rng, 1, 512)])
    B = _spread(rng, 1, 64 if q_hi <= 4 else 2)
    topk = _spread(rng, 1, 2048)
    hi = max(q_hi, _spread(rng, 1, 65536 if B * q_hi <= 256 else 16384))
    return _attend("", fmt, B, H, topk, rng.choice([min(1, q_hi), q_hi]), q_hi, rng.choice([1, hi]), hi, page,
                   rng.random() < 0.3, lens)


# ---- rows of the cache -------------------------------------------------------------------------

def _pow2(e):
    """2^e in fp64, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exponent(a):
    """floor(log2 a) of positive fp64 values."""
    return (a.view(torch.int64) >> 52) - 1023


def _steps(a, least, bits):
    """The distance between neighbours of a >= 0 in a format of `bits` mantissa bits, normal down to 2^least."""
    return _pow2(_exponent(a.clamp(min=2.0 ** least)) - bits)


def _e4m3(x):
    step = _steps(x.abs(), -6, 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _row_exponent(c, top):
    """The smallest E with amax |c| <= top 2^E, per row."""
    t = c.abs().amax(1) / top
    e = _exponent(t.clamp(min=2.0 ** -200))
    return torch.where(t > 0, torch.where(t == _pow2(e), e, e + 1).clamp(-60, 60), 0)


def _bytes(x):
    return x.contiguous().view(torch.uint8)


def _pack(c, r, fmt):
    """Cache rows [n, bytes] of latent values c [n, 512] (fp64) and rotary values r [n, 64] (bf16)."""
    n = c.shape[0]
    E = _row_exponent(c, 448.0 if fmt == "fp8" else 432.0)
    rope = _bytes((r.double() / _pow2(E)[:, None]).to(torch.bfloat16))
    y = c / _pow2(E)[:, None]
    if fmt == "fp8":
        codes = _bytes(_e4m3(y).to(torch.float8_e4m3fn))
        scale = _bytes(_pow2(E).float()[:, None])
        return torch.cat([codes, rope, scale, torch.zeros((n, 12), dtype=torch.uint8, device=c.device)], 1)
    b = y.view(n, 32, 16)
    t = b.abs().amax(2) / 6.0
    step = _steps(t, -5, 3)
    s = (torch.ceil(t / step) * step).clamp(min=2.0 ** -5, max=72.0)
    k = _exponent(s)
    scale = ((k + 5) * 8 + ((s / _pow2(k) - 1.0) * 8.0).long()).to(torch.uint8)
    u = (b.abs() / s[:, :, None]).clamp(max=6.0)
    step = _steps(u, 0, 1)
    q = torch.round(u / step) * step
    mag = torch.where(q < 2, q * 2, torch.where(q < 4, q + 2, q / 2 + 4)).to(torch.int32).view(n, 64, 8)
    neg = (b < 0).to(torch.int32).view(n, 64, 8)
    at = torch.arange(8, device=c.device)
    sign_bit = torch.where(at < 4, 8 * at + 7, 8 * (at - 4) + 3)
    word = ((mag.long() << (4 * at)) | (neg.long() << sign_bit)).sum(2)
    word = (word - ((word >> 31) << 32)).to(torch.int32)
    hidden = ((E[:, None] + 128) >> torch.arange(8, device=c.device)) & 1
    scale[:, :8] += (hidden * 128).to(torch.uint8)
    return torch.cat([_bytes(word), rope, scale], 1)


def _unpack(rows, fmt):
    """(c [..., 512], r [..., 64]) fp32 of cache rows [..., bytes]."""
    if fmt == "fp8":
        scale = rows[..., 640:644].contiguous().view(torch.float32)
        return (rows[..., :512].contiguous().view(torch.float8_e4m3fn).float() * scale,
                rows[..., 512:640].contiguous().view(torch.bfloat16).float() * scale)
    dev, lead = rows.device, rows.shape[:-1]
    byte = rows[..., 384:416].int()
    E = ((byte[..., :8] >> 7) << torch.arange(8, device=dev, dtype=torch.int32)).sum(-1) - 128
    scale = ((E + 127) << 23).to(torch.int32).view(torch.float32)[..., None]
    code = byte & 127
    s = (1.0 + (code & 7).float() / 8.0) * ((((code >> 3) - 5 + 127) << 23).to(torch.int32).view(torch.float32))
    word = rows[..., :256].contiguous().view(torch.int32)[..., None]
    at = torch.arange(8, device=dev, dtype=torch.int32)
    sign_bit = torch.where(at < 4, 8 * at + 7, 8 * (at - 4) + 3)
    levels = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=dev)
    q = levels[((word >> (4 * at)) & 7).long()]
    q = torch.where(((word >> sign_bit) & 1) == 1, -q, q)
    v = (q.view(*lead, 32, 16) * s[..., None]).to(torch.float8_e4m3fn).float().view(*lead, R)
    return v * scale, rows[..., 256:384].contiguous().view(torch.bfloat16).float() * scale


# ---- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _sums(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def prepare(case, seed):
    g = _gen(seed)
    lengths, page, fmt = _lengths(case), case["page"], case["fmt"]
    need = [_cdiv(n, page) for _, n in lengths]
    total = sum(need) + 8
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    first = _ints(_sums(need)[:-1])
    j = torch.arange(max(1, max(need)), device="cuda")[None, :]
    bt = torch.where(j < _ints(need)[:, None], perm[(first[:, None] + j).clamp(max=total - 1)], -1).to(torch.int32)
    # rows as a model leaves them: normalised latent values, a channel's size its own
    pool = 16384
    channel = torch.exp(0.3 * _normal((R,), g, torch.float64))
    rows = _pack(_normal((pool, R), g, torch.float64) * channel, _normal((pool, P), g), fmt)
    cache = rows[torch.randint(0, pool, (total * page,), generator=g, device="cuda")].view(total, page, ROW[fmt])
    s = {"op": case["op"], "fmt": fmt, "page": page, "cache": cache, "bt": bt}
    if case["op"] == "read":
        lens = [n for _, n in lengths]
        return dict(s, cu=_ints(_sums(lens)), total=sum(lens), starts=None)
    T = sum(q for q, _ in lengths)
    cu = _ints(_sums([q for q, _ in lengths]))
    b = torch.repeat_interleave(torch.arange(case["B"], device="cuda"), _ints([q for q, _ in lengths]).long(), output_size=T)
    starts = _ints([n - q for q, n in lengths])
    pos = (starts.long()[b] + torch.arange(T, device="cuda") - cu.long()[b]).to(torch.int32)
    if case["op"] == "store":
        freq = 10000.0 ** (-torch.arange(0, P, 2, device="cuda", dtype=torch.float64) / P)
        ang = torch.arange(FAR, device="cuda", dtype=torch.float64)[:, None] * freq
        kv = _normal((T, R + P), g)  # the projection's output: both parts are views of its rows
        slots = bt[b, (pos // page).long()].long() * page + pos % page
        return dict(s, c=kv[:, :R], r=kv[:, R:], slots=slots, pos=pos if case["rope"] else None, cu=cu, total=T, starts=starts,
                    weight=channel.float() if case["norm"] else None, interleaved=case["interleaved"],
                    cos=ang.cos().float() if case["rope"] else None, sin=ang.sin().float() if case["rope"] else None)
    H, k = case["H"], case["topk"]
    if case["packed"]:
        q = _normal((T, H, R + P), g)
        qn, qr = q[:, :, :R], q[:, :, R:]
    else:
        qn, qr = _normal((T, H, R), g), _normal((T, H, P), g)
    longest = max(n for _, n in lengths)
    topk = None
    if k:  # a random choice of the positions that a query sees, in no order, then -1
        w = min(k, longest)
        chance = torch.rand((T, longest), generator=g, device="cuda")
        seen = torch.arange(longest, device="cuda")[None, :] <= pos[:, None]
        best, where = torch.where(seen, chance, -1.0).topk(w, dim=1)
        topk = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
        topk[:, :w] = torch.where(best >= 0, where, -1).to(torch.int32)
    return dict(s, qn=qn, qr=qr, cu=cu, seq_lens=_ints([n for _, n in lengths]), topk=topk, longest=longest,
                scale=(R + P) ** -0.5)


# ---- plain forms -------------------------------------------------------------------------------

def _plain_store(s):
    c = s["c"].double()  # values next to a border between two codes need more than 32 bits
    r = s["r"].float()
    if s["weight"] is not None:
        c = s["weight"].double() * c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-6)
    if s["cos"] is not None:
        cos, sin = s["cos"][s["pos"].long()], s["sin"][s["pos"].long()]
        if s["interleaved"]:
            a, b = r[:, 0::2], r[:, 1::2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], 2).reshape(r.shape)
        else:
            a, b = r[:, : P // 2], r[:, P // 2:]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], 1)
    s["cache"].view(-1, ROW[s["fmt"]])[s["slots"]] = _pack(c, r.to(torch.bfloat16), s["fmt"])
    return _plain_read(s)


def _plain_read(s):
    cu = s["cu"].long()
    t = torch.arange(s["total"], device=cu.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    p = t - cu[b] if s["starts"] is None else t - cu[b] + s["starts"].long()[b]
    slot = s["bt"][b, p // s["page"]].long() * s["page"] + p % s["page"]
    c, r = _unpack(s["cache"].view(-1, ROW[s["fmt"]])[slot], s["fmt"])
    return {"c": c.to(torch.bfloat16), "r": r.to(torch.bfloat16)}


def _plain_attend(s):
    q = torch.cat([s["qn"], s["qr"]], 2).float()
    T, dev = q.shape[0], q.device
    cu, n, page = s["cu"].long(), s["seq_lens"].long(), s["page"]
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:], t, right=True)
    if s["topk"] is not None:
        where = s["topk"].long()
        seen = where >= 0
    else:
        where = torch.arange(s["longest"], device=dev).expand(T, -1)
        seen = where <= (n[b] - cu[b + 1] + t)[:, None]
    where = where.clamp(min=0)
    slot = s["bt"][b[:, None], where // page].long().clamp(min=0) * page + where % page
    c, r = _unpack(s["cache"].view(-1, ROW[s["fmt"]])[slot], s["fmt"])
    x = (q[:, :, :R] @ c.transpose(1, 2) + q[:, :, R:] @ r.transpose(1, 2)) * s["scale"]
    x = torch.where(seen[:, None, :], x, -math.inf)
    m = x.amax(2, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(2, keepdim=True)
    return {"out": ((e @ c) / total).to(torch.bfloat16), "lse": (m + torch.log(total))[:, :, 0]}


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    if not own:
        return {"store": _plain_store, "read": _plain_read, "attend": _plain_attend}[s["op"]](s)
    import sparse_attention_token_gb300 as dsa
    if s["op"] == "attend":
        out, lse = dsa.dsa_quant_mla(s["qn"], s["qr"], s["cache"], s["bt"], s["cu"], s["seq_lens"], s["topk"],
                                     scale=s["scale"])
        return {"out": out, "lse": lse}
    if s["op"] == "store":
        dsa.dsa_mla_quant_append(s["c"], s["r"], s["slots"], s["cache"], norm_weight=s["weight"], rope_cos=s["cos"],
                                 rope_sin=s["sin"], positions=s["pos"], rope_interleaved=s["interleaved"])
    c, r = dsa.dsa_mla_quant_read(s["cache"], s["bt"], s["cu"], total=s["total"], starts=s["starts"])
    return {"c": c, "r": r}


def work(case):
    lengths, row = _lengths(case), ROW[case["fmt"]]
    T = sum(q for q, _ in lengths)
    if case["op"] == "read":
        n = sum(n for _, n in lengths)
        return {"bytes": n * (row + 2 * (R + P)), "flops": n * (R + P)}
    if case["op"] == "store":
        extra = 8 * T + (4 * R if case["norm"] else 0) + (T * (4 + 4 * P) if case["rope"] else 0)
        return {"bytes": T * (2 * 2 * (R + P) + 2 * row) + extra, "flops": T * (8 * R + 3 * P)}
    H, k = case["H"], case["topk"]
    sees = [n - q + i + 1 for q, n in lengths for i in range(q)]
    keys = [min(k, x) if k else x for x in sees]
    # rows that are read: every request's own, once; a selection's are counted once per query up to that
    rows, at = 0, 0
    for q, n in lengths:
        rows += min(n, sum(keys[at:at + q]))
        at += q
    return {"bytes": rows * row + T * H * (2 * (R + P) + 2 * R + 4) + (4 * T * k if k else 0),
            "flops": 2 * sum(keys) * H * (R + P + R)}


# ---- the definition in 64 bits -----------------------------------------------------------------

def _e4m3_values():
    """Every non-negative e4m3 value, ascending: its place in the list is its code."""
    return torch.tensor([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127],
                        dtype=torch.float64, device="cuda")


def _nearest(x, values):
    """The index of the value nearest to each |x|, an even one where two are as near."""
    i = torch.searchsorted(values, x.abs()).clamp(1, len(values) - 1)
    lo, hi = x.abs() - values[i - 1], values[i] - x.abs()
    return torch.where((lo < hi) | ((lo == hi) & (i % 2 == 1)), i - 1, i)


def _values_of(c, fmt):
    """What the codes of latent rows c [n, 512] (fp64) stand for."""
    grid = _e4m3_values()
    top = 448.0 if fmt == "fp8" else 432.0
    powers = 2.0 ** torch.arange(-60, 61, dtype=torch.float64, device="cuda")
    amax = c.abs().amax(1)
    E = powers[torch.searchsorted(powers * top, amax).clamp(max=120)][:, None]
    E = torch.where(amax[:, None] > 0, E, 1.0)
    y = c / E
    if fmt == "fp8":
        return torch.copysign(grid[_nearest(y, grid)], y) * E
    scales = torch.tensor([(1 + m / 8) * 2.0 ** k for k in range(-5, 7) for m in range(8)][:90], dtype=torch.float64, device="cuda")
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    b = y.view(-1, 32, 16)
    s = scales[torch.searchsorted(scales * 6, b.abs().amax(2)).clamp(max=89)][:, :, None]
    q = level[_nearest(b / s, level)] * s
    return torch.copysign(grid[_nearest(q, grid)], b).view(c.shape) * E


def _decode(rows, fmt):
    """(c, r) in fp64 of cache rows [n, bytes], byte by byte."""
    grid = _e4m3_values()
    if fmt == "fp8":
        byte = rows[:, :512].long()
        scale = rows[:, 640:644].contiguous().view(torch.float32).double()
        c = grid[(byte & 127).clamp(max=126)] * torch.where(byte > 127, -1.0, 1.0)
        return c * scale, rows[:, 512:640].contiguous().view(torch.bfloat16).double() * scale
    byte, tail = rows[:, :256].long(), rows[:, 384:].long()
    scale = sum((tail[:, i] >> 7) << i for i in range(8)).double()
    scale = torch.exp2(torch.round(scale - 128.0))[:, None]
    c = torch.zeros((rows.shape[0], R), dtype=torch.float64, device="cuda")
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    tail = tail & 127
    s = (1 + (tail % 8) / 8).double() * torch.exp2((tail // 8 - 5).double())
    for i in range(8):
        b4 = byte[:, i // 2::4]  # the byte that holds value i's nibble, in each of the 64 words
        mag = (b4 >> (4 * (i % 2))) & 7
        sign = (byte[:, i % 4::4] >> (7 if i < 4 else 3)) & 1
        v = level[mag] * s.repeat_interleave(2, 1)
        c[:, i::8] = grid[_nearest(v, grid)] * (1 - 2 * sign)
    return c * scale, rows[:, 256:384].contiguous().view(torch.bfloat16).double() * scale


def exact(case, seed):
    s = prepare(case, seed)
    fmt, page, lengths = case["fmt"], case["page"], _lengths(case)
    flat = s["cache"].view(-1, ROW[fmt])

    def slots_of(b, p):
        return s["bt"][b].long()[p // page] * page + p % page

    if case["op"] == "read":
        slot = torch.cat([slots_of(b, torch.arange(n, device="cuda")) for b, (_, n) in enumerate(lengths)])
        c, r = _decode(flat[slot], fmt)
        return {"c": c, "r": r}
    if case["op"] == "store":
        c, r = s["c"].double(), s["r"].double()
        if case["norm"]:
            c = c * s["weight"].double() / (torch.linalg.vector_norm(c, dim=1, keepdim=True) ** 2 / R + 1e-6).sqrt()
        if case["rope"]:
            z = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"].long()]
            first, second = torch.arange(0, P // 2, device="cuda"), torch.arange(P // 2, P, device="cuda")
            if case["interleaved"]:
                first, second = 2 * first, 2 * first + 1
            y = torch.complex(r[:, first], r[:, second]) * z
            r = r.clone()
            r[:, first], r[:, second] = y.real, y.imag
        return {"c": _values_of(c, fmt), "r": r}
    H, T = case["H"], s["qn"].shape[0]
    if work(case)["flops"] > 1.2e12:
        return None
    out = torch.zeros((T, H, R), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for b, (q, n) in enumerate(lengths):
        for i in range(q):
            if s["topk"] is None:
                where = torch.arange(n - q + i + 1, device="cuda")
            else:
                where = s["topk"][t]
                where = where[where >= 0].long()
            c, r = _decode(flat[slots_of(b, where)], fmt)
            x = (s["qn"][t].double() @ c.T + s["qr"][t].double() @ r.T) * s["scale"]
            lse[t] = torch.logsumexp(x, 1)
            out[t] = torch.exp(x - lse[t, :, None]) @ c
            t += 1
    return {"out": out, "lse": lse}
