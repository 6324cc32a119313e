"""Requests served from a latent cache in 8 or 4 bits.

Every step plans its tables and slots (dsa_page_plan), writes its latent rows as codes
(dsa_mla_quant_append) and attends over the codes (dsa_quant_mla): a layer over every position, and
one over the keys that dsa_indexer selects.  A prompt of many tokens reads its request's rows back as
bf16 instead (dsa_mla_quant_read) and attends over them with dsa_prefix_mla, which goes through them
once for all of its tokens.

    python examples/quantised_cache_step.py [--requests 16] [--heads 64] [--prompt 3000] [--steps 8] [--topk 2048] [--bits 8]

Activations are random; the projections around the attention belong to the model and are left out.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_token_gb300 as dsa  # noqa: E402

KV_RANK, ROPE_DIM, PAGE = 512, 64, 64
INDEX_HEADS, INDEX_DIM = 64, 128
SCALE = (KV_RANK + ROPE_DIM) ** -0.5


class Batch:
    """The cache in `bits` bits, the tables and the lengths of a batch."""

    def __init__(self, requests, heads, max_len, bits=8, device="cuda", seed=0):
        self.device, self.heads, self.max_len = device, heads, max_len
        self.gen = torch.Generator(device=device).manual_seed(seed)
        width = -(-max_len // PAGE)
        pages = requests * width
        row = dsa.dsa_mla_quant_row_bytes(dsa.DSA_FP8_E4M3 if bits == 8 else dsa.DSA_FP4_E2M1)
        self.cache = torch.empty((pages, PAGE, row), dtype=torch.uint8, device=device)
        self.cache_k = torch.empty((pages, PAGE, INDEX_DIM), dtype=torch.bfloat16, device=device)
        self.free = torch.randperm(pages, generator=self.gen, device=device).to(torch.int32)
        self.tables = torch.full((requests, width), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(requests, dtype=torch.int32, device=device)
        self.norm = torch.ones(KV_RANK, device=device)
        freq = 10000.0 ** (-torch.arange(0, ROPE_DIM, 2, dtype=torch.float64, device=device) / ROPE_DIM)
        angle = torch.arange(max_len, dtype=torch.float64, device=device)[:, None] * freq
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def _randn(self, *shape):
        return torch.randn(shape, generator=self.gen, device=self.device).to(torch.bfloat16)

    def _write(self, new_tokens):
        """Plans and writes a step's rows; the queries' offsets."""
        q_lens = torch.tensor(new_tokens, dtype=torch.int32, device=self.device)
        self.lens += q_lens
        total = sum(new_tokens)
        cu, slots, positions, used = dsa.dsa_page_plan(q_lens, self.lens, self.tables, self.free, page_size=PAGE, total_q=total)
        kv = self._randn(total, KV_RANK + ROPE_DIM)  # the down-projection's output
        dsa.dsa_mla_quant_append(kv[:, :KV_RANK], kv[:, KV_RANK:], slots, self.cache, norm_weight=self.norm, rope_cos=self.cos,
                                 rope_sin=self.sin, positions=positions)
        dsa.dsa_indexer_cache_append(self._randn(total, INDEX_DIM), slots, self.cache_k)
        self.free = self.free[int(used):].contiguous()
        return cu, self._randn(total, self.heads, KV_RANK + ROPE_DIM)  # absorbed queries

    def prompt(self, new_tokens):
        """Attention output and lse of prompts, over rows read back into pages of bf16."""
        cu, q = self._write(new_tokens)
        # every request's rows in whole pages, one request behind the other: what follows a sequence's end in its last page may be
        # anything, no query sees it
        held = (self.lens + PAGE - 1) // PAGE
        ends = torch.nn.functional.pad(held.cumsum(0), (1, 0)).to(torch.int32)
        total = int(ends[-1])
        c, r = dsa.dsa_mla_quant_read(self.cache, self.tables, ends * PAGE, total=total * PAGE)
        page = torch.arange(int(held.max()), dtype=torch.int32, device=self.device)[None]
        pages = torch.where(page < held[:, None], ends[:-1, None] + page, -1)
        return dsa.dsa_prefix_mla(q[..., :KV_RANK], q[..., KV_RANK:], c.view(-1, PAGE, KV_RANK), r.view(-1, PAGE, ROPE_DIM), pages, cu,
                                  self.lens, prefix_len=0, scale=SCALE)

    def step(self, new_tokens, topk):
        """(out, lse) over every position and over topk selected keys a query."""
        cu, q = self._write(new_tokens)
        total = q.shape[0]
        attend = lambda keys: dsa.dsa_quant_mla(q[..., :KV_RANK], q[..., KV_RANK:], self.cache, self.tables, cu, self.lens, keys, scale=SCALE)
        keys = dsa.dsa_indexer(self._randn(total, INDEX_HEADS, INDEX_DIM), self._randn(total, INDEX_HEADS).float(), self.cache_k, cu,
                               self.lens, self.tables, max_seq_len=self.max_len, topk_limit=topk)
        return attend(None), attend(keys)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--heads", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=3000)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--topk", type=int, default=2048)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 4))
    a = ap.parse_args()
    prompts = [max(1, a.prompt - 7 * b) for b in range(a.requests)]
    batch = Batch(a.requests, a.heads, a.prompt + a.steps + 1, a.bits)
    out, lse = batch.prompt(prompts)
    print(f"prompts: {sum(prompts)} tokens, out {tuple(out.shape)}, lse {lse.min().item():.2f} .. {lse.max().item():.2f}, "
          f"cache {batch.cache.numel() / 1e6:.1f} MB (bf16: {batch.cache.numel() // batch.cache.shape[2] * 1152 / 1e6:.1f})")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    every, selected = batch.step([1] * a.requests, a.topk)
    start.record()
    for _ in range(a.steps - 1):
        every, selected = batch.step([1] * a.requests, a.topk)
    end.record()
    torch.cuda.synchronize()
    status = dsa.dsa_check_device_status()
    if status != dsa.DSA_OK:
        raise dsa.DsaError(status, "quantised_cache_step")
    print(f"decode: {a.requests} x {a.heads} rows a step, {start.elapsed_time(end) / max(a.steps - 1, 1):.3f} ms a step")
    if a.topk >= batch.lens.max().item():
        worst = (selected[0].float() - every[0].float()).abs().max().item()
        print(f"every key selected: the two layers' outputs differ by at most {worst:.4f} "
              f"(the larger {every[0].float().abs().max().item():.2f})")


if __name__ == "__main__":
    main()
