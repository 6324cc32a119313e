"""Requests that begin with the same prompt, served with one copy of it.

A batch of requests shares a system prompt.  Its whole pages are filled once; then every step
makes the tables and slots of its new tokens (dsa_page_plan), writes their latent rows into the
paged cache (dsa_mla_cache_append) and attends over the prompt and each request's own tokens
(dsa_prefix_mla).  A layer that selects its keys runs on the same tables, slots and latent rows: its
index keys go through the same slots, dsa_indexer picks --topk keys a query, dsa_sparse_mla attends
over them; while a sequence has no more keys than that, both layers attend over the same ones.

    python examples/shared_prefix_step.py [--requests 32] [--heads 64] [--prompt 4100] [--steps 8] [--topk 2048]

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


def rope_tables(rows, device):
    freq = 10000.0 ** (-torch.arange(0, ROPE_DIM, 2, dtype=torch.float64, device=device) / ROPE_DIM)
    angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


class Batch:
    """The cache, the tables and the lengths of a batch behind one prompt."""

    def __init__(self, requests, heads, prompt, max_len, device="cuda", seed=0):
        self.device, self.heads, self.max_len = device, heads, max_len
        self.gen = torch.Generator(device=device).manual_seed(seed)
        shared = prompt // PAGE                       # whole pages are shared, the rest is each request's own
        width = -(-max_len // PAGE)
        pages = shared + requests * (width - shared)
        self.free = torch.randperm(pages, generator=self.gen, device=device).to(torch.int32)
        self.prefix_pages, self.free = self.free[:shared].contiguous(), self.free[shared:].contiguous()
        self.prefix_len = shared * PAGE
        self.cache_c = torch.empty((pages, PAGE, KV_RANK), dtype=torch.bfloat16, device=device)
        self.cache_r = torch.empty((pages, PAGE, ROPE_DIM), dtype=torch.bfloat16, device=device)
        self.cache_k = torch.empty((pages, PAGE, INDEX_DIM), dtype=torch.bfloat16, device=device)
        self.tables = torch.full((requests, width), -1, dtype=torch.int32, device=device)
        self.lens = torch.full((requests,), self.prefix_len, dtype=torch.int32, device=device)
        self.cos, self.sin = rope_tables(max_len, device)
        self.norm = torch.ones(KV_RANK, device=device)
        # the prompt's whole pages, once: one "request" that owns exactly the shared pages
        one = torch.full((1,), self.prefix_len, dtype=torch.int32, device=device)
        table = torch.full((1, max(shared, 1)), -1, dtype=torch.int32, device=device)
        _, slots, positions, _ = dsa.dsa_page_plan(one, one, table, self.prefix_pages, page_size=PAGE,
                                                   total_q=self.prefix_len)
        self._append(slots, positions)

    def _randn(self, *shape):
        return torch.randn(shape, generator=self.gen, device=self.device).to(torch.bfloat16)

    def _append(self, slots, positions):
        kv = self._randn(slots.shape[0], KV_RANK + ROPE_DIM)  # the down-projection's output
        dsa.dsa_mla_cache_append(kv[:, :KV_RANK], kv[:, KV_RANK:], slots, self.cache_c, self.cache_r,
                                 norm_weight=self.norm, rope_cos=self.cos, rope_sin=self.sin, positions=positions)
        dsa.dsa_indexer_cache_append(self._randn(slots.shape[0], INDEX_DIM), slots, self.cache_k)

    def step(self, new_tokens, topk=0):
        """A step of new_tokens[b] tokens of request b: latent attention output [total, heads, 512] and
        lse over all keys, and (topk > 0) the output over topk selected keys a query, else None."""
        q_lens = torch.tensor(new_tokens, dtype=torch.int32, device=self.device)
        self.lens += q_lens
        total = sum(new_tokens)
        cu, slots, positions, used = dsa.dsa_page_plan(q_lens, self.lens, self.tables, self.free, page_size=PAGE,
                                                       total_q=total, prefix_pages=self.prefix_pages)
        self._append(slots, positions)
        q = self._randn(total, self.heads, KV_RANK + ROPE_DIM)  # absorbed queries
        out, lse = dsa.dsa_prefix_mla(q[..., :KV_RANK], q[..., KV_RANK:], self.cache_c, self.cache_r, self.tables, cu,
                                      self.lens, self.prefix_pages, prefix_len=self.prefix_len, scale=SCALE)
        selected = None
        if topk > 0:
            index_q, index_w = self._randn(total, INDEX_HEADS, INDEX_DIM), self._randn(total, INDEX_HEADS).float()
            keys = dsa.dsa_indexer(index_q, index_w, self.cache_k, cu, self.lens, self.tables, max_seq_len=self.max_len,
                                   topk_limit=topk)
            selected = dsa.dsa_sparse_mla(q[..., :KV_RANK].contiguous(), q[..., KV_RANK:].contiguous(), self.cache_c,
                                          self.cache_r, self.tables, cu, self.lens, keys, scale=SCALE)
        self.free = self.free[int(used):].contiguous()  # the pages taken leave the free list
        return out, lse, selected


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=32)
    ap.add_argument("--heads", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=4100)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--topk", type=int, default=2048, help="keys that the selecting layer keeps (0: no such layer)")
    a = ap.parse_args()
    rest = a.prompt % PAGE
    own = [rest + 3 + 5 * b for b in range(a.requests)]  # what the shared pages do not hold, and the request's text
    batch = Batch(a.requests, a.heads, a.prompt, a.prompt + max(own) + a.steps + PAGE)
    out, lse, _ = batch.step(own)
    print(f"prompts: {sum(own)} tokens behind {batch.prefix_len} shared, out {tuple(out.shape)}, "
          f"lse {lse.min().item():.2f} .. {lse.max().item():.2f}")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    batch.step([1] * a.requests, a.topk)
    start.record()
    for _ in range(a.steps - 1):
        out, lse, selected = batch.step([1] * a.requests, a.topk)
    end.record()
    torch.cuda.synchronize()
    status = dsa.dsa_check_device_status()
    if status != dsa.DSA_OK:
        raise dsa.DsaError(status, "shared_prefix_step")
    print(f"decode: {a.requests} x {a.heads} rows a step, lengths {batch.lens.min().item()} .. "
          f"{batch.lens.max().item()}, {start.elapsed_time(end) / max(a.steps - 1, 1):.3f} ms a step")
    if a.steps > 1 and a.topk >= batch.lens.max().item():
        worst = (selected - out.float()).abs().max().item()
        print(f"every key selected: the two layers' outputs differ by at most {worst:.4f} "
              f"(the larger {out.float().abs().max().item():.2f})")


if __name__ == "__main__":
    main()
