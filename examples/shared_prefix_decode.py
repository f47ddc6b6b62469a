"""Decoding a batch of requests about one shared document, with every cache on a budget.

    python examples/shared_prefix_decode.py [--requests 8] [--prefix 4096] [--steps 96]

One attention layer with random weights.  A decode step is
  1. idx_add_rmsnorm_quant  the residual's sum and norm, e4m3 rows with scales per 128 columns,
                            the projections' input (dequantised here: the projections are torch's);
  2. the new K and V rows go to each request's next slot (page table);
  3. idx_prefix_attention   over the document, read once for all requests, and the own slots,
                            adding up what every own slot receives;
  4. idx_cache_evict        once a request is over its budget: the slots that gathered least go.
Beside it the sparse path: the document's index keys are normed straight to the k and k_scale
that idx_score_topk reads, and the selected positions become cache slots through the page table.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_tiles_gb300 as idx  # noqa: E402

HEADS, KV_HEADS, DIM, HIDDEN, PAGE = 16, 4, 128, 1024, 64


def dequantise(codes, scale, group):
    return (codes.float().reshape(*scale.shape, group) * scale[..., None]).reshape(codes.shape)


class Decoder:
    def __init__(self, requests=8, prefix=4096, budget=128, room=64, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.B, self.prefix, self.budget, self.dev = requests, prefix, budget, device
        self.max_len = budget + room  # slots of a request: the budget and what may come before an eviction
        own = -(-self.max_len // PAGE)
        pages = -(-prefix // PAGE)
        ids = torch.randperm(pages + requests * own, generator=g, device=device).to(torch.int32)
        self.prefix_table = ids[:pages].contiguous()
        self.table = ids[pages:].reshape(requests, own).contiguous()
        shape = (len(ids), KV_HEADS, PAGE, DIM)
        self.k, self.v = (rand(*shape).to(torch.bfloat16) for _ in range(2))
        slots = (requests, KV_HEADS, own * PAGE)
        self.lens = torch.zeros(requests, dtype=torch.int32, device=device)
        self.seen = torch.zeros_like(self.lens)
        # double-buffered: a step reads one and writes the other
        self.weights = [torch.zeros(slots, device=device) for _ in range(2)]
        self.positions = [torch.full(slots, -1, dtype=torch.int32, device=device) for _ in range(2)]
        self.norm = (1 + 0.1 * rand(HIDDEN)).to(torch.bfloat16)
        self.qkv = rand((HEADS + 2 * KV_HEADS) * DIM, HIDDEN) / HIDDEN ** 0.5
        self.proj = rand(HIDDEN, HEADS * DIM) / (HEADS * DIM) ** 0.5
        self.residual = rand(requests, HIDDEN).to(torch.bfloat16)
        self.delta = torch.zeros_like(self.residual)  # what the layer before adds
        self.ws_attn = torch.empty(idx.idx_prefix_attention_workspace(
            requests, 1, HEADS, KV_HEADS, DIM, prefix, self.max_len, True), dtype=torch.uint8, device=device)
        self.ws_evict = torch.empty(max(256, idx.idx_cache_evict_workspace(
            requests, KV_HEADS, budget, self.max_len)), dtype=torch.uint8, device=device)
        # the index side of the document: one key per position
        self.index_norm = (1 + 0.1 * rand(DIM)).to(torch.bfloat16)
        self.index_keys = idx.idx_add_rmsnorm_quant(rand(prefix, DIM).to(torch.bfloat16), self.index_norm)
        self.n = 0  # host copy of lens: every request decodes one token a step

    def step(self):
        """One token for every request; the attention's (q, out, lse)."""
        codes, scale = idx.idx_add_rmsnorm_quant(self.delta, self.norm, residual=self.residual,
                                                 residual_out=self.residual, group=128)
        x = dequantise(codes, scale, 128) @ self.qkv.t()
        q, k, v = (t.reshape(self.B, -1, DIM).to(torch.bfloat16)
                   for t in x.split([HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], 1))
        page = self.table[:, self.n // PAGE].long()
        self.k[page, :, self.n % PAGE], self.v[page, :, self.n % PAGE] = k, v
        self.positions[0][:, :, self.n] = self.seen[:, None]
        self.lens += 1
        self.seen += 1
        self.n += 1
        out, lse, _ = idx.idx_prefix_attention(
            q[:, None].contiguous(), self.k, self.v, self.table, self.lens, prefix_table=self.prefix_table,
            prefix_len=self.prefix, max_len=self.max_len, weights=self.weights[0],
            weights_out=self.weights[1], ws=self.ws_attn)
        self.weights.reverse()
        self.delta = (out.reshape(self.B, -1).float() @ self.proj.t()).to(torch.bfloat16)
        return q, out[:, 0], lse[:, 0]

    def evict(self):
        """Back to the budget: the last quarter of it and the first two tokens stay in any case."""
        self.lens, _, _ = idx.idx_cache_evict(
            self.k, self.v, self.table, self.lens, self.weights[0], self.positions[0], self.seen, self.budget,
            recent=self.budget // 4, sink=2, max_len=self.max_len, weights_out=self.weights[1],
            positions_out=self.positions[1], ws=self.ws_evict)
        self.weights.reverse()
        self.positions.reverse()
        self.n = min(self.n, self.budget)

    def select(self, q, topk=256):
        """The sparse path: cache slots of the document's topk keys by the indexer, per request."""
        codes, scale = idx.idx_add_rmsnorm_quant(q.reshape(-1, DIM), self.index_norm)
        rows = torch.arange(self.B, dtype=torch.int32, device=self.dev)
        at = idx.idx_score_topk(codes.reshape(self.B, HEADS, DIM), *self.index_keys,
                                scale.reshape(self.B, HEADS) / HEADS, torch.zeros_like(rows),
                                torch.full_like(rows, self.prefix), topk)
        return idx.idx_page_table_transform(at, self.prefix_table[None], PAGE, row_map=torch.zeros_like(rows))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prefix", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=96)
    a = ap.parse_args()
    d = Decoder(a.requests, a.prefix, budget=48, room=16)
    evictions = 0
    for _ in range(a.steps):
        q, out, lse = d.step()
        if d.n == d.max_len:
            d.evict()
            evictions += 1
    slots = d.select(q)
    torch.cuda.synchronize()
    print(f"{a.steps} steps of {a.requests} requests behind {a.prefix} tokens: {d.n} slots kept of {int(d.seen[0])} "
          f"tokens after {evictions} evictions; |out| {float(out.float().abs().mean()):.4f}, lse "
          f"{float(lse.mean()):.3f}; the indexer picked {int((slots >= 0).sum())} slots")


if __name__ == "__main__":
    main()
