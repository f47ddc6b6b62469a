"""Beam search over a paged cache in 4 bits, with a sliding window and first tokens that stay visible.

    python examples/mxfp4_beam_decode.py [--beams 4] [--prompt 600] [--steps 64] [--window 256] [--sink 4]

One attention layer with random weights.  A prompt's rows go through
  1. idx_cache_resize            pages for the prompt;
  2. idx_cache_append_mxfp4      its keys and values, slices of one projection, into the pages;
  3. idx_window_attention_mxfp4  all of its tokens at once;
and idx_cache_fork hands its pages to every beam.  A decode step is the same three calls with one token per
beam (a beam that grows into a page it shares gets a copy of it), and a fork that lets every beam go on from one of
the best; idx_cache_compact moves what is left to the front of the pool.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_tiles_gb300 as idx  # noqa: E402

HEADS, KV_HEADS, DIM, HIDDEN, PAGE = 16, 4, 128, 512, 32


class Beams:
    def __init__(self, beams=4, longest=1024, window=256, sink=4, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.B, self.window, self.sink, self.longest, self.gen, self.dev = beams, window, sink, longest, g, device
        width = -(-longest // PAGE)
        pages = beams * width + beams
        ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device=device)  # noqa: E731
        shape = (pages, KV_HEADS, PAGE)
        self.cache = [torch.zeros(*shape, DIM // n, dtype=torch.uint8, device=device) for n in (2, 32, 2, 32)]
        self.refs, self.table, self.lens = ints(pages), ints(beams, width) - 1, ints(beams)
        self.qkv = rand((HEADS + 2 * KV_HEADS) * DIM, HIDDEN) / HIDDEN ** 0.5
        self.proj = rand(HIDDEN, HEADS * DIM) / (HEADS * DIM) ** 0.5
        self.hidden = None                       # the layer's input of the next step
        self.ws = torch.empty(max(256, idx.idx_cache_fork_workspace(beams, width),
                                  idx.idx_cache_resize_workspace(beams, pages, width),
                                  idx.idx_cache_compact_workspace(beams, pages)), dtype=torch.uint8, device=device)
        self.stats = idx.Stats(torch.device(device, torch.cuda.current_device()))
        self.said = None                         # (k, v) [beams, tokens, ...] as appended, on the host, when kept

    def attend(self, x, new):
        """The layer on x [T, HIDDEN], new[b] tokens of row b: (q, out, lse)."""
        T = x.shape[0]
        grow = self.lens + torch.tensor(new, dtype=torch.int32, device=self.dev)
        idx.idx_cache_resize(self.cache, self.refs, self.table, self.lens, grow, page_size=PAGE, refs_out=self.refs,
                             table_out=self.table, lens_out=self.lens, ws=self.ws, stats=self.stats)
        # a row for which the pages did not suffice has no slots for its new tokens: it sits this call out
        lens = torch.where(self.lens == grow, self.lens, 0)
        rows = (x @ self.qkv.t()).to(torch.bfloat16)
        q, k, v = (t.unflatten(1, (-1, DIM)) for t in rows.split([HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], 1))
        start = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device=self.dev)
        idx.idx_cache_append_mxfp4(k, v, *self.cache, self.table, lens, q_start=start, stats=self.stats)
        out, lse = idx.idx_window_attention_mxfp4(q, *self.cache, self.table, lens, q_start=start, max_q=max(new),
                                                  max_len=self.longest, window=self.window, sink=self.sink,
                                                  stats=self.stats)
        if self.said is not None:
            at = 0
            for b, n in enumerate(new):
                self.said[b] = [torch.cat([old, t[at:at + n].cpu()]) for old, t in zip(self.said[b], (k, v))]
                at += n
        return q, out, lse

    def prompt(self, tokens):
        """The prompt through row 0, whose pages every beam then holds."""
        x = torch.randn(tokens, HIDDEN, generator=self.gen, device=self.dev)
        if self.said is None and getattr(self, "keep", False):
            empty = torch.zeros(0, KV_HEADS, DIM, dtype=torch.bfloat16)
            self.said = [[empty, empty] for _ in range(self.B)]
        got = self.attend(x, [tokens] + [0] * (self.B - 1))
        self.follow([0] * self.B)
        self.hidden = (got[1][-1:].flatten(1).float() @ self.proj.t()).expand(self.B, -1)
        return got

    def step(self):
        """One token for every beam."""
        x = self.hidden + torch.randn(self.B, HIDDEN, generator=self.gen, device=self.dev)
        got = self.attend(x, [1] * self.B)
        self.hidden = got[1].flatten(1).float() @ self.proj.t()
        return got

    def follow(self, parents):
        """Beam b goes on from beam parents[b]."""
        parent = torch.tensor(parents, dtype=torch.int32, device=self.dev)
        idx.idx_cache_fork(self.refs, self.table, self.lens, parent, page_size=PAGE, refs_out=self.refs,
                           table_out=self.table, lens_out=self.lens, ws=self.ws, stats=self.stats)
        if self.hidden is not None:
            self.hidden = self.hidden[parent.long()]
        if self.said is not None:
            self.said = [list(self.said[p]) for p in parents]

    def compact(self):
        """The live pages to the front of the pool; how many there are."""
        return idx.idx_cache_compact(self.cache, self.refs, self.table, self.lens, page_size=PAGE, refs_out=self.refs,
                                     table_out=self.table, ws=self.ws, stats=self.stats)[2]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=600)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--window", type=int, default=256)
    ap.add_argument("--sink", type=int, default=4)
    a = ap.parse_args()
    d = Beams(a.beams, a.prompt + a.steps, a.window, a.sink)
    d.prompt(a.prompt)
    for i in range(a.steps):
        _, out, lse = d.step()
        # the beams that see the most stand for the best ones here
        best = lse.mean(1).topk(max(1, a.beams // 2)).indices.tolist()
        d.follow([best[b % len(best)] for b in range(a.beams)])
    live = d.compact()
    print(f"{a.beams} beams of {int(d.lens[0])} tokens behind a window of {a.window}: {int(live)} pages of {PAGE} live "
          f"({a.beams * -(-int(d.lens[0]) // PAGE)} without sharing), |out| {float(out.float().abs().mean()):.4f}, "
          f"status {d.stats.read()['status']}")


if __name__ == "__main__":
    main()
