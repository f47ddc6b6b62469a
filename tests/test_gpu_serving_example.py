"""The shared-prefix decoding example: its steps against a plain 64-bit attention over the
tokens that the cache should hold, with a host-side book of what every eviction kept."""
import os
import sys

import pytest
import torch

import _serve_ref as ref

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_decode_steps_and_evictions():
    import __graft_entry__
    __graft_entry__.build()
    import shared_prefix_decode as ex
    d = ex.Decoder(requests=3, prefix=700, budget=48, room=16, seed=5)
    for step in range(100):
        before = d.weights[0].cpu().clone()
        q, out, lse = d.step()
        if step % 9 == 0 or d.n == d.max_len:
            torch.cuda.synchronize()
            cpu = lambda t: t.cpu()  # noqa: E731
            want = ref.attention(cpu(q)[:, None], cpu(d.k), cpu(d.v), cpu(d.table), cpu(d.lens), cpu(d.prefix_table),
                                 d.prefix, None, before)
            ref.check_attention([cpu(out)[:, None], cpu(lse)[:, None], cpu(d.weights[0])], want, torch.bfloat16,
                                d.prefix + d.n, ex.DIM, lens=cpu(d.lens))
        if d.n == d.max_len:
            state = [t.cpu().clone() for t in (d.k, d.v, d.table, d.lens, d.weights[0], d.positions[0], d.seen)]
            d.evict()
            k, v, lens, w, pos = ref.evict(*state, 48, 12, 2)
            assert torch.equal(d.lens.cpu(), lens) and d.n == 48
            assert torch.equal(d.weights[0].cpu()[:, :, :48], w[:, :, :48])
            assert torch.equal(d.positions[0].cpu()[:, :, :48], pos[:, :, :48])
            assert torch.equal(d.k.cpu().view(torch.int16), k.view(torch.int16))
    assert int(d.seen[0]) == 100
    # every head still holds the sinks and the last tokens
    kept = d.positions[0].cpu()[:, :, :d.n].long().sort(2).values
    assert (kept[:, :, :2] == torch.arange(2)).all() and (kept[:, :, -1] == 99).all()
    slots = d.select(q, 64)
    pages = set(d.prefix_table.tolist())
    assert slots.shape == (3, 64) and all(s // ex.PAGE in pages for s in slots.flatten().tolist())
