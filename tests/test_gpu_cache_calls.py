"""The operators of the cache in 4 bits and of its pages as a program calls them: on streams of their own, captured and
replayed, with guarded workspaces, one after another without synchronisation, and the beam search example."""
import os
import sys

import pytest
import torch

from _cache_ref import append, attention, check_attention, counts, held, quantise, starts
from test_gpu_window_attention import problem

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
DEV = "cuda"
GUARD = 4096


@pytest.fixture(scope="module")
def idx():
    import sparse_attention_indexer_tiles_gb300 as pkg
    pkg.load()
    return pkg


def on_gpu(p):
    return {n: [c.to(DEV) for c in t] if isinstance(t, list) else t.to(DEV) for n, t in p.items()}


def state(seed=0, new=(3, 1, 40)):
    p = problem([200, 77, 300], list(new), 4, 2, 128, 16, "bf16", seed=seed)
    d = on_gpu(p)
    g = torch.Generator().manual_seed(seed)
    d["k"], d["v"] = (torch.randn(sum(new), 2, 128, generator=g).bfloat16().to(DEV) for _ in range(2))
    pages = d["cache"][0].shape[0]
    d["refs"] = counts(held(p["table"], p["lens"], 16), pages).to(DEV)
    d["wide"] = torch.nn.functional.pad(d["table"], (0, 3), value=-1)
    d["parent"] = torch.tensor([1, 1, 0], dtype=torch.int32, device=DEV)
    d["new_lens"] = torch.tensor([205, 70, 320], dtype=torch.int32, device=DEV)
    return d


def calls(idx, d, **kw):
    """Every operator, with all that it can leave to the call left to it."""
    def appended():
        idx.idx_cache_append_mxfp4(d["k"], d["v"], *d["cache"], d["table"], d["lens"], q_start=d["q_start"], **kw)
        return d["cache"]
    pages = (d["refs"], d["wide"], d["lens"])
    return {
        "append": appended,
        "attention": lambda: idx.idx_window_attention_mxfp4(d["q"], *d["cache"], d["table"], d["lens"], q_start=d["q_start"],
                                                            window=50, sink=3, **kw),
        "dense": lambda: idx.idx_window_attention_mxfp4(d["q"], *d["cache"], d["table"], d["lens"], q_start=d["q_start"],
                                                        options={"row_split": 1}, **kw),
        "fork": lambda: idx.idx_cache_fork(*pages, d["parent"], page_size=16, **kw),
        "resize": lambda: idx.idx_cache_resize(d["cache"], *pages, d["new_lens"], page_size=16, **kw),
        "compact": lambda: idx.idx_cache_compact(d["cache"], *pages, page_size=16, **kw)}


NAMES = ["append", "attention", "dense", "fork", "resize", "compact"]


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_on_a_stream_of_its_own(idx, name, handle):
    """The caller's stream is busy before the call and takes memory of the call's sizes after it."""
    want = [t.clone() for t in calls(idx, state())[name]()]
    torch.cuda.synchronize()
    a = torch.randn(4096, 4096, device=DEV)
    side = torch.cuda.Stream()
    for _ in range(4):
        d = state()
        torch.cuda.synchronize()
        for _ in range(8):
            a @ a
        got = calls(idx, d, stream=side.cuda_stream if handle else side)[name]()
        trash = [torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) for n in [1 << k for k in range(9, 25)] * 2]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), name
        del trash, got


def chain(idx, d, ws):
    """A step as a serving loop makes it, everything in place."""
    kw = dict(refs_out=d["refs"], table_out=d["wide"], lens_out=d["lens"], ws=ws)
    idx.idx_cache_fork(d["refs"], d["wide"], d["lens"], d["parent"], page_size=16, **kw)
    torch.add(d["lens"], 1, out=d["new_lens"])
    idx.idx_cache_resize(d["cache"], d["refs"], d["wide"], d["lens"], d["new_lens"], page_size=16, **kw)
    idx.idx_cache_append_mxfp4(d["k"], d["v"], *d["cache"], d["wide"], d["lens"])
    idx.idx_window_attention_mxfp4(d["q"], *d["cache"], d["wide"], d["lens"], window=60, sink=2, max_len=400, out=d["out"],
                                   lse=d["lse"], ws=ws)
    kw.pop("lens_out")
    idx.idx_cache_compact(d["cache"], d["refs"], d["wide"], d["lens"], page_size=16, live=d["live"], **kw)
    d["k"].copy_(d["out"][:, :2] * 0.5)


def chain_state():
    d = state(4, (1, 1, 1))
    d["wide"] = torch.nn.functional.pad(d["wide"], (0, 10), value=-1)
    pages = d["cache"][0].shape[0] + 40
    d["cache"] = [torch.cat([c, torch.zeros(40, *c.shape[1:], dtype=c.dtype, device=DEV)]) for c in d["cache"]]
    d["refs"] = torch.cat([d["refs"], torch.zeros(40, dtype=torch.int32, device=DEV)])
    assert d["refs"].numel() == pages
    d["out"], d["lse"] = torch.zeros_like(d["q"]), torch.zeros(3, 8, device=DEV)
    d["live"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return d


KEYS = ("out", "lse", "lens", "refs", "wide", "live", "k")


def test_a_chain_of_calls_eager_and_captured(idx):
    """Without any synchronisation, and replayed from two graphs that share the workspace, the same bits."""
    ws = torch.full((1 << 22,), 0x77, dtype=torch.uint8, device=DEV)
    d, want = chain_state(), []
    for _ in range(12):
        chain(idx, d, ws)
        torch.cuda.synchronize()
        want.append([d[n].clone() for n in KEYS] + [c.clone() for c in d["cache"]])
    d = chain_state()
    for _ in range(12):
        chain(idx, d, ws)
    assert all(torch.equal(x, y) for x, y in zip([d[n] for n in KEYS] + d["cache"], want[-1]))
    d, copy = chain_state(), chain_state()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        chain(idx, copy, ws)
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                chain(idx, d, ws)
            graphs.append(g)
    torch.cuda.synchronize()
    for i in range(12):
        ws.fill_(i)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip([d[n] for n in KEYS] + d["cache"], want[i])), i


def guarded(n):
    buf = torch.full((n + GUARD,), 0x5A, dtype=torch.uint8, device=DEV)
    return buf, buf[:n]


@pytest.mark.parametrize("lens,new,group,heads,D,path", [
    ([40, 7], [1, 1], 4, 2, 64, 0), ([300, 1000, 5], [3, 16, 1], 7, 2, 128, 0), ([9000], [1], 8, 1, 128, 0),
    ([5000], [4], 16, 2, 128, 0), ([6000, 400], [20, 30], 16, 1, 64, 1), ([900], [300], 8, 2, 128, 1),
    ([700] * 20, [2] * 20, 8, 1, 64, -1)])
def test_the_attention_stays_inside_its_workspace(idx, lens, new, group, heads, D, path):
    p = problem(lens, new, group, heads, D, 32, "fp16", seed=1)
    d = on_gpu(p)
    T, Hq = d["q"].shape[:2]
    need = idx.idx_window_attention_mxfp4_workspace(len(lens), T, max(new), Hq, heads, D, max(lens), 0, 0)
    buf, ws = guarded(need)
    kw = dict(q_start=d["q_start"], max_q=max(new), max_len=max(lens), options={"row_split": path})
    a = idx.idx_window_attention_mxfp4(d["q"], *d["cache"], d["table"], d["lens"], ws=ws, **kw)
    b = idx.idx_window_attention_mxfp4(d["q"], *d["cache"], d["table"], d["lens"], **kw)
    torch.cuda.synchronize()
    assert (buf[-GUARD:] == 0x5A).all() and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", ["fork", "resize", "compact"])
@pytest.mark.parametrize("B,width,pages", [(1, 1, 1), (3, 4, 9), (200, 9, 1000), (700, 30, 30000)])
def test_the_pages_calls_stay_inside_their_workspaces(idx, name, B, width, pages):
    """Tables full of pages that all may change hands, and every page free at first for the resize."""
    g = torch.Generator().manual_seed(B)
    table = torch.randint(0, pages, (B, width), generator=g, dtype=torch.int32).to(DEV)
    refs = torch.randint(0, 2, (pages,), generator=g, dtype=torch.int32).to(DEV)
    lens = torch.full((B,), 16 * width, dtype=torch.int32, device=DEV)
    cache = torch.zeros(pages, 16, dtype=torch.uint8, device=DEV)
    if name == "fork":
        buf, ws = guarded(idx.idx_cache_fork_workspace(B, width))
        idx.idx_cache_fork(refs, table, lens, torch.zeros_like(lens), page_size=16, table_out=table, lens_out=lens, ws=ws)
    elif name == "resize":
        buf, ws = guarded(idx.idx_cache_resize_workspace(B, pages, width))
        refs.zero_()
        idx.idx_cache_resize([cache], refs, table, torch.zeros_like(lens), lens, page_size=16, ws=ws)
    else:
        buf, ws = guarded(idx.idx_cache_compact_workspace(B, pages))
        idx.idx_cache_compact([cache], refs, table, lens, page_size=16, ws=ws)
    torch.cuda.synchronize()
    assert (buf[-GUARD:] == 0x5A).all()


def test_the_binding_refuses_what_does_not_fit(idx):
    d = state()
    cache, args = d["cache"], (d["table"], d["lens"])
    bad = [
        lambda: idx.idx_window_attention_mxfp4(d["q"].float(), *cache, *args, q_start=d["q_start"]),
        lambda: idx.idx_window_attention_mxfp4(d["q"][:, :, :64], *cache, *args, q_start=d["q_start"]),
        lambda: idx.idx_window_attention_mxfp4(d["q"].transpose(0, 1), *cache, *args, q_start=d["q_start"]),
        lambda: idx.idx_window_attention_mxfp4(d["q"], cache[0], cache[0], cache[2], cache[3], *args, q_start=d["q_start"]),
        lambda: idx.idx_window_attention_mxfp4(d["q"], *cache, d["table"].long(), d["lens"], q_start=d["q_start"]),
        lambda: idx.idx_window_attention_mxfp4(d["q"], *cache, d["table"], d["lens"][:2], q_start=d["q_start"]),
        lambda: idx.idx_window_attention_mxfp4(d["q"], *cache, *args, q_start=d["q_start"][:3]),
        lambda: idx.idx_window_attention_mxfp4(d["q"], *cache, *args, q_start=d["q_start"], out=d["q"][1:]),
        lambda: idx.idx_window_attention_mxfp4(d["q"], *(c.cpu() for c in cache), *args, q_start=d["q_start"]),
        lambda: idx.idx_cache_append_mxfp4(d["k"], d["v"][1:], *cache, *args, q_start=d["q_start"]),
        lambda: idx.idx_cache_append_mxfp4(d["k"], d["v"].half(), *cache, *args, q_start=d["q_start"]),
        lambda: idx.idx_cache_append_mxfp4(d["k"][:, :1], d["v"][:, :1], *cache, *args, q_start=d["q_start"]),
        lambda: idx.idx_cache_fork(d["refs"], d["table"], d["lens"], d["parent"].long(), page_size=16),
        lambda: idx.idx_cache_fork(d["refs"], d["table"], d["lens"], d["parent"], page_size=16, table_out=d["wide"]),
        lambda: idx.idx_cache_resize([cache[0][1:]], d["refs"], d["table"], d["lens"], d["lens"], page_size=16),
        lambda: idx.idx_cache_resize(cache * 3, d["refs"], d["table"], d["lens"], d["lens"], page_size=16),
        lambda: idx.idx_cache_resize([None], d["refs"], d["table"], d["lens"], d["lens"], page_size=16),
        lambda: idx.idx_cache_compact([cache[0].transpose(2, 3)], d["refs"], d["table"], d["lens"], page_size=16)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, idx.IdxError)):  # (a type that libidx names but this call does not take: its own)
            f()
            pytest.fail(str(i))
    with pytest.raises(TypeError):
        idx.idx_cache_resize(5, d["refs"], d["table"], d["lens"], d["lens"], page_size=16)
    with pytest.raises(idx.IdxError):
        idx.idx_cache_resize([torch.zeros(d["refs"].numel(), 5, dtype=torch.uint8, device=DEV)], d["refs"], d["table"],
                             d["lens"], d["lens"], page_size=16)
    with pytest.raises(idx.IdxError):
        idx.idx_window_attention_mxfp4(d["q"], *cache, *args)          # 44 tokens of 3 requests


def test_beams_over_a_cache_in_4_bits(idx):
    """The example: what every beam should hold, quantised on the host, against the attention's results, the pages and the
    counts after each step."""
    import mxfp4_beam_decode as ex
    d = ex.Beams(beams=3, longest=200, window=40, sink=3, seed=3)
    d.keep = True
    g = torch.Generator().manual_seed(1)

    def cache_of(said):
        """One request's (k, v) rows as a cache of a single page row each."""
        out = []
        for x in said:
            codes, sf = quantise(x)
            n = -(-x.shape[0] // 16) * 16
            pad = lambda t: torch.cat([t, torch.zeros(n - x.shape[0], *t.shape[1:], dtype=t.dtype)])  # noqa: E731
            out += [pad(t).unflatten(0, (-1, 16)).transpose(1, 2).contiguous() for t in (codes, sf)]
        return out

    def check(q, out, lse, new):
        at = 0
        for b, n in enumerate(new):
            if n:
                length = d.said[b][0].shape[0]
                table = torch.arange(-(-length // 16), dtype=torch.int32)[None]
                ref = attention(q[at:at + n].cpu(), cache_of(d.said[b]), table, torch.tensor([length]), starts([n]), 40, 3)
                check_attention([out[at:at + n].cpu(), lse[at:at + n].cpu()], ref, torch.bfloat16, length, 128)
            at += n

    got = d.prompt(90)
    check(*got, [90, 0, 0])
    for step in range(60):
        got = d.step()
        if step % 10 == 0:
            check(*got, [1, 1, 1])
        d.follow(torch.randint(0, 3, (3,), generator=g).tolist())
        if step % 20 == 7:
            live = int(d.compact())
            assert live == len({p for r in held(d.table.cpu(), d.lens.cpu(), ex.PAGE) for p in r}) == int((d.refs > 0).sum())
    assert d.lens.tolist() == [150] * 3 and d.stats.read()["status"] == 0
    rows = held(d.table.cpu(), d.lens.cpu(), ex.PAGE)
    assert torch.equal(d.refs.cpu(), counts(rows, d.refs.numel()))
    for b in range(3):
        table = torch.tensor(rows[b], dtype=torch.int32)[None]
        empty = [torch.zeros_like(c).cpu() for c in d.cache]
        want = append(*d.said[b], empty, table, torch.tensor([150]), starts([150]))
        for page in rows[b]:
            for c, w in zip(d.cache, want):
                used = 150 - ex.PAGE * rows[b].index(page)
                assert torch.equal(c[page, :, :used].cpu(), w[page, :, :used])
