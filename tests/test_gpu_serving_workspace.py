"""The serving operators' workspaces: exactly the bytes that are asked for, with guard bytes behind
them, and one buffer over calls of several sizes."""
import pytest
import torch

from test_gpu_prefix_attention import BF16, DEV, FP16, idx, make  # noqa: F401
from test_gpu_evict import make as make_cache

pytestmark = pytest.mark.gpu
GUARD = 4096


def guarded(n):
    buf = torch.full((n + GUARD,), 0x5A, dtype=torch.uint8, device=DEV)
    return buf, buf[:n]


def attention(idx, s, ws, max_len):  # noqa: F811
    d = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in s.items()}
    got = idx.idx_prefix_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], prefix_table=d["prefix_table"],
                                   prefix_len=d["prefix_len"], weights=d["w"], max_len=max_len, ws=ws)
    torch.cuda.synchronize()
    return got


def size(idx, s, max_len):  # noqa: F811
    B, Q, Hq, D = s["q"].shape
    return idx.idx_prefix_attention_workspace(B, Q, Hq, s["k"].shape[1], D, s["prefix_len"], max_len,
                                              s["w"] is not None)


SHAPES = [([40, 7], 1, 4, 2, 64, 100, BF16), ([300, 1000, 5], 3, 7, 2, 128, 700, FP16), ([900], 1, 8, 1, 128, 0, BF16),
          ([50] * 33, 1, 8, 4, 128, 5000, BF16), ([700] * 24, 16, 8, 4, 128, 40, BF16), ([20000], 4, 8, 2, 64, 64, BF16)]


@pytest.mark.parametrize("shape", SHAPES)
def test_attention_stays_inside(idx, shape):  # noqa: F811
    lens, Q, G, Hkv, D, prefix, dtype = shape
    for weights in (True, False):
        s = make(lens, Q, G, Hkv, D, prefix, 32, dtype, seed=1, weights=weights)
        buf, ws = guarded(size(idx, s, max(lens)))
        a = attention(idx, s, ws, max(lens))
        assert (buf[-GUARD:] == 0x5A).all()
        b = attention(idx, s, None, max(lens))
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_one_attention_workspace_for_all(idx):  # noqa: F811
    """Sized for the largest of every argument, used by calls of all the shapes in turn, twice."""
    need = idx.idx_prefix_attention_workspace(33, 16, 32, 4, 128, 5000, 20000, True)
    buf, ws = guarded(need)
    for _ in range(2):
        for lens, Q, G, Hkv, D, prefix, dtype in SHAPES:
            s = make(lens, Q, G, Hkv, D, prefix, 32, dtype, seed=2)
            want = attention(idx, s, None, max(lens))
            assert all(torch.equal(x, y) for x, y in zip(attention(idx, s, ws, max(lens)), want))
    assert (buf[-GUARD:] == 0x5A).all()


@pytest.mark.parametrize("lens,budget", [([2049] * 3, 2048), ([5000, 300], 1000), ([70001], 512), ([64], 1)])
def test_eviction_stays_inside(idx, lens, budget):  # noqa: F811
    s = make_cache(lens, 2, 64, 32, seed=3)
    buf, ws = guarded(idx.idx_cache_evict_workspace(len(lens), 2, budget, max(lens)))
    got = []
    for w in (ws, None):
        d = {n: t.to(DEV) for n, t in s.items()}
        out = idx.idx_cache_evict(d["k"], d["v"], d["table"], d["lens"], d["w"], d["pos"], d["next"], budget,
                                  max_len=max(lens), ws=w)
        torch.cuda.synchronize()
        got.append([*out, d["k"], d["v"]])
    assert (buf[-GUARD:] == 0x5A).all()
    assert all(torch.equal(x, y) for x, y in zip(*got))
