"""idx_cache_evict with weights that are not numbers: a NaN of either sign ranks with -inf."""
import pytest
import torch

import _serve_ref as ref
from test_gpu_evict import DEV, idx, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,budget", [([900, 400], 700), ([900, 400], 100), ([5000, 2000], 1900), ([70001], 2048)])
def test_nan_weights_rank_with_minus_infinity(idx, lens, budget):  # noqa: F811
    s = make(lens, 2, 64, 64, seed=21)
    n = min(lens)
    s["w"][:, 0, 1:n:5] = float("nan")
    s["w"][:, 0, 2:n:5] = -float("nan")
    assert s["w"].view(torch.int32)[0, 0, 2] < 0
    s["w"][:, 0, 3:n:50] = -float("inf")
    s["w"][:, 1, 1:n:9] = -float("nan")
    d = {k: t.to(DEV) for k, t in s.items()}
    ln, w, pos = idx.idx_cache_evict(d["k"], d["v"], d["table"], d["lens"], d["w"], d["pos"], d["next"], budget,
                                     recent=20, sink=3)
    torch.cuda.synchronize()
    ranked = torch.where(torch.isnan(s["w"]), -float("inf"), s["w"])
    k, v, lr, _, pr = ref.evict(s["k"], s["v"], s["table"], s["lens"], ranked, s["pos"], s["next"], budget, 20, 3)
    assert torch.equal(ln.cpu(), lr) and torch.equal(pos.cpu(), pr)
    assert torch.equal(d["k"].cpu().view(torch.int16), k.view(torch.int16))
    # the weights move with their slots, NaN as NaN
    _, _, _, wr, _ = ref.evict(s["k"], s["v"], s["table"], s["lens"], ranked, s["pos"], s["next"], budget, 20, 3)
    got = w.cpu()
    assert torch.equal(torch.where(torch.isnan(got), -float("inf"), got), wr)
