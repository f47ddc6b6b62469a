"""idx_window_attention_mxfp4 at the bottom of fp16's range: what a cache in 4 bits holds there reaches the result as fp16
holds it, on the tensor cores' dense path as on tiles of few rows."""
import math

import pytest
import torch

from _cache_ref import attention, check_attention, values
from test_gpu_window_attention import call, idx, problem  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path", [-1, 1])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lowest", [103, 99, 92, 0])
def test_small_values_of_v(idx, lowest, D, path):
    """Behind a window of 1 a row's result is the V of its own slot, its weight off by d <= 2^-11 + 2^-20 (half a step of
    fp16, and the sum).  The dense path takes V in fp16, rounded once, ties to even: where that is k 2^-24, k <= 24, the
    result is nearest to the same step, so equal.  Tiles of few rows take v itself: v (1 + d) is rounded, by half a step
    of 2^-24 or of fp16 at most (a v between two steps may go to either)."""
    T, G = 90, 4
    p = problem([T], [T], G, 2, D, 16, "fp16", seed=D + lowest)
    g = torch.Generator().manual_seed(lowest)
    sf = p["cache"][3]
    sf.copy_(torch.randint(lowest, 106 if lowest else 128, sf.shape, generator=g))
    if lowest == 0:                              # any scale up to 2^0 in one block and another
        sf[..., 0] = torch.randint(97, 106, sf[..., 0].shape, generator=g)
    got, st = call(idx, p, window=1, options={"row_split": path})
    at = torch.arange(T)
    ids = p["table"][0].long()[at // 16]
    v = values(p["cache"][2][ids, :, at % 16], sf[ids, :, at % 16])
    want = v.to(torch.float16)                   # rounded once, ties to even
    assert st == 0
    if path == 1 and lowest:
        assert (want.abs() * 2.0 ** 24 <= 24).all() and ((v != 0) & (want.double() == v)).any()
        assert torch.equal(got[0], want.repeat_interleave(G, 1))
    else:
        want = (want.double() if path == 1 else v).repeat_interleave(G, 1)
        assert ((got[0].double() - want).abs() <= want.abs() * (2.0 ** -10 + 2.0 ** -19) + 2.0 ** -25).all()



@pytest.mark.parametrize("path", [-1, 1])
@pytest.mark.parametrize("sf,codes", [(102, [0, 4, 6, 7]), (101, [0, 6]), (103, [0, 2, 4, 5, 6, 7]), (104, list(range(8)))])
def test_small_values_of_k(idx, sf, codes, path):
    """Only values that fp16 holds, so that the logits are the definition's."""
    p = problem([150], [70], 4, 1, 128, 16, "fp16", seed=sf)
    g = torch.Generator().manual_seed(sf)
    pick = torch.tensor([c + s for c in codes for s in (0, 8)], dtype=torch.uint8)
    shape = p["cache"][0].shape
    lo, hi = (pick[torch.randint(0, len(pick), shape, generator=g)] for _ in range(2))
    p["cache"][0].copy_(lo | hi << 4)
    p["cache"][1].fill_(sf)
    p["q"] = (p["q"].float() * 256).half()
    scale = 2.0 ** 11
    got, st = call(idx, p, scale=scale, options={"row_split": path})
    ref = attention(p["q"], p["cache"], p["table"], p["lens"], p["q_start"], scale=scale)
    assert float(ref[1].max() - ref[1].min()) > 0.05 and not math.isnan(float(ref[1].sum()))
    assert float((ref[1] - torch.log(torch.arange(81, 151).double())[:, None]).abs().max()) > 0.1  # the logits matter
    assert st == 0
    check_attention(got, ref, torch.float16, 150, 128)
