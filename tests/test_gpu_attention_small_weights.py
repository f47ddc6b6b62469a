"""Softmax weights far below the largest one: they are rounded to the tensors' type for the second
product, and fp16 has few bits left below 2^-14.  Every sixteenth key holds a large weight and has V =
0; the output is what the keys between them, of about 2^-19 of that weight, add up to."""
import math

import pytest
import torch

from test_gpu_prefix_attention import BF16, FP16, check, idx, make  # noqa: F401
from test_gpu_attention_dense import plan

pytestmark = pytest.mark.gpu


def tails(s, b, n):
    """The slots 0 .. n - 1 of request b (of the prefix when b is None)."""
    page = s["k"].shape[2]
    table = (s["prefix_table"] if b is None else s["table"][b]).long()
    j = torch.arange(n)
    s["k"][table[j // page], :, j % page] = 0
    s["v"][table[j // page], :, j % page] = 1
    j = j[::16]
    s["k"][table[j // page], :, j % page, 0] = 8.0
    s["v"][table[j // page], :, j % page] = 0


@pytest.mark.parametrize("part", ["prefix", "private", "dense"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("steps", [24.5, 21.5, 27.5])
def test_many_small_weights(idx, part, D, dtype, steps):  # noqa: F811
    """Each of them `steps` times 2^-24 of the largest: halfway between two fp16 numbers there."""
    if part == "dense":
        s = make([4000] * 8, 16, 16, 1, D, 0, 64, dtype, seed=1, weights=False)
        assert plan(idx, s)["private_dense"]
        for b in range(8):
            tails(s, b, 4000)
        s["lens"][:] = 4000
    else:
        n = 2000
        s = make([n, n], 1, 8, 1, D, n if part == "prefix" else 0, 64, dtype, seed=1, weights=False)
        s["lens"][:] = n if part == "private" else 0
        assert part == "prefix" or not plan(idx, s)["private_dense"]
        for b in range(2):
            tails(s, None if part == "prefix" else b, n)
    s["q"][:] = 0
    s["q"][..., 0] = 2.0
    check(idx, s, scale=(24 - math.log2(steps)) / 16 * math.log(2))
