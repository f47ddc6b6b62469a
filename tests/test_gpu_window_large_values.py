"""idx_window_attention_mxfp4 at the top of bf16's range on the tensor cores' dense path: means of large values are as
finite as the values, however many keys add up and however far the logits run ahead of a row's first ones."""
import math

import pytest
import torch

from _cache_ref import attention, check_attention
from test_gpu_window_attention import DENSE, call, idx, problem  # noqa: F401

pytestmark = pytest.mark.gpu


def check(idx, p, window=0, sink=0, **kw):
    got, st = call(idx, p, window=window, sink=sink, options=DENSE, **kw)
    assert st == 0
    ref = attention(p["q"], p["cache"], p["table"], p["lens"], p["q_start"], window, sink, kw.get("scale"))
    # exponents next to -40 are rounded to 2^-19: 32 units more than check_attention's
    check_attention(got, ref, torch.bfloat16, int(p["lens"].max()) + 32, p["q"].shape[2])
    return got, ref


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [[40], [90], [300, 60]])
@pytest.mark.parametrize("power", [86, 87, 88, 110, 118, 121, 124, 125])
def test_many_equal_weights(idx, power, new, D):
    """One row tile and two, rows that see 1 to 700 keys, all with the same weight; signs from even to one only."""
    lens = [700, 60][:len(new)]
    p = problem(lens, new, 4, 1, D, 32, "bf16", seed=power)
    p["q"].zero_()
    p["cache"][3].fill_(127 + power)
    check(idx, p)
    p["cache"][2] &= 0x77                        # all positive: the sums grow with the keys
    check(idx, p)
    check(idx, p, 200, 30)


def ladder(step, power, seed, tokens=70, keys=400):
    """Keys whose logits rise by `step` (in powers of two) from one 80th to the next."""
    p = problem([keys], [tokens], 4, 1, 128, 16, "bf16", seed=seed)
    k, ksf = p["cache"][0], p["cache"][1]
    k.zero_()
    ksf.fill_(127)
    code = {0: 0, 1: 2, 2: 4, 3: 5, 4: 6, 5: 7}  # 0, 1, 2, 3, 4, 6
    for j in range(keys):
        k[int(p["table"][0, j // 16]), 0, j % 16, 0] = code[min(j // 80, 5)]
    p["q"].zero_()
    p["q"][..., 0] = step * math.log(2)
    p["cache"][3].fill_(127 + power)
    return p


@pytest.mark.parametrize("step", [7.8, 8.2, -7.8, 3.0, 60.0])
@pytest.mark.parametrize("power", [110, 119, 123, 125])
def test_logits_that_run_ahead(idx, power, step):
    """A maximum that grows by a little less, and a little more, than what renews a row's."""
    p = ladder(step, power, 7)
    p["cache"][2] &= 0x77
    check(idx, p, scale=1.0)


@pytest.mark.parametrize("power", [100, 121, 125])
def test_large_values_here_and_there(idx, power):
    """In some slots and blocks of columns only: the other blocks keep their bits."""
    for seed, every in ((1, 7), (2, 64), (3, 190)):
        p = ladder(6.0, -1, seed)
        p["q"] += 0.1 * torch.randn(p["q"].shape, generator=torch.Generator().manual_seed(seed)).bfloat16()
        sf = p["cache"][3]
        for j in range(seed, 400, every):
            sf[int(p["table"][0, j // 16]), 0, j % 16, 1] = 127 + power
        got, ref = check(idx, p, scale=1.0)
        assert float(got[0][..., :32].abs().max()) < 8


def test_splits_of_large_values(idx):
    p = problem([20000], [20], 16, 1, 128, 64, "bf16", seed=6)
    made = idx.idx_window_attention_mxfp4_plan(1, 20, 20, 16, 1, 128, 20000, 0, 0)
    assert made["dense"] and made["splits"] > 1
    p["cache"][3].fill_(127 + 124)
    p["cache"][2] &= 0x77
    check(idx, p)


def test_the_first_scale_that_bf16_does_not_hold(idx):
    p = problem([120], [60], 4, 1, 64, 16, "bf16", seed=13)
    page = int(p["table"][0, 5])
    p["cache"][3][page, 0, 4, 1] = 127 + 125
    check(idx, p, 30, 2)
    p["cache"][3][page, 0, 4, 1] = 127 + 126
    seen = dict(p, cache=[c.clone() for c in p["cache"]])
    seen["cache"][3][page, 0, 4, 1] = 255
    got, st = call(idx, p, window=30, sink=2, options=DENSE)
    ref = attention(p["q"], seen["cache"], p["table"], p["lens"], p["q_start"], 30, 2)
    assert st == 0 and torch.isnan(ref[1]).any() and not torch.isnan(ref[1]).all()
    check_attention(got, ref, torch.bfloat16, 120, 64)


@pytest.mark.parametrize("D", [64, 128])
def test_large_values_that_no_row_sees_change_no_bit(idx, D):
    """In the part of a unit of slots that lies outside the window, past the first tokens and behind the last slot."""
    p = problem([257, 100], [7, 33], 4, 2, D, 16, "bf16", seed=D)
    window, sink = 37, 5
    want, st = call(idx, p, window=window, sink=sink, options=DENSE)
    assert st == 0
    for x in p["cache"][1::2]:
        seen = torch.zeros(x.shape[0], 16, dtype=torch.bool)
        for b, (n, new) in enumerate(((257, 7), (100, 33))):
            for j in range(n):
                if j < sink or j > n - new - window:
                    seen[int(p["table"][b, j // 16]), j % 16] = True
        x.copy_(torch.where(seen[:, None, :, None], x, torch.tensor(247, dtype=torch.uint8)))
    got, st = call(idx, p, window=window, sink=sink, options=DENSE)
    assert st == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
