"""idx_window_attention_mxfp4: calls of the tensor cores' dense path that only tiles of few rows were tested with, and which
of the ways to join splits a call takes."""
import pytest
import torch

from _cache_ref import attention, check_attention
from test_gpu_window_attention import DENSE, call, check, idx, problem  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,dt", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("window,sink", [(0, 0), (90, 0), (90, 20)])
@pytest.mark.parametrize("scale", [-0.1, -1.0, 0.0, 1e-3])
def test_factors_of_any_sign(idx, scale, window, sink, D, dt):
    p = problem([330, 100], [130, 70], 4, 2, D, 16, dt, seed=D)
    check(idx, p, window, sink, scale=scale, options=DENSE)


@pytest.mark.parametrize("window,sink", [(0, 0), (40, 3)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("scale", [None, -0.2])
def test_queries_that_are_not_finite(idx, scale, dt, window, sink):
    """Their own rows are NaN, in one row tile and in two, and no other."""
    p = problem([300, 100], [90, 20], 4, 1, 128, 32, dt, seed=3)
    bad = [(0, 1), (31, 0), (89, 3), (95, 2)]
    for n, (t, h) in enumerate(bad):
        p["q"][t, h, 5 + n] = [float("nan"), float("inf"), -float("inf"), float("nan")][n]
    got, st = call(idx, p, window=window, sink=sink, scale=scale, options=DENSE)
    assert st == 0
    rows = torch.zeros(110, 4, dtype=torch.bool)
    for t, h in bad:
        rows[t, h] = True
    assert torch.isnan(got[0][rows]).all() and torch.isnan(got[1][rows]).all()
    clean = dict(p, q=torch.where(rows[..., None], 0.0, p["q"].float()).to(p["q"].dtype))
    ref = list(attention(clean["q"], p["cache"], p["table"], p["lens"], p["q_start"], window, sink, scale))
    got = [torch.where(rows[..., None], ref[0].to(got[0].dtype), got[0]), torch.where(rows, ref[1].float(), got[1])]
    check_attention(got, ref, p["q"].dtype, 300, 128)


@pytest.mark.parametrize("path", [-1, 1])
@pytest.mark.parametrize("page", [16, 64])
def test_pages_in_the_windows_gap_need_not_exist(idx, page, path):
    p = problem([640, 400], [70, 3], 4, 2, 64, page, "fp16", seed=5)
    window, sink, options = 50, 4, {"row_split": path}
    full = check(idx, p, window, sink, options=options)
    for b, (n, new) in enumerate(((640, 70), (400, 3))):
        first = (n - new - window + 1) // page   # the oldest row's oldest page
        gone = torch.tensor([-1, -7, 1 << 30, 2 ** 31 - 1] * 20, dtype=torch.int32)
        p["table"][b, 1:first] = gone[:first - 1]
        assert first > 2
    got, st = call(idx, p, window=window, sink=sink, options=options)
    assert st == 0 and torch.equal(got[0], full[0]) and torch.equal(got[1], full[1])


@pytest.mark.parametrize("B,D,longest,launches", [(4, 64, 4096, 1), (4, 64, 8192, 2), (200, 128, 8192, 2)])
def test_both_ways_to_join_splits(idx, B, D, longest, launches):
    """Few tiles of few splits join them in clusters, in the launch itself; a second launch joins more than eight, and those
    whose blocks do not all run at once."""
    made = idx.idx_window_attention_mxfp4_plan(B, B, 1, 8, 1, D, longest, 0, 0)
    assert not made["dense"] and made["splits"] > 1 and (made["splits"] <= 8 or (B, launches) == (4, 2))
    p = problem([longest, 1, 33, 2000] * (B // 4), [1] * B, 8, 1, D, 128, "bf16", seed=B)
    before = idx.idx_launch_count()
    got, st = call(idx, p)
    assert st == 0 and idx.idx_launch_count() - before == launches
    some = torch.tensor([0, 1, 2, 3, B - 4, B - 3, B - 2, B - 1])
    ref = attention(p["q"][some], p["cache"], p["table"][some], p["lens"][some], torch.arange(9))
    check_attention([x[some] for x in got], ref, torch.bfloat16, longest, D)
