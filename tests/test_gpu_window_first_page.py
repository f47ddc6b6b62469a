"""idx_window_attention_mxfp4: a half of a step of keys that no row sees is filled from a page that is seen, and never from
a page of somebody else's."""
import pytest
import torch

from test_gpu_window_attention import call, check, idx, problem  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 32])
def test_any_first_page(idx, page):
    """What the pool's first page holds reaches no row that does not see it, whatever it is."""
    p = problem([100, 41, 77], [1, 1, 3], 4, 2, 64, page, "bf16", seed=2)
    p["table"][p["table"] >= 0] += 1             # page 0 is nobody's
    p["cache"] = [torch.cat([torch.full_like(c[:1], 255), c]) for c in p["cache"]]
    want = check(idx, p, 20, 3)
    for c in p["cache"]:
        c[0] = 77
    got, st = call(idx, p, window=20, sink=3)
    assert st == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("window,sink", [(1, 0), (3, 1), (16, 16), (17, 3), (30, 33), (40, 48)])
@pytest.mark.parametrize("D,dt", [(64, "fp16"), (128, "bf16")])
def test_halves_of_steps(idx, window, sink, D, dt):
    """Pages of 16 slots, so that a step of 32 keys lies in two: the older one, the newer one or both are seen."""
    lens = list(range(1, 100, 7)) + [112, 113, 128, 129]
    check(idx, problem(lens, [1] * len(lens), 4, 2, D, 16, dt, seed=window), window, sink, options={"row_split": -1})
    check(idx, problem(lens, [min(n, 5) for n in lens], 2, 2, D, 16, dt, seed=window), window, sink, options={"row_split": -1})
