"""Uses of the serving operators that the other files do not have: the norm's residual_out without a
residual, and evictions in the steady state, when positions are scattered and next_pos is far above
the lengths."""
import pytest
import torch

import _serve_ref as ref
from test_gpu_evict import check, make
from test_gpu_norm_quant import BF16, DEV, FP16, FP32, idx, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("cols", [1, 100, 129, 512, 5003, 8192])
def test_residual_out_without_a_residual(idx, dtype, cols):  # noqa: F811
    """It is x; for a column slice, x without its pitch."""
    x, w, _ = inputs(37, cols + 24, dtype, False, seed=cols)
    d, w = x.to(DEV)[:, 8:8 + cols], w[:cols]
    ro = torch.full((37, cols), float("nan"), dtype=dtype, device=DEV)
    out, scale = idx.idx_add_rmsnorm_quant(d, w.to(DEV), residual_out=ro)
    bare, bare_scale = idx.idx_add_rmsnorm_quant(d, w.to(DEV))
    torch.cuda.synchronize()
    assert torch.equal(ro, d)
    assert torch.equal(out.view(torch.uint8), bare.view(torch.uint8)) and torch.equal(scale, bare_scale)
    ref.check_norm(out.cpu(), scale.cpu(), x[:, 8:8 + cols], w)


@pytest.mark.parametrize("over", [1, 2, 7, 31, 32, 33, 64, 100])
@pytest.mark.parametrize("budget,heads,D", [(256, 2, 64), (2048, 3, 128)])
def test_a_few_slots_over_the_budget_long_after_the_start(idx, over, budget, heads, D):  # noqa: F811
    """Positions are any of the 100000 so far, the newest among them in the last slots; the first
    sinks are still there.  Some requests are over by fewer, exactly at, or below the budget."""
    lens = [budget + over, budget + max(1, over // 2), budget, budget - 5, budget + over]
    s = make(lens, heads, D, 64, seed=over + budget)
    g = torch.Generator().manual_seed(over)
    s["next"][:] = 100000
    for b, n in enumerate(lens):
        for h in range(heads):
            s["pos"][b, h, :n] = torch.randperm(99000, generator=g)[:n].to(torch.int32) + 10
            s["pos"][b, h, n - over:n] = torch.arange(100000 - over, 100000, dtype=torch.int32)
            s["pos"][b, h, torch.randperm(n - over, generator=g)[:4]] = torch.arange(4, dtype=torch.int32)
    s["w"][1] = torch.randint(0, 4, s["w"][1].shape, generator=g).float()  # many ties
    check(idx, s, budget, recent=min(128, budget // 2), sink=4)
    check(idx, s, budget, recent=over, sink=0, in_place=True)
