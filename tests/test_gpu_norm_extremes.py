"""idx_add_rmsnorm_quant at fp32's ends: rows whose sum of squares leaves it, and values that are not
finite, give NaN scales and codes instead of ones that look like a row's; everything inside is right."""
import math

import pytest
import torch

import _serve_ref as ref
from test_gpu_norm_quant import BF16, FP16, FP32, idx, inputs, run  # noqa: F401

pytestmark = pytest.mark.gpu

WIDTHS = [(100, 0), (128, 128), (256, 32), (500, 0), (926, 0), (2048, 64), (5003, 0), (8192, 128), (20000, 0)]


def check(got, x, w, r, lost, group, eps):
    """The rows of `lost` are NaN (their sum is kept all the same), the others within the bounds."""
    out, scale, ro = got
    live = torch.ones(len(x), dtype=torch.bool)
    live[lost] = False
    part = lambda t, m: None if t is None else t[m]  # noqa: E731
    ref.check_norm(out.view(torch.uint8)[live].view(out.dtype), scale[live], x[live], w, part(r, live),
                   part(ro, live), eps=eps, group=group)
    assert torch.isnan(scale[lost]).all() and torch.isnan(out.float()[lost]).all()
    if ro is not None:
        want = (x[lost].double() + r[lost].double()).to(x.dtype)
        assert torch.equal(ro[lost], want)


@pytest.mark.parametrize("cols,group", WIDTHS)
@pytest.mark.parametrize("dtype,residual", [(BF16, True), (BF16, False), (FP32, True)])
def test_large_rows(idx, cols, group, dtype, residual):  # noqa: F811
    """Sums of squares just inside fp32 (2^127) and outside (2^129 and more)."""
    x, w, r = inputs(300, cols, dtype, residual, seed=cols)
    if residual:
        r[:8] = 0
    for row, total in ((0, 126.9), (3, 100.0), (4, 129.1), (5, 170.0), (299, 240.0)):
        x[row] = 2.0 ** (total / 2) / cols ** 0.5 * torch.where(x[row] < 0, -1.0, 1.0)
    x[6] = 0
    x[6, cols // 2] = 2.0 ** 63.4
    x[7, 0] = -2.0 ** 64.2
    if residual:
        r[299] = 0
    check(run(idx, x, w, r, group=group), x, w, r, [4, 5, 7, 299], group, 1e-6)


@pytest.mark.parametrize("cols,group", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_small_rows_without_eps(idx, cols, group, dtype):  # noqa: F811
    x, w, _ = inputs(300, cols, dtype, False, seed=cols)
    sign = torch.where(x < 0, -1.0, 1.0)
    for row, rms in ((0, 1e-6), (3, 1e-12), (4, 1e-17), (69, 1e-25), (70, 1e-36), (299, 0.0)):
        x[row] = rms * sign[row]
    check(run(idx, x, w, group=group, eps=0.0), x, w, None, [69, 70, 299], group, 0.0)
    check(run(idx, x, w, group=group, eps=1e-30), x, w, None, [], group, 1e-30)


@pytest.mark.parametrize("cols,group", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_values_that_are_not_finite(idx, cols, group, dtype):  # noqa: F811
    """In a row: all of it is NaN; in the weight: the scales and codes it enters.  Nothing else
    changes."""
    x, w, _ = inputs(300, cols, dtype, False, seed=cols)
    clean = run(idx, x, w, group=group)
    at = cols - 1
    x[5, at] = math.nan
    x[6, at] = math.inf
    x[200] = -math.inf
    out, scale, _ = run(idx, x, w, group=group)
    lost = [5, 6, 200]
    assert torch.isnan(scale[lost]).all() and torch.isnan(out.float()[lost]).all()
    keep = torch.ones(300, dtype=torch.bool)
    keep[lost] = False
    assert torch.equal(out.view(torch.uint8)[keep], clean[0].view(torch.uint8)[keep])
    assert torch.equal(scale[keep], clean[1][keep])
    first = at // group * group if group else 0
    w[at] = math.nan
    out, scale, _ = run(idx, x[:5], w, group=group)
    scale, codes = scale.reshape(5, -1), out.float()
    assert torch.isnan(scale[:, -1]).all() and torch.isnan(codes[:, first:]).all()
    assert torch.equal(scale[:, :-1], clean[1].reshape(300, -1)[:5, :-1])
    assert torch.equal(codes[:, :first], clean[0].float()[:5, :first])
