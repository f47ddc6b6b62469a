"""idx_add_rmsnorm_quant on slices of wider tensors: one row, whose pitch leads to no other row and does
not matter to its alignment, and fp32 rows, which are on 16-byte boundaries at a pitch of four columns."""
import pytest
import torch

import _serve_ref as ref
from test_gpu_norm_quant import BF16, DEV, FP32, idx, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cols,wide", [(128, 259), (256, 261), (4096, 4099)])
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("rows", [1, 3])
def test_a_row_of_an_odd_pitch(idx, dtype, cols, wide, group, rows):  # noqa: F811
    x, _, _ = inputs(rows, wide, dtype, False, seed=wide)
    _, w, _ = inputs(1, cols, dtype, False, seed=cols)
    d = x.to(DEV)[:, :cols]
    if rows > 1 and group:  # the other rows are off their 16-byte boundaries
        with pytest.raises(idx.IdxError) as e:
            idx.idx_add_rmsnorm_quant(d, w.to(DEV), group=group)
        assert e.value.code == 2
        return
    out, scale = idx.idx_add_rmsnorm_quant(d, w.to(DEV), group=group)
    torch.cuda.synchronize()
    ref.check_norm(out.cpu(), scale.cpu(), x[:, :cols], w, group=group)


@pytest.mark.parametrize("cols,wide,start", [(128, 132, 0), (128, 300, 4), (256, 268, 12), (4096, 4100, 4)])
@pytest.mark.parametrize("group", [0, 64])
def test_fp32_rows_on_16_byte_boundaries(idx, cols, wide, start, group):  # noqa: F811
    """Four fp32 columns are 16 bytes: a pitch or a start of an odd multiple of four is enough."""
    x, _, _ = inputs(9, wide, FP32, False, seed=wide)
    _, w, _ = inputs(1, cols, FP32, False, seed=cols)
    out, scale = idx.idx_add_rmsnorm_quant(x.to(DEV)[:, start:start + cols], w.to(DEV), group=group)
    torch.cuda.synchronize()
    ref.check_norm(out.cpu(), scale.cpu(), x[:, start:start + cols], w, group=group)
