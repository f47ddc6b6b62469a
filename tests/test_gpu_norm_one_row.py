"""idx_add_rmsnorm_quant on one row of a wider tensor: its pitch leads to no other row, so it does not
matter to the row's alignment."""
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
