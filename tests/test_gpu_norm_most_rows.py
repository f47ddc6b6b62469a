"""idx_add_rmsnorm_quant on as many rows as an int holds: their count rounded up to a block's rows
does not fit one."""
import pytest
import torch

from test_gpu_norm_quant import BF16, DEV, idx  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 8])
def test_rows_up_to_the_largest_int(idx, rows):  # noqa: F811
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB")
    x = torch.full((rows, 1), 2.0, dtype=BF16, device=DEV)
    x[-1], x[rows // 2] = -3.0, 0.0
    out, scale = idx.idx_add_rmsnorm_quant(x, torch.full((1,), 4.0, dtype=BF16, device=DEV), eps=0.25)
    torch.cuda.synchronize()
    for row, h in ((0, 2.0), (rows // 2, 0.0), (rows // 2 + 1, 2.0), (rows - 2, 2.0), (rows - 1, -3.0)):
        y = 4 * h / (h * h + 0.25) ** 0.5
        assert float(out[row].float()) == (448 if h > 0 else -448 if h < 0 else 0)
        assert abs(float(scale[row]) - max(abs(y) / 448, 2.0 ** -100)) <= 2.0 ** -18 * abs(y) / 448 + 2.0 ** -100
    del x, out, scale
    torch.cuda.empty_cache()
