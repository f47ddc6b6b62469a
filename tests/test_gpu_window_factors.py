"""idx_window_attention_mxfp4 with factors next to the largest number."""
import pytest

from test_gpu_window_attention import check, idx, problem  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path", [-1, 1])
@pytest.mark.parametrize("scale", [3e38, -3e38])
def test_factors_next_to_the_largest_number(idx, scale, path):
    """A logit of 0 stays 0 under any factor."""
    p = problem([200], [70], 4, 1, 64, 16, "bf16", seed=1)
    p["q"].zero_()
    check(idx, p, scale=scale, options={"row_split": path})
