"""Which tokens idx_cache_append_mxfp4 writes when a request's numbers do not fit the call."""
import pytest
import torch

from _cache_ref import append, starts
from test_gpu_cache_append import cache, idx, rows, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("start", [[0, 2, 7], [0, 2, 2 ** 31 - 1], [3, 4, 9]])
def test_requests_that_end_behind_the_call(idx, start):
    """The positions of such a request's tokens are not known: none is written, and it is reported."""
    k, v = rows(6, 1, 64, "bf16", 5), rows(6, 1, 64, "bf16", 6)
    c, lens = cache(4, 1, 16, 64), torch.tensor([20, 30], dtype=torch.int32)
    table = torch.tensor([[0, 2], [3, 1]], dtype=torch.int32)
    got, st = run(idx, k.cuda(), v.cuda(), c, table, lens, torch.tensor(start, dtype=torch.int32))
    first = torch.tensor([start[0], start[1], start[1]], dtype=torch.int32)  # the second request without tokens
    assert st == 2
    for a, b in zip(got, append(k, v, c, table, lens, first)):
        assert torch.equal(a, b)
