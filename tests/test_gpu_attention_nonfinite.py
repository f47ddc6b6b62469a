"""idx_prefix_attention with values that are not finite in keys that a row sees: they reach
that row's results and no other's."""
import math

import pytest
import torch

from test_gpu_prefix_attention import BF16, FP16, call, idx, make  # noqa: F401

pytestmark = pytest.mark.gpu

# (lens, Q, G, Hkv, D, dtype, prefix): a few rows per key head, more than eight, and enough of
# them (and of requests) for the private parts' dense path; with a prefix in one or two row tiles
SHAPES = [([40, 100, 9], 1, 4, 2, 128, BF16, 0), ([40, 100, 9], 1, 4, 2, 64, FP16, 200),
          ([70, 300], 2, 16, 1, 128, BF16, 90), ([90] * 3, 4, 32, 2, 64, BF16, 1000),
          ([700, 79, 80] * 8, 16, 8, 4, 128, BF16, 0), ([300, 81, 640] * 10, 16, 16, 2, 64, FP16, 40)]


def put(s, cache, b, j, h, value):
    """Slot j of request b (of the prefix when b is None), key head h."""
    page = s[cache].shape[2]
    table = s["prefix_table"] if b is None else s["table"][b]
    s[cache][table.long()[j // page], h, j % page] = value


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("cache,value", [("k", math.nan), ("v", math.nan), ("k", math.inf)])
def test_a_private_key_that_is_not_finite(idx, shape, cache, value):  # noqa: F811
    lens, Q, G, Hkv, D, dtype, prefix = shape
    weights = D == 128  # with weights the private parts of D 64 do not take the dense path
    s = make(lens, Q, G, Hkv, D, prefix, 32, dtype, seed=5, weights=weights)
    s["q"] = s["q"].abs() + 0.5  # an infinite key: an infinite logit
    clean = call(idx, s)
    put(s, cache, 1, 5, Hkv - 1, value)
    got = call(idx, s)
    heads = torch.zeros(Hkv * G, dtype=torch.bool)
    heads[(Hkv - 1) * G:] = True
    assert not torch.isfinite(got[0][1][:, heads]).any(), "out of the rows that see the key"
    if cache == "k":
        assert not torch.isfinite(got[1][1][:, heads]).any(), "lse of the rows that see the key"
        if weights:
            assert not torch.isfinite(got[2][1, Hkv - 1, :lens[1]]).any()
    else:
        assert torch.equal(got[1], clean[1])
    for x, y in zip(got[:2], clean[:2]):
        x, y = x.clone(), y.clone()
        x[1][:, heads] = y[1][:, heads] = 0
        assert torch.equal(x, y), "the other rows"


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[6]])
@pytest.mark.parametrize("cache,value", [("k", math.nan), ("v", math.nan), ("k", math.inf)])
def test_a_prefix_key_that_is_not_finite(idx, shape, cache, value):  # noqa: F811
    lens, Q, G, Hkv, D, dtype, prefix = shape
    s = make(lens, Q, G, Hkv, D, prefix, 32, dtype, seed=6, weights=False)
    s["q"] = s["q"].abs() + 0.5
    clean = call(idx, s)
    put(s, cache, None, 33, Hkv - 1, value)
    got = call(idx, s)
    assert not torch.isfinite(got[0][:, :, (Hkv - 1) * G:]).any()
    if cache == "k":
        assert not torch.isfinite(got[1][:, :, (Hkv - 1) * G:]).any()
    for x, y in zip(got, clean):
        assert torch.equal(x[:, :, :(Hkv - 1) * G], y[:, :, :(Hkv - 1) * G])
