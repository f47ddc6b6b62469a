"""idx_prefix_attention with values that are not finite in keys that a row sees: they reach
that row's results and no other's."""
import math

import pytest
import torch

import _serve_ref as ref
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


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[1] > 1])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("back", [1, 2])
def test_a_later_tokens_value_that_is_not_finite(idx, shape, value, back):  # noqa: F811
    """V of one of the newest tokens: the tokens before it do not see it."""
    lens, Q, G, Hkv, D, dtype, prefix = shape
    s = make(lens, Q, G, Hkv, D, prefix, 32, dtype, seed=7, weights=D == 128)
    for b in range(0, len(lens), 2):
        put(s, "v", b, lens[b] - back, 0, value)
    got = call(idx, s)
    want = ref.attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["prefix_table"], prefix, None, s["w"])
    blind = Q - back  # tokens before the one with the value
    cut = lambda t: t[:, :blind]  # noqa: E731
    assert torch.isfinite(want[0][:, :blind]).all()
    ref.check_attention([cut(got[0]), cut(got[1])], [*map(cut, want[:4]), None], dtype, prefix + max(lens), D)
    assert not torch.isfinite(got[0][0::2, blind:, :G]).any()
    assert torch.isfinite(got[0][1::2]).all() and torch.isfinite(got[1]).all()
    if s["w"] is not None:
        for b, n in enumerate(lens):
            assert torch.isfinite(got[2][b, :, :n]).all()
