"""The private parts of idx_prefix_attention on the tensor cores' dense path, at shapes for which the
plan takes it (asked of the plan, so that another plan shows here), and the early end of its kernel."""
import pytest
import torch

from test_gpu_prefix_attention import BF16, DEV, FP16, call, check, idx, make  # noqa: F401

pytestmark = pytest.mark.gpu


def plan(idx, s):  # noqa: F811
    B, Q, Hq, D = s["q"].shape
    most = s["table"].shape[1] * s["k"].shape[2]
    return idx.idx_prefix_attention_plan(B, Q, Hq, s["k"].shape[1], D, s["prefix_len"], most, s["w"] is not None)


def dense(idx, s, tiles):  # noqa: F811
    """Is the path taken, with at least `tiles` key tiles a part?"""
    p = plan(idx, s)
    assert p["private_dense"], p
    assert p["private_keys"] >= tiles * (80 if s["q"].shape[3] == 128 else 128), p


def lengths(B, Q, most):
    """The longest first, then ones around the tiles' ends and below the number of tokens."""
    some = [most // 2, 1, 0, Q - 1, Q, 80, 81, 127, 129, most - 1, most // 3, 161, 640]
    return ([most] + [min(n, most) for n in some] * 3)[:B]


# B, Q, G, Hkv, prefix, longest: one row tile per request (its even and odd key tiles run apart), two,
# three, and seven tokens of 16 heads
SHAPES = [(1, 4, 8, 8, 64, 20000), (6, 5, 7, 4, 50, 6000), (2, 3, 40, 2, 64, 30000), (8, 16, 16, 1, 0, 4000),
          (4, 2, 128, 1, 0, 5000), (12, 7, 16, 4, 0, 2000), (3, 7, 40, 2, 0, 4000), (30, 16, 16, 2, 40, 700)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("D,dtype,weights", [(128, BF16, True), (128, FP16, False), (64, FP16, False), (64, BF16, False)])
def test_against_64_bits(idx, shape, D, dtype, weights):  # noqa: F811
    B, Q, G, Hkv, prefix, most = shape
    s = make(lengths(B, Q, most), Q, G, Hkv, D, prefix, 64, dtype, seed=B + Q, weights=weights)
    dense(idx, s, 3)
    check(idx, s)


@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("D,weights", [(128, True), (64, False)])
def test_pages_and_a_negative_scale(idx, page, D, weights):  # noqa: F811
    s = make(lengths(8, 16, 4000), 16, 16, 1, D, 0, page, BF16, seed=page, weights=weights)
    dense(idx, s, 4)
    check(idx, s, scale=-0.07)
    s = make([20000], 4, 8, 8, D, 64, page, FP16, seed=page + 1, weights=weights)
    dense(idx, s, 6)
    check(idx, s, scale=-0.05)


@pytest.mark.parametrize("D,weights", [(128, True), (64, False)])
def test_rising_logits(idx, D, weights):  # noqa: F811
    """Every tile brings a larger maximum."""
    s = make([4000] * 8, 16, 16, 1, D, 0, 64, BF16, seed=3, weights=weights)
    dense(idx, s, 4)
    s["q"][:] = 0
    s["q"][..., 0] = 4.0
    j = torch.arange(4000)
    for b in range(8):
        s["k"][s["table"][b].long()[j // 64], :, j % 64, 0] = (j.float() / 8).to(BF16)[:, None]
    check(idx, s)


@pytest.mark.parametrize("shape", [(1, 4, 8, 8, 0, 20000), (8, 16, 16, 1, 0, 4000), (2, 3, 40, 2, 60000, 30000)])
@pytest.mark.parametrize("D", [64, 128])
def test_a_wait_that_runs_out_ends_the_kernel(idx, shape, D):  # noqa: F811
    """Key tile 1 of every part is withheld: the kernel gives up, raises the timeout bit and leaves
    nothing in flight; the next call gives what the one before gave."""
    B, Q, G, Hkv, prefix, most = shape
    s = make([most] * B, Q, G, Hkv, D, prefix, 64, BF16, seed=4, weights=False)
    dense(idx, s, 2)
    want = call(idx, s)
    stats = idx.Stats(torch.device(DEV))
    call(idx, s, stats, options=idx.Options(test_stall_us=2000))
    assert stats.read()["status"] & 1
    assert all(torch.equal(x, y) for x, y in zip(call(idx, s), want))


def test_the_plan_refuses_what_the_call_refuses(idx):  # noqa: F811
    for sizes in ((1, 17, 8, 2, 128, 0, 64), (1, 1, 258, 2, 128, 0, 64), (1, 1, 8, 2, 96, 0, 64)):
        with pytest.raises(idx.IdxError) as e:
            idx.idx_prefix_attention_plan(*sizes, False)
        assert e.value.code == 4
