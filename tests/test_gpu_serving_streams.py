"""The serving operators on a stream of their own, with every output and the workspace left to the
call, while the caller's stream is busy before it and takes memory after it."""
import pytest
import torch

from test_gpu_serving_order import B, DEV, HQ, PREFIX, SLOTS, idx, state  # noqa: F401

pytestmark = pytest.mark.gpu


def calls(idx, d, stream):  # noqa: F811
    return {
        "norm": lambda: idx.idx_add_rmsnorm_quant(d["x"], d["weight"], residual=d["add"], stream=stream),
        "attention": lambda: idx.idx_prefix_attention(d["q"], d["k"], d["v"], d["table"], d["lens"],
                                                      prefix_table=d["prefix"], prefix_len=PREFIX, weights=d["w"],
                                                      stream=stream),
        "evict": lambda: idx.idx_cache_evict(d["k"], d["v"], d["table"], d["lens"], d["w"], d["pos"], d["next"], 100,
                                             recent=16, sink=4, max_len=SLOTS, stream=stream)}


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["norm", "attention", "evict"])
def test_outputs_and_workspace_of_the_call(idx, name, handle):  # noqa: F811
    bits = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t  # noqa: E731
    d = state()
    g = torch.Generator(device=DEV).manual_seed(1)
    d["q"].copy_(torch.randn(B, 1, HQ, 128, generator=g, device=DEV))
    want = calls(idx, d, None)[name]()
    torch.cuda.synchronize()
    want = [bits(t).clone() for t in want]
    a = torch.randn(4096, 4096, device=DEV)
    side = torch.cuda.Stream()
    for _ in range(5):
        e = state()
        e["q"].copy_(d["q"])
        torch.cuda.synchronize()
        for _ in range(8):  # some milliseconds that a fill on this stream would have to wait for
            a @ a
        got = calls(idx, e, side.cuda_stream if handle else side)[name]()
        # memory of the call's sizes, overwritten on this stream at once
        trash = [torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) for n in [1 << k for k in range(9, 25)] * 2]
        torch.cuda.synchronize()
        assert all(torch.equal(bits(x), y) for x, y in zip(got, want)), name
        del trash, got
