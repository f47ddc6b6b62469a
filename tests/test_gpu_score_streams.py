"""The scoring calls on a stream of their own, with the output and the workspace left to the call,
while the caller's stream is busy before it and takes memory after it."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def idx():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_indexer_tiles_gb300 as pkg
    return pkg


@pytest.mark.parametrize("name", ["idx_score_topk", "idx_score_topk_routed", "idx_score_topk_noalloc"])
def test_output_and_workspace_of_the_call(idx, name):
    inp = synth.indexer_inputs(64, 6000, 32, 128, 64, "fp8", seed=3)
    g = [getattr(inp, n).to(DEV) for n in ("q", "k", "k_scale", "w", "ks", "ke")]
    call = getattr(idx, name)
    want = call(*g, 64)
    torch.cuda.synchronize()
    a = torch.randn(4096, 4096, device=DEV)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        for _ in range(8):
            a @ a
        got = call(*g, 64, stream=stream)
        trash = [torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) for n in [1 << k for k in range(9, 25)] * 2]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del trash, got
