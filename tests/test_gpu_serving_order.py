"""The serving operators on one stream, each reading what the call before it wrote.  Their
kernels may be launched while the one before them ends, so a chain of calls without any
synchronisation has to give, bit by bit, what the same calls give one at a time; and so have
graphs of them, behind copies, fills and joins of streams too."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, HKV, HQ, D, PAGE, PREFIX, SLOTS, ROWS, N = 6, 2, 16, 128, 32, 700, 256, 192, 2048


@pytest.fixture(scope="module")
def idx():
    import sparse_attention_indexer_tiles_gb300 as pkg
    return pkg


def state():
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g)
    per, pre = SLOTS // PAGE, (PREFIX + PAGE - 1) // PAGE
    pages = pre + B * per
    order = torch.randperm(pages, generator=g).int()
    d = dict(x=r(ROWS, N).bfloat16(), add=r(ROWS, N).bfloat16(), weight=r(N).bfloat16(),
             k=r(pages, HKV, PAGE, D).bfloat16(), v=r(pages, HKV, PAGE, D).bfloat16(),
             prefix=order[:pre].clone(), table=order[pre:].view(B, per).clone(),
             lens=torch.randint(150, SLOTS + 1, (B,), generator=g).int(),
             w=r(B, HKV, SLOTS).abs(),
             pos=torch.arange(SLOTS).int().expand(B, HKV, SLOTS).contiguous())
    d["next"] = d["lens"].clone()
    d = {n: t.to(DEV) for n, t in d.items()}
    e = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device=DEV)
    d.update(h=e(ROWS, N, t=torch.bfloat16), code=e(ROWS, N, t=torch.float8_e4m3fn), scale=e(ROWS),
             q=e(B, 1, HQ, D, t=torch.bfloat16), o=e(B, 1, HQ, D, t=torch.bfloat16), lse=e(B, 1, HQ),
             w2=torch.zeros(B, HKV, SLOTS, device=DEV), lens2=torch.empty_like(d["lens"]),
             ws=e(1 << 24, t=torch.uint8), x0=d["x"].clone(), q0=e(B, 1, HQ, D, t=torch.bfloat16))
    return d


def steps(idx, d, prefix, budget):
    """One layer's calls, each on the outputs of the one before."""
    def norm():
        idx.idx_add_rmsnorm_quant(d["x"], d["weight"], residual=d["add"], residual_out=d["h"],
                                  out=d["code"], scale=d["scale"])

    def norm_again():  # of the sum just written
        idx.idx_add_rmsnorm_quant(d["h"], d["weight"], residual=d["x"], residual_out=d["x"],
                                  out=d["code"], scale=d["scale"])

    def query():
        n = d["q"].numel()
        d["q"].view(-1).copy_(d["code"].view(-1)[:n].bfloat16() * (1 / 64))

    def attend():
        idx.idx_prefix_attention(d["q"], d["k"], d["v"], d["table"], d["lens"],
                                 prefix_table=d["prefix"] if prefix else None,
                                 prefix_len=PREFIX if prefix else 0, weights=d["w"],
                                 weights_out=d["w2"], out=d["o"], lse=d["lse"], ws=d["ws"])

    def attend_again():  # with the output as the query
        idx.idx_prefix_attention(d["o"], d["k"], d["v"], d["table"], d["lens"],
                                 prefix_table=d["prefix"] if prefix else None,
                                 prefix_len=PREFIX if prefix else 0, weights=d["w2"],
                                 weights_out=d["w"], out=d["q"], lse=d["lse"], ws=d["ws"])

    def evict():
        idx.idx_cache_evict(d["k"], d["v"], d["table"], d["lens"], d["w"], d["pos"], d["next"],
                            budget, recent=16, sink=4, max_len=SLOTS, lens_out=d["lens2"],
                            weights_out=d["w"], positions_out=d["pos"], ws=d["ws"])

    def feed():  # the next layer's input
        d["add"].view(-1)[:d["q"].numel()].copy_(d["q"].view(-1))
        d["lens"].copy_(d["lens2"])

    return [norm, norm_again, query, attend, attend_again, evict, feed]


def run(fs, sync):
    for f in fs:
        f()
        if sync:
            torch.cuda.synchronize()


NAMES = ("x", "h", "q", "o", "lse", "w", "w2", "pos", "lens", "k", "v", "scale")


@pytest.mark.parametrize("prefix", [True, False])
def test_a_chain_of_calls(idx, prefix):
    want, got = state(), state()
    for layer in range(4):
        run(steps(idx, want, prefix, 140 - 20 * layer), True)
    torch.cuda.synchronize()
    for layer in range(4):
        run(steps(idx, got, prefix, 140 - 20 * layer), False)
    torch.cuda.synchronize()
    for n in NAMES:
        assert torch.equal(want[n], got[n]), n
    assert torch.isfinite(want["o"]).all()


@pytest.mark.parametrize("before", ["nothing", "copy", "fill", "join", "call"])
def test_graphs_behind_other_work(idx, before):
    """Each operator as the first one behind a copy, a fill, a join of two streams or another
    operator, captured."""
    want, got = state(), state()
    run(steps(idx, want, True, 140), True)
    warm = state()
    run(steps(idx, warm, True, 140), True)
    side = torch.cuda.Stream()
    other = torch.empty(1 << 22, device=DEV)

    def work(d, f):
        main = torch.cuda.current_stream()
        if before == "copy":
            d["q0"].copy_(d["q"])
            d["x0"].copy_(d["x"])
        elif before == "fill":
            other.zero_()
        elif before == "join":
            side.wait_stream(main)
            with torch.cuda.stream(side):
                other.fill_(1.0)
            d["x0"].copy_(d["x"])
            main.wait_stream(side)
        elif before == "call":
            idx.idx_add_rmsnorm_quant(d["x0"], d["weight"], out=torch.empty_like(d["code"]),
                                      scale=torch.empty_like(d["scale"]))
        f()

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for f in steps(idx, got, True, 140):
            work(got, f)
    g.replay()
    torch.cuda.synchronize()
    for n in NAMES:
        assert torch.equal(want[n], got[n]), n
