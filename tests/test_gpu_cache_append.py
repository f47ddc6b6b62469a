"""idx_cache_append_mxfp4, bit for bit: the blocks' scales and codes, where they go, and what is left alone."""
import pytest
import torch

from _cache_ref import append, quantise, starts

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def idx():
    import sparse_attention_indexer_tiles_gb300 as pkg
    pkg.load()
    return pkg


def cache(pages, heads, page, D, fill=0x5a):
    return [torch.full((pages, heads, page, D // n), fill, dtype=torch.uint8) for n in (2, 32, 2, 32)]


def run(idx, k, v, c, table, lens, q_start=None):
    stats = idx.Stats()
    dev = [x.cuda() for x in c]
    idx.idx_cache_append_mxfp4(k, v, *dev, table.cuda(), lens.cuda(),
                               q_start=None if q_start is None else q_start.cuda(), stats=stats)
    torch.cuda.synchronize()
    return [x.cpu() for x in dev], stats.read()["status"]


def rows(T, heads, D, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, heads, D, generator=g) * torch.exp(3 * torch.randn(T, heads, D // 32, generator=g)).repeat_interleave(32, 2)
    return x.to(TYPES[dt])


@pytest.mark.parametrize("D,page,heads,dt", [(64, 16, 1, "bf16"), (128, 64, 3, "fp16"), (128, 128, 8, "bf16"), (64, 32, 5, "fp16")])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([40, 17, 64], [40, 1, 5]), ([100, 0, 33, 128], [3, 0, 33, 20])])
def test_against_the_definition(idx, D, page, heads, dt, lens, new):
    width = -(-max(lens) // page)
    table = torch.randperm(len(lens) * width + 1).to(torch.int32)[:len(lens) * width].view(len(lens), width)
    T = sum(new)
    k, v = rows(T, heads, D, dt, 1), rows(T, heads, D, dt, 2)
    c, lens, start = cache(len(table) * width + 1, heads, page, D), torch.tensor(lens, dtype=torch.int32), starts(new)
    got, st = run(idx, k.cuda(), v.cuda(), c, table, lens, start)
    assert st == 0
    for a, b in zip(got, append(k, v, c, table, lens, start)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_every_rounding(idx, dt):
    """Blocks around each border between two codes, at every power of two that the type has."""
    base = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0])
    u = torch.finfo(TYPES[dt]).eps
    block = torch.cat([base, base * (1 + u) * torch.tensor([1.0, -1.0] * 8)])
    block[16] = -0.0
    powers = range(-14, 14) if dt == "fp16" else list(range(-126, -100)) + list(range(-9, 9)) + list(range(110, 125))
    blocks = [block * 2.0 ** p for p in powers] + [(block - 1e-3) * 2.0 ** p for p in powers]
    x = torch.stack(blocks).to(TYPES[dt])
    T = -(-len(x) // 2)
    x = torch.cat([x, x])[:2 * T].reshape(T, 1, 64)
    c, table = cache(-(-T // 16), 1, 16, 64), torch.arange(-(-T // 16), dtype=torch.int32)[None]
    got, st = run(idx, x.cuda(), (-x).cuda(), c, table, torch.tensor([T], dtype=torch.int32))
    assert st == 0
    for i, y in enumerate((x, -x)):
        codes, sf = quantise(y)
        assert torch.equal(got[2 * i].transpose(1, 2).reshape(-1, 1, 32)[:T], codes)
        assert torch.equal(got[2 * i + 1].transpose(1, 2).reshape(-1, 1, 2)[:T], sf)


def test_blocks_that_are_not_finite_zero_or_tiny(idx):
    x = torch.randn(6, 1, 128).to(torch.bfloat16)
    x[0, 0, 5], x[1, 0, 40], x[2, 0, 70] = float("nan"), float("inf"), float("-inf")
    x[3] = 0
    x[4] = -0.0
    x[5] = 2.0 ** -133
    c, table = cache(1, 1, 16, 128), torch.zeros(1, 1, dtype=torch.int32)
    got, st = run(idx, x.cuda(), x.cuda(), c, table, torch.tensor([6], dtype=torch.int32))
    codes, sf = quantise(x)
    assert st == 0 and torch.equal(got[0][0, 0, :6], codes[:, 0]) and torch.equal(got[1][0, 0, :6], sf[:, 0])
    assert sf[0, 0].tolist()[0] == 255 and sf[3, 0].tolist() == [127] * 4


@pytest.mark.parametrize("offset,extra", [(0, 0), (8, 8), (1, 0), (0, 3), (5, 7)])
def test_slices_of_a_projection(idx, offset, extra):
    """At any element: rows on 16-byte boundaries take wide loads, others single ones."""
    T, heads, D = 9, 2, 64
    k, v = rows(T, heads, D, "bf16", 3), rows(T, heads, D, "bf16", 4)
    wide = torch.zeros(T, 2 * heads * D + offset + extra, dtype=torch.bfloat16)
    n = heads * D
    wide[:, offset:offset + n], wide[:, offset + n:offset + 2 * n] = k.flatten(1), v.flatten(1)
    wide = wide.cuda()
    parts = [wide[:, offset + i * n:offset + (i + 1) * n].unflatten(1, (heads, D)) for i in range(2)]
    c, table, lens = cache(3, heads, 16, D), torch.tensor([[2, 0]], dtype=torch.int32), torch.tensor([20], dtype=torch.int32)
    got, st = run(idx, *parts, c, table, lens)
    assert st == 0
    for a, b in zip(got, append(k, v, c, table, lens, starts([T]))):
        assert torch.equal(a, b)


def test_tokens_that_are_not_kept(idx):
    """Negative pages, tokens behind the last request, positions and pages that do not exist."""
    k, v = rows(12, 1, 64, "fp16", 5), rows(12, 1, 64, "fp16", 6)
    c, lens, start = cache(4, 1, 16, 64), torch.tensor([20, 9], dtype=torch.int32), starts([8, 2])
    table = torch.tensor([[-1, 2], [3, -5]], dtype=torch.int32)
    got, st = run(idx, k.cuda(), v.cuda(), c, table, lens, start)
    assert st == 0
    for a, b in zip(got, append(k, v, c, table, lens, start)):
        assert torch.equal(a, b)
    for bad_lens, bad_table in (([20, 1], table), ([20, 33], table), ([20, -4], table), ([20, 9], torch.tensor([[-1, 2], [4, 0]]))):
        got, st = run(idx, k.cuda(), v.cuda(), c, bad_table.to(torch.int32), torch.tensor(bad_lens, dtype=torch.int32), start)
        assert st == 2
        assert (got[0][1] == 0x5a).all() and torch.equal(got[0][2], append(k, v, c, table, lens, start)[0][2])


@pytest.mark.parametrize("B", [1, 2, 31, 32, 33, 63, 64, 65, 1000, 1025, 3000])
def test_the_request_of_a_token(idx, B):
    """Any number of requests, empty ones among them: every token's row holds its number."""
    g = torch.Generator().manual_seed(B)
    new = torch.randint(0, 4, (B,), generator=g).tolist()
    if sum(new) == 0:
        new[0] = 1
    T = sum(new)
    k = torch.zeros(T, 1, 64)
    t = torch.arange(T)
    for i in range(16):
        k[:, 0, i] = (t >> i & 1).float()
    k[:, 0, 31] = 4.0
    c, table = cache(B, 1, 16, 64, 0), torch.randperm(B, generator=g).to(torch.int32)[:, None]
    got, st = run(idx, k.half().cuda(), k.half().cuda(), c, table, torch.tensor(new, dtype=torch.int32), starts(new))
    assert st == 0
    for a, b in zip(got, append(k, k, c, table, torch.tensor(new), starts(new))):
        assert torch.equal(a, b)
