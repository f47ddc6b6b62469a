"""idx_prefix_attention against 64 bits: head layouts, lengths from nothing on, pages that
end inside a tile, values that are not finite in slots no row sees, and the refusals."""
import math

import pytest
import torch

import _serve_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def idx():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_indexer_tiles_gb300 as pkg
    return pkg


def make(lens, Q, G, Hkv, D, prefix, page, dtype, seed, weights=True, spare=0, qscale=2.0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    most = -(-max(lens) // page) + spare
    pp = -(-prefix // page)
    pages = pp + B * most + 2
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    s = {"q": (qscale * rand(B, Q, Hkv * G, D)).to(dtype), "k": rand(pages, Hkv, page, D).to(dtype),
         "v": rand(pages, Hkv, page, D).to(dtype), "prefix_table": ids[:pp], "prefix_len": prefix,
         "table": ids[pp:pp + B * most].reshape(B, most), "lens": torch.tensor(lens, dtype=torch.int32),
         "w": torch.rand(B, Hkv, most * page, generator=g) * 5 if weights else None}
    # slots that no row sees hold values that would spoil any sum they enter
    if prefix % page:
        s["k"][ids[pp - 1].long(), :, prefix % page:] = math.nan
        s["v"][ids[pp - 1].long(), :, prefix % page:] = math.inf
    for b, n in enumerate(lens):
        for j in range(n // page, most):
            at = s["table"][b, j].long()
            s["k"][at, :, (n % page if j == n // page else 0):] = math.inf
            s["v"][at, :, (n % page if j == n // page else 0):] = math.nan
    return s


def call(idx, s, stats=None, **kw):
    d = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in s.items()}
    got = idx.idx_prefix_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], prefix_table=d["prefix_table"],
                                   prefix_len=d["prefix_len"], weights=d["w"], stats=stats, **kw)
    torch.cuda.synchronize()
    return [t.cpu() for t in got]


def check(idx, s, scale=None, **kw):
    stats = idx.Stats(torch.device(DEV))
    if scale is not None:
        kw["scale"] = scale
    got = call(idx, s, stats, **kw)
    assert stats.read()["status"] == 0
    want = ref.attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["prefix_table"], s["prefix_len"], scale,
                         s["w"])
    ref.check_attention(got, want, s["q"].dtype, s["prefix_len"] + int(s["lens"].max()), s["q"].shape[3],
                        lens=s["lens"])
    return got


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 63, 64, 65, 127, 128, 129, 300, 1000, 2049])
@pytest.mark.parametrize("D,dtype,page", [(128, BF16, 64), (64, FP16, 16)])
def test_prefix_lengths(idx, prefix, D, dtype, page):
    check(idx, make([3, 17, 0, 40], 1, 4, 2, D, prefix, page, dtype, seed=prefix))


@pytest.mark.parametrize("lens", [[1], [0], [15, 16, 17], [63, 64, 65, 0, 1], [300, 2, 1000], [1500]])
@pytest.mark.parametrize("prefix", [0, 70])
def test_private_lengths(idx, lens, prefix):
    check(idx, make(lens, 1, 3, 2, 128, prefix, 32, BF16, seed=sum(lens)))


@pytest.mark.parametrize("G,Hkv", [(1, 1), (1, 8), (2, 4), (5, 2), (7, 1), (8, 2), (16, 1), (17, 1), (32, 2), (64, 1),
                                   (96, 1), (128, 1)])
def test_head_layouts(idx, G, Hkv):
    check(idx, make([40, 70], 1, G, Hkv, 64, 150, 16, BF16, seed=G * Hkv))


@pytest.mark.parametrize("Q", [1, 2, 3, 5, 16])
@pytest.mark.parametrize("G", [1, 4, 7])
def test_several_tokens(idx, Q, G):
    """Tokens see the ones before them; some requests are shorter than Q."""
    check(idx, make([Q + 40, Q, 2, 0, 100], Q, G, 2, 64, 33, 32, FP16, seed=Q * G))


@pytest.mark.parametrize("lens", [[400], [81, 79, 80, 400, 0, 3, 161], [129, 127, 128, 256, 1, 640]])
@pytest.mark.parametrize("Q,G,Hkv", [(16, 8, 1), (16, 16, 2), (7, 16, 1), (5, 7, 2), (16, 2, 1), (3, 40, 1), (2, 128, 1)])
@pytest.mark.parametrize("D,dtype,page,prefix", [(128, BF16, 16, 0), (64, FP16, 64, 50), (128, FP16, 128, 200)])
def test_many_rows_per_key_head(idx, lens, Q, G, Hkv, D, dtype, page, prefix):
    """Private parts on the dense path: row tiles of one request, its last tokens' masks, lengths
    around the key tiles and below the number of new tokens."""
    check(idx, make(lens, Q, G, Hkv, D, prefix, page, dtype, seed=Q * G + len(lens)))


@pytest.mark.parametrize("B,Q,G,Hkv", [(24, 16, 8, 4), (30, 16, 16, 2), (30, 7, 16, 4), (40, 5, 7, 8), (20, 3, 40, 4)])
@pytest.mark.parametrize("D,dtype,weights", [(128, BF16, True), (64, FP16, False), (64, BF16, False)])
def test_many_requests_of_many_rows(idx, B, Q, G, Hkv, D, dtype, weights):
    """Batches for which the dense path is the cheaper at either head size, their lengths around
    its key tiles and down to nothing."""
    lens = [0, 1, 3, Q - 1, Q, 15, 16, 79, 80, 81, 127, 128, 129, 159, 160, 161, 240, 300, 511, 512, 513, 640, 699]
    check(idx, make([700] + (2 * lens)[:B - 1], Q, G, Hkv, D, 40, 64, dtype, seed=B + Q, weights=weights))


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, FP16)])
def test_many_rows_over_long_private_parts(idx, D, dtype):
    """Several parts and many tiles per part, for an odd and an even number of row tiles."""
    check(idx, make([5000, 777, 2600], 4, 16, 2, D, 100, 64, dtype, seed=1))
    check(idx, make([3000, 1], 16, 16, 1, D, 0, 32, dtype, seed=2, weights=False))
    check(idx, make([20000], 4, 8, 8, D, 64, 64, dtype, seed=3), scale=-0.05)


def test_several_tokens_without_a_prefix_leave_rows_empty(idx):
    got = check(idx, make([2, 5, 0], 5, 2, 1, 64, 0, 16, BF16, seed=1))
    assert (got[1][0, :3] == -math.inf).all() and (got[0][2] == 0).all()


@pytest.mark.parametrize("B", [1, 3, 33, 70])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_batches_and_pages(idx, B, page):
    lens = [(7 * b) % 90 for b in range(B)]
    lens[0] = 90
    check(idx, make(lens, 1, 4, 1, 128, 260, page, BF16, seed=B + page))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
def test_long_prefix(idx, dtype, D):
    check(idx, make([30, 500], 1, 8, 1, D, 20000, 64, dtype, seed=D), max_len=500)


@pytest.mark.parametrize("B,Q,prefix", [(2, 1, 24000), (3, 3, 30011), (70, 1, 12000)])
@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, FP16)])
def test_many_tiles_per_part(idx, B, Q, prefix, D, dtype):
    """Eight key heads leave few parts per head, so every one has many key tiles: more than
    the ring of copies holds, for one row tile (its even and odd tiles run apart) and for two."""
    check(idx, make([5 + Q] * B, Q, 2, 8, D, prefix, 64, dtype, seed=B, weights=False))


def test_sharp_and_flat_logits(idx):
    """One key holds all the weight; all keys hold the same."""
    s = make([200, 90], 1, 4, 2, 128, 500, 64, BF16, seed=2, qscale=12.0)
    check(idx, s)
    s["q"].zero_()
    check(idx, s)
    s = make([200, 90], 1, 4, 2, 128, 500, 64, BF16, seed=2)
    check(idx, s, scale=0.37)
    check(idx, s, scale=-0.2)


def test_rising_logits(idx):
    """Every tile brings a larger maximum: the running maximum is renewed throughout."""
    s = make([600], 1, 2, 1, 64, 1500, 16, BF16, seed=3)
    s["q"][:] = 0
    s["q"][..., 0] = 4.0
    for table, n in ((s["prefix_table"], 1500), (s["table"][0], 600)):
        j = torch.arange(n)
        s["k"][table.long()[j // 16], :, j % 16, 0] = (j.float() / 8).to(BF16)[:, None]
    check(idx, s)


def test_without_weights_and_lse_given(idx):
    s = make([40, 7], 1, 4, 2, 64, 100, 16, BF16, seed=4)
    with_w = check(idx, s)
    s["w"] = None
    lse = torch.empty(2, 1, 8, device=DEV)
    got = check(idx, s, lse=lse)
    assert torch.equal(got[0], with_w[0]) and torch.equal(lse.cpu(), with_w[1])


def test_weights_in_place_keep_the_slots_past_the_length(idx):
    s = make([40, 7], 1, 4, 2, 64, 100, 16, BF16, seed=5, spare=3)
    want = check(idx, s, max_len=40)[2]
    w = s["w"].to(DEV)
    got = call(idx, dict(s, w=w), weights_out=w, max_len=40)[2]
    for b, n in enumerate((40, 7)):
        assert torch.equal(got[b, :, :n], want[b, :, :n])
        assert torch.equal(got[b, :, n:], s["w"][b, :, n:])


def test_the_same_result_twice(idx):
    s = make([400, 700, 33], 2, 4, 2, 128, 3000, 64, BF16, seed=6)
    a, b = call(idx, s), call(idx, s)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_no_requests(idx):
    s = make([4], 1, 4, 2, 64, 20, 16, BF16, seed=7)
    d = {n: t.to(DEV) for n, t in s.items() if isinstance(t, torch.Tensor)}
    out, lse = idx.idx_prefix_attention(d["q"][:0], d["k"], d["v"], d["table"][:0], d["lens"][:0],
                                        prefix_table=d["prefix_table"], prefix_len=20)
    assert out.shape == (0, 1, 8, 64) and lse.shape == (0, 1, 8)


def test_bad_pages_and_lengths_raise_the_range_bit(idx):
    s = make([100, 60, 30], 1, 4, 2, 64, 0, 16, BF16, seed=8)
    clean = call(idx, s)
    stats = idx.Stats(torch.device(DEV))
    s["table"][1, 2] = -7
    got = call(idx, s, stats)
    assert stats.read()["status"] == 2
    assert torch.equal(got[0][0], clean[0][0]) and torch.equal(got[0][2], clean[0][2])
    s["table"][1, 2] = 1 << 20
    stats.reset()
    got = call(idx, s, stats)
    assert stats.read()["status"] == 2 and torch.equal(got[0][2], clean[0][2])
    s = make([100, 60, 30], 1, 4, 2, 64, 300, 16, BF16, seed=8)
    s["prefix_table"][5] = 1 << 30
    stats.reset()
    call(idx, s, stats)
    assert stats.read()["status"] == 2
    s["prefix_table"][5] = -1
    stats.reset()
    call(idx, s, stats)
    assert stats.read()["status"] == 2
    s = make([100, 60, 30], 1, 4, 2, 64, 0, 16, BF16, seed=8, weights=False)
    stats.reset()
    clean = call(idx, s)
    s["lens"] = torch.tensor([100, 5000, -3], dtype=torch.int32)
    got = call(idx, s, stats, max_len=100)
    assert stats.read()["status"] == 2
    assert torch.equal(got[0][0], clean[0][0]) and (got[0][2] == 0).all()


def test_other_stream_and_graph(idx):
    s = make([300, 20], 1, 8, 2, 128, 700, 64, BF16, seed=9)
    want = call(idx, s)
    d = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in s.items()}
    out = dict(out=torch.empty_like(d["q"]), lse=torch.empty(2, 1, 16, device=DEV), weights_out=torch.zeros_like(d["w"]),
               ws=torch.empty(idx.idx_prefix_attention_workspace(2, 1, 16, 2, 128, 700, 300, True), dtype=torch.uint8,
                              device=DEV))
    run = lambda **kw: idx.idx_prefix_attention(d["q"], d["k"], d["v"], d["table"], d["lens"],  # noqa: E731
                                                prefix_table=d["prefix_table"], prefix_len=700, max_len=300,
                                                weights=d["w"], **out, **kw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    run(stream=st)
    st.synchronize()
    names = ("out", "lse", "weights_out")
    n0, n1 = 300, 20
    same = lambda: all(torch.equal(out[n].cpu(), w) for n, w in zip(names[:2], want)) and \
        torch.equal(out["weights_out"].cpu()[0, :, :n0], want[2][0, :, :n0]) and \
        torch.equal(out["weights_out"].cpu()[1, :, :n1], want[2][1, :, :n1])  # noqa: E731
    assert same()
    for n in names:
        out[n].zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    g.replay()
    torch.cuda.synchronize()
    assert same()


def test_offsets_past_32_bits(idx):
    """A cache of more than 2^31 elements: the last pages hold the keys."""
    free, _ = torch.cuda.mem_get_info()
    pages = (1 << 31) // (2 * 64 * 128) + 64
    if free < 4 * pages * 2 * 64 * 128 * 2:
        pytest.skip("needs 18 GB")
    s = make([100, 40], 1, 4, 2, 128, 200, 64, BF16, seed=10)
    small = s["k"].shape[0]
    big = {n: torch.zeros(pages, 2, 64, 128, dtype=BF16, device=DEV) for n in ("k", "v")}
    for n in big:
        big[n][pages - small:] = s[n].to(DEV)
    shift = pages - small
    got = idx.idx_prefix_attention(s["q"].to(DEV), big["k"], big["v"], s["table"].to(DEV) + shift, s["lens"].to(DEV),
                                   prefix_table=s["prefix_table"].to(DEV) + shift, prefix_len=200,
                                   weights=s["w"].to(DEV))
    torch.cuda.synchronize()
    want = call(idx, s)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])


def test_refusals(idx):
    s = make([40, 7], 1, 4, 2, 64, 100, 16, BF16, seed=11)
    d = {n: t.to(DEV) for n, t in s.items() if isinstance(t, torch.Tensor)}

    def run(**kw):
        a = dict(q=d["q"], k=d["k"], v=d["v"], table=d["table"], lens=d["lens"])
        opt = dict(prefix_table=d["prefix_table"], prefix_len=100, weights=d["w"])
        for n, t in kw.items():
            (a if n in a else opt)[n] = t
        return idx.idx_prefix_attention(a["q"], a["k"], a["v"], a["table"], a["lens"], **opt)

    for kw in (dict(q=d["q"].float()), dict(q=d["q"].half()), dict(table=d["table"].long()), dict(lens=d["lens"][:1]),
               dict(prefix_table=None), dict(prefix_table=d["prefix_table"][:2]), dict(weights=d["w"].half()),
               dict(weights=None, weights_out=d["w"]), dict(q=d["q"].transpose(0, 2)), dict(lens=d["lens"].cpu()),
               dict(q=d["q"][..., :32].contiguous())):
        with pytest.raises(ValueError):
            run(**kw)
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    odd = d["k"][:, :, :12].contiguous()
    for kw, code in ((dict(ws=small), 3), (dict(max_len=1000), 1), (dict(scale=math.inf), 1),
                     (dict(q=d["q"][:, :, :7].contiguous()), 1), (dict(k=odd, v=odd, prefix_len=0), 4),
                     (dict(q=d["q"].expand(2, 17, 8, 64).contiguous()), 4),
                     (dict(weights=d["w"][:, :, :20].contiguous(), max_len=40), 1)):
        with pytest.raises(idx.IdxError) as e:
            run(**kw)
        assert e.value.code == code, (kw.keys(), e.value)


@pytest.mark.parametrize("B", [3, 90])
def test_a_wait_that_runs_out_ends_the_prefix_kernel(idx, B):
    """Key tile 1 of every part of the prefix is withheld (60000 keys: several tiles a part):
    the kernel gives up, raises the timeout bit and leaves nothing in flight; the next call
    gives what the one before gave."""
    s = make([20] * B, 1, 4, 1, 128, 60000, 64, BF16, seed=12)
    want = call(idx, s)
    stats = idx.Stats(torch.device(DEV))
    call(idx, s, stats, options=idx.Options(test_stall_us=2000))
    assert stats.read()["status"] & 1
    assert all(torch.equal(x, y) for x, y in zip(call(idx, s), want))
