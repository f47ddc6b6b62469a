"""idx_cache_evict against plain lists, entry for entry: which slots stay, which hole
takes which slot, the K and V rows, weights and positions."""
import pytest
import torch

import _serve_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def idx():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_indexer_tiles_gb300 as pkg
    return pkg


def make(lens, Hkv, D, page, seed, dtype=torch.bfloat16, pages_each=None, ties=False):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    most = pages_each or max(1, -(-max(lens) // page))
    k, v = (torch.randn(B * most + 3, Hkv, page, D, generator=g).to(dtype) for _ in range(2))
    table = torch.randperm(B * most + 3, generator=g)[:B * most].reshape(B, most).to(torch.int32)
    slots = most * page
    w = torch.exp(1.5 * torch.randn(B, Hkv, slots, generator=g))
    if ties:
        w = torch.randint(0, 3, (B, Hkv, slots), generator=g).float()
    pos = torch.stack([torch.stack([torch.randperm(slots, generator=g) for _ in range(Hkv)]) for _ in range(B)])
    return {"k": k, "v": v, "table": table, "lens": torch.tensor(lens, dtype=torch.int32), "w": w,
            "pos": pos.to(torch.int32), "next": torch.full((B,), slots, dtype=torch.int32)}


def check(idx, s, budget, recent=0, sink=0, in_place=False, max_len=0):
    d = {n: t.to(DEV) for n, t in s.items()}
    kw = dict(weights_out=d["w"], positions_out=d["pos"]) if in_place else {}
    stats = idx.Stats(torch.device(DEV))
    lens, w, pos = idx.idx_cache_evict(d["k"], d["v"], d["table"], d["lens"], d["w"], d["pos"], d["next"], budget,
                                       recent=recent, sink=sink, max_len=max_len, stats=stats, **kw)
    torch.cuda.synchronize()
    assert stats.read()["status"] == 0
    k, v, lens_r, w_r, pos_r = ref.evict(s["k"], s["v"], s["table"], s["lens"], s["w"], s["pos"], s["next"],
                                         budget, recent, sink)
    assert torch.equal(lens.cpu(), lens_r)
    for b, n in enumerate(lens_r.tolist()):
        assert torch.equal(w.cpu()[b, :, :n], w_r[b, :, :n]), "weights"
        assert torch.equal(pos.cpu()[b, :, :n], pos_r[b, :, :n]), "positions"
    if not in_place:
        assert torch.equal(w.cpu(), w_r) and torch.equal(pos.cpu(), pos_r)
    bits = lambda t: t.view(torch.int16)  # noqa: E731
    assert torch.equal(bits(d["k"].cpu()), bits(k)) and torch.equal(bits(d["v"].cpu()), bits(v))


@pytest.mark.parametrize("lens,budget,recent,sink", [
    ([1], 1, 0, 0), ([0, 1, 2, 3], 1, 0, 0), ([33, 32, 31, 64], 32, 4, 2), ([100], 99, 10, 4), ([65, 40], 64, 64, 0),
    ([1000, 20, 999, 0], 500, 100, 3), ([1025, 1024, 1023], 1024, 0, 0), ([2049, 2048], 2048, 128, 4),
    ([5000, 3], 7, 3, 4), ([4097, 8192], 4096, 256, 4)])
@pytest.mark.parametrize("page,D", [(16, 64), (64, 128)])
def test_lengths_and_budgets(idx, lens, budget, recent, sink, page, D):
    check(idx, make(lens, 2, D, page, seed=sum(lens) + page), budget, recent, sink)


@pytest.mark.parametrize("n,budget", [(40000, 2048), (40000, 30000), (70001, 512), (70001, 69000), (260000, 2048),
                                      (410000, 4096)])
def test_long_rows(idx, n, budget):
    check(idx, make([n, n // 3], 1, 64, 128, seed=n), budget, 32, 4)


def test_many_requests(idx):
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 700, (200,), generator=g).tolist()
    check(idx, make(lens, 3, 64, 32, seed=5), 250, 40, 2)


@pytest.mark.parametrize("budget", [1, 50, 777, 1500])
def test_ties_go_to_the_lower_slot(idx, budget):
    check(idx, make([3000, 1600, 2000], 2, 64, 32, seed=6, ties=True), budget)


def test_all_weights_equal(idx):
    s = make([4000], 2, 64, 64, seed=7)
    s["w"].fill_(0.25)
    check(idx, s, 1000)
    s["w"].zero_()
    check(idx, s, 1000, 500, 4)


def test_special_weights(idx):
    """Zeros of both signs tie; infinities and denormals keep the float order."""
    s = make([900], 1, 64, 64, seed=8)
    s["w"][0, 0, :900:7] = -0.0
    s["w"][0, 0, 3:900:7] = 0.0
    s["w"][0, 0, 5:900:31] = float("inf")
    s["w"][0, 0, 6:900:29] = 1e-42
    for budget in (10, 40, 600, 700, 850):
        check(idx, s, budget, 8, 2)


@pytest.mark.parametrize("budget,recent,sink", [(64, 60, 4), (64, 0, 64), (64, 64, 0), (300, 290, 1)])
def test_protected_slots_fill_the_budget(idx, budget, recent, sink):
    check(idx, make([1000, 64, 2000], 2, 64, 32, seed=9), budget, recent, sink)


def test_in_place_and_repeated(idx):
    """The inputs' own arrays, then a second eviction from what the first left."""
    s = make([3000, 100, 2500], 2, 128, 64, seed=10)
    check(idx, s, 1000, 50, 4, in_place=True)
    k, v, lens, w, pos = ref.evict(s["k"], s["v"], s["table"], s["lens"], s["w"], s["pos"], s["next"], 1000, 50, 4)
    s2 = dict(s, k=k, v=v, lens=lens, w=w, pos=pos)
    check(idx, s2, 300, 50, 4, in_place=True)


def test_wider_arrays_and_bounds(idx):
    """Slots past the lengths hold anything; max_len below the table's width."""
    s = make([70, 90], 2, 64, 32, seed=11, pages_each=40)
    s["w"][:, :, 90:] = float("nan")
    s["pos"][:, :, 90:] = 1 << 30
    d = {n: t.to(DEV) for n, t in s.items()}
    lens, w, pos = idx.idx_cache_evict(d["k"], d["v"], d["table"], d["lens"], d["w"], d["pos"], d["next"], 50,
                                       max_len=90)
    torch.cuda.synchronize()
    _, _, lr, wr, pr = ref.evict(s["k"], s["v"], s["table"], s["lens"], s["w"], s["pos"], s["next"], 50, 0, 0)
    assert torch.equal(lens.cpu(), lr) and torch.equal(w.cpu(), wr) and torch.equal(pos.cpu(), pr)


def test_bad_lengths_and_pages_raise_the_range_bit(idx):
    s = make([400, 300, 200], 2, 64, 32, seed=12)
    s["table"][1, 0] = -1
    s["table"][2, 6] = 1 << 20
    d = {n: t.to(DEV) for n, t in s.items()}
    stats = idx.Stats(torch.device(DEV))
    lens, w, _ = idx.idx_cache_evict(d["k"], d["v"], d["table"], d["lens"], d["w"], d["pos"], d["next"], 100,
                                     stats=stats)
    torch.cuda.synchronize()
    assert stats.read()["status"] == 2
    _, _, lr, wr, _ = ref.evict(s["k"], s["v"], s["table"].clamp(0, 5), s["lens"], s["w"], s["pos"], s["next"],
                                100, 0, 0)
    assert torch.equal(lens.cpu(), lr) and torch.equal(w.cpu(), wr)  # the selection does not read the pages
    stats.reset()
    d["lens"] = torch.tensor([500, -5, 200], dtype=torch.int32, device=DEV)
    d["table"] = make([400, 300, 200], 2, 64, 32, seed=12)["table"].to(DEV)
    lens, _, _ = idx.idx_cache_evict(d["k"], d["v"], d["table"], d["lens"], d["w"], d["pos"], d["next"], 100,
                                     stats=stats)
    torch.cuda.synchronize()
    assert stats.read()["status"] == 2 and lens.tolist() == [100, 0, 100]


def test_graph_capture(idx):
    s = make([800, 600], 2, 64, 32, seed=13)
    d = {n: t.to(DEV) for n, t in s.items()}
    out = dict(lens_out=torch.empty_like(d["lens"]), weights_out=torch.zeros_like(d["w"]),
               positions_out=torch.full_like(d["pos"], -1),
               ws=torch.empty(idx.idx_cache_evict_workspace(2, 2, 300, 800), dtype=torch.uint8, device=DEV))
    call = lambda: idx.idx_cache_evict(d["k"], d["v"], d["table"], d["lens"], d["w"], d["pos"], d["next"], 300,  # noqa: E731
                                       max_len=800, **out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    g.replay()
    torch.cuda.synchronize()
    k, v, lr, wr, pr = ref.evict(s["k"], s["v"], s["table"], s["lens"], s["w"], s["pos"], s["next"], 300, 0, 0)
    assert torch.equal(out["lens_out"].cpu(), lr) and torch.equal(out["weights_out"].cpu(), wr)
    assert torch.equal(d["k"].cpu().view(torch.int16), k.view(torch.int16))


def test_refusals(idx):
    s = make([100, 50], 2, 64, 32, seed=14)
    d = {n: t.to(DEV) for n, t in s.items()}
    args = [d[n] for n in ("k", "v", "table", "lens", "w", "pos", "next")]
    for budget, kw, code in ((0, {}, 1), (10, dict(recent=8, sink=3), 1), (10, dict(recent=-1), 1),
                             (10, dict(max_len=1000), 1), (10, dict(lens_out=d["lens"]), 1),
                             (10, dict(ws=torch.empty(256, dtype=torch.uint8, device=DEV)), 3)):
        with pytest.raises(idx.IdxError) as e:
            idx.idx_cache_evict(*args, budget, **kw)
        assert e.value.code == code, (budget, kw)
    for at, t in ((0, d["k"].float()), (2, d["table"].long()), (3, d["lens"][:1]), (4, d["w"][:, :1]),
                  (5, d["pos"].float()), (0, d["k"].cpu())):
        with pytest.raises(ValueError):
            idx.idx_cache_evict(*[t if i == at else x for i, x in enumerate(args)], 10)
