"""idx_cache_fork, idx_cache_resize and idx_cache_compact against plain loops: every result equal, out of place and in
place, with one CTA ranking pages and with a cluster."""
import pytest
import torch

from _cache_ref import compact, counts, fork, held, laid_out, pages_of, resize

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def idx():
    import sparse_attention_indexer_tiles_gb300 as pkg
    pkg.load()
    return pkg


def pool(B, page, hi, pages, seed, shared=0, zeros=0):
    """A table of B rows whose first `shared` pairs are forks, in a pool of `pages`."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(1, hi + 1, (B,), generator=g)
    lens[torch.rand(B, generator=g) < zeros] = 0
    for i in range(shared):
        lens[2 * i + 1] = lens[2 * i]
    width = pages_of(hi, page) + 1
    ids = torch.randperm(pages, generator=g).tolist()
    rows = []
    for i, n in enumerate(lens.tolist()):
        if i % 2 and i < 2 * shared:
            rows.append(list(rows[-1]))
        else:
            rows.append([ids.pop() for _ in range(pages_of(n, page))])
    table = laid_out(rows, torch.zeros(B, width, dtype=torch.int32))
    return table, lens.to(torch.int32), counts(rows, pages)


def arrays(pages, seed, sizes=((4, 64), (3, 16))):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, 256, (pages, *s), generator=g, dtype=torch.uint8) for s in sizes]


def outputs(in_place, refs, table, lens):
    if in_place:
        return dict(refs_out=refs, table_out=table, lens_out=lens)
    return dict(refs_out=torch.full_like(refs, 99), table_out=torch.full_like(table, -1), lens_out=torch.full_like(lens, 99))


def used(table, lens, page):
    return held(table.cpu(), lens.cpu(), page)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,hi,page", [(1, 5, 16), (4, 100, 16), (37, 700, 32), (300, 5000, 64), (5000, 40, 16)])
def test_fork(idx, B, hi, page, in_place):
    pages = B * pages_of(hi, page) + 7
    table, lens, refs = pool(B, page, hi, pages, B, shared=B // 3, zeros=0.1)
    g = torch.Generator().manual_seed(B)
    parent = torch.randint(-1, B, (B,), generator=g).to(torch.int32)
    parent[::3] = torch.arange(B, dtype=torch.int32)[::3]
    rows, new = fork(table, lens, parent, page)
    d = [x.cuda() for x in (refs, table, lens)]
    stats = idx.Stats()
    r, t, n = idx.idx_cache_fork(*d, parent.cuda(), page_size=page, stats=stats, **outputs(in_place, *d))
    assert stats.read()["status"] == 0
    assert torch.equal(n.cpu(), new) and used(t, n, page) == rows
    assert torch.equal(r.cpu(), counts(rows, pages))
    if not in_place:
        assert torch.equal(t.cpu(), laid_out(rows, table))
        assert all(torch.equal(a.cpu(), b) for a, b in zip(d, (refs, table, lens)))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,width,pages", [(32, 64, 4096), (33, 64, 4096), (32, 65, 4096), (32, 64, 4097),
                                           (33, 512, 16384), (32, 1, 40)])
def test_fork_at_the_limits_of_one_launch(idx, B, width, pages, in_place):
    g = torch.Generator().manual_seed(B + width + pages)
    lens = torch.randint(0, 16 * min(width, pages // B) + 1, (B,), generator=g)
    lens[0] = 16 * min(width, pages // B)
    ids = torch.randperm(pages, generator=g).tolist()
    table = laid_out([[ids.pop() for _ in range(pages_of(n, 16))] for n in lens.tolist()],
                     torch.zeros(B, width, dtype=torch.int32))
    lens = lens.to(torch.int32)
    refs = counts(held(table, lens, 16), pages)
    parent = torch.randint(-1, B, (B,), generator=g).to(torch.int32)
    parent[B // 2:B // 2 + 5] = 0
    rows, new = fork(table, lens, parent, 16)
    d = [x.cuda() for x in (refs, table, lens)]
    stats = idx.Stats()
    r, t, n = idx.idx_cache_fork(*d, parent.cuda(), page_size=16, stats=stats, **outputs(in_place, *d))
    assert stats.read()["status"] == 0
    assert torch.equal(n.cpu(), new) and used(t, n, 16) == rows and torch.equal(r.cpu(), counts(rows, pages))
    if not in_place:
        assert all(torch.equal(a.cpu(), b) for a, b in zip(d, (refs, table, lens)))


def test_fork_reports_what_it_cannot_follow(idx):
    table, lens, refs = pool(4, 16, 60, 40, 1)
    parent = torch.tensor([4, -2, 1, 0], dtype=torch.int32)
    stats = idx.Stats()
    r, t, n = idx.idx_cache_fork(refs.cuda(), table.cuda(), lens.cuda(), parent.cuda(), page_size=16, stats=stats)
    rows, new = fork(table, lens, torch.tensor([0, 1, 1, 0]), 16)
    assert stats.read()["status"] == 2 and used(t, n, 16) == rows and torch.equal(r.cpu(), counts(rows, 40))
    bad = lens.clone()
    bad[0], bad[1] = -1, 16 * table.shape[1] + 1
    stats = idx.Stats()
    r, t, n = idx.idx_cache_fork(refs.cuda(), table.cuda(), bad.cuda(), torch.tensor([0, 0, 1, 3], dtype=torch.int32).cuda(),
                                 page_size=16, stats=stats)
    assert stats.read()["status"] == 2 and n.tolist() == [0, 0, 0, int(lens[3])]
    wild = table.clone()
    wild[2, 0] = 1000
    stats = idx.Stats()
    r, t, n = idx.idx_cache_fork(refs.cuda(), wild.cuda(), lens.cuda(), torch.tensor([0, 1, 2, 2], dtype=torch.int32).cuda(),
                                 page_size=16, stats=stats)
    assert stats.read()["status"] == 2 and int(t[3, 0]) == 1000


def check_resize(idx, table, lens, refs, new, page, in_place, seed=0, caches=None):
    pages = refs.numel()
    caches = arrays(pages, seed) if caches is None else caches
    want, rows, served, enough = resize(caches, table, lens, new, page, pages)
    d = [x.cuda() for x in (refs, table, lens)]
    c = [x.cuda() for x in caches]
    stats = idx.Stats()
    r, t, n = idx.idx_cache_resize(c, *d, new.cuda(), page_size=page, stats=stats, **outputs(in_place, *d))
    assert stats.read()["status"] == (0 if enough else 8)
    assert torch.equal(n.cpu(), served)
    assert used(t, n, page) == rows
    assert torch.equal(r.cpu().clamp_min(0), counts(rows, pages))
    for a, b in zip(c, want):
        assert torch.equal(a.cpu(), b)
    if not in_place:
        assert torch.equal(t.cpu(), laid_out(rows, table))
        assert all(torch.equal(a.cpu(), b) for a, b in zip(d, (refs, table, lens)))
    return r, t, n, c


def lengths(lens, kind, hi, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "step":
        return lens + 1
    if kind == "ends":
        return lens * (torch.rand(lens.shape, generator=g) < 0.5)
    return torch.randint(0, hi + 1, lens.shape, generator=g).to(torch.int32)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["step", "ends", "any"])
@pytest.mark.parametrize("B,hi,page,spare", [(1, 10, 16, 3), (5, 90, 16, 40), (64, 400, 32, 500), (700, 300, 16, 5000),
                                             (1100, 100, 16, 20000)])
def test_resize(idx, B, hi, page, spare, kind, in_place):
    pages = B * pages_of(hi, page) + spare
    table, lens, refs = pool(B, page, hi, pages, B, shared=B // 3, zeros=0.1)
    check_resize(idx, table, lens, refs, lengths(lens, kind, hi, B).to(torch.int32), page, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("left", [0, 1, 5, 30, 31, 32])
def test_resize_when_the_pages_do_not_suffice(idx, left, in_place):
    """All rows grow and a third of them copies: rows are served in their order, the rest is left."""
    B, page, hi = 40, 16, 50
    table, lens, refs = pool(B, page, hi, B * 4 + 10, 9, shared=12)
    free = (refs == 0).nonzero()[:, 0]
    refs[free[left:]] = 1                        # held by another table
    caches = arrays(refs.numel(), 1)
    new = lens + 17
    held_by_others = refs - counts(held(table, lens, page), refs.numel())
    d = [x.cuda() for x in (refs, table, lens)]
    c = [x.cuda() for x in caches]
    stats = idx.Stats()
    r, t, n = idx.idx_cache_resize(c, *d, new.cuda(), page_size=page, stats=stats, **outputs(in_place, *d))
    # the same without the pages that others hold: a pool of what is left
    keep = {p: i for i, p in enumerate(torch.nonzero(held_by_others == 0)[:, 0].tolist())}
    small = laid_out([[keep[p] for p in row] for row in held(table, lens, page)], table)
    want, rows, served, enough = resize([x[list(keep)] for x in caches], small, lens, new, page, len(keep))
    back = {i: p for p, i in keep.items()}
    assert not enough and stats.read()["status"] == 8
    assert torch.equal(n.cpu(), served)
    assert used(t, n, page) == [[back[p] for p in row] for row in rows]
    assert torch.equal(r.cpu(), counts([[back[p] for p in row] for row in rows], refs.numel()) + held_by_others)
    for a, b in zip(c, want):
        assert torch.equal(a.cpu()[list(keep)], b)


@pytest.mark.parametrize("holders", [2, 3, 8])
def test_every_holder_of_a_shared_page_copies_it(idx, holders):
    page = 16
    table = torch.full((holders, 3), -1, dtype=torch.int32)
    table[:, 0], table[:, 1] = 5, 2
    lens, refs = torch.full((holders,), 20, dtype=torch.int32), torch.zeros(12, dtype=torch.int32)
    refs[5] = refs[2] = holders
    new = torch.full((holders,), 21, dtype=torch.int32)
    r, t, n, _ = check_resize(idx, table, lens, refs, new, page, False)
    assert int(r[2]) == 0 and int(r[5]) == holders
    # a holder that does not grow keeps it; one that grows from a page's end shares on
    new[0] = 20
    check_resize(idx, table, lens, refs, new, page, True)
    full = torch.full((holders,), 32, dtype=torch.int32)
    check_resize(idx, table, full, refs, full + 1, page, False)
    # a row that shrinks leaves the page to the others first
    new = torch.full((holders,), 21, dtype=torch.int32)
    new[1:] = 16
    r, t, n, _ = check_resize(idx, table, lens, refs, new, page, False)
    assert int(t[0, 1]) == 2


def test_resize_leaves_rows_that_it_cannot_follow(idx):
    table, lens, refs = pool(5, 16, 60, 40, 3)
    caches = arrays(40, 2)
    new = lens + 20
    new[1], new[2] = -1, 16 * table.shape[1] + 1
    stats = idx.Stats()
    r, t, n = idx.idx_cache_resize([c.cuda() for c in caches], refs.cuda(), table.cuda(), lens.cuda(), new.cuda(),
                                   page_size=16, stats=stats)
    ok = new.clone()
    ok[1], ok[2] = lens[1], lens[2]
    _, rows, served, _ = resize(caches, table, lens, ok, 16, 40)
    assert stats.read()["status"] == 2 and torch.equal(n.cpu(), served) and used(t, n, 16) == rows
    bad = lens.clone()
    bad[0] = -3
    stats = idx.Stats()
    r, t, n = idx.idx_cache_resize([], refs.cuda(), table.cuda(), bad.cuda(), lens.cuda(), page_size=16, stats=stats)
    assert stats.read()["status"] == 2 and int(n[0]) == -3 and torch.equal(n[1:].cpu(), lens[1:])


def test_resize_of_no_rows_and_no_pages(idx):
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    table = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    refs = torch.arange(9, dtype=torch.int32, device="cuda")
    r, _, _ = idx.idx_cache_resize([], refs, table, none, none, page_size=16)
    assert torch.equal(r, refs)
    r, _, _ = idx.idx_cache_fork(refs, table, none, none, page_size=16)
    assert torch.equal(r, refs)
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    table = torch.zeros(3, 0, dtype=torch.int32, device="cuda")
    r, t, n = idx.idx_cache_resize([], none, table, lens, lens, page_size=16)
    assert n.tolist() == [0, 0, 0] and t.shape == (3, 0)
    assert idx.idx_cache_compact([], none, table, lens, page_size=16)[2].tolist() == [0]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,hi,page,spare", [(1, 10, 16, 0), (1, 10, 16, 1), (9, 200, 16, 50), (60, 900, 32, 3000),
                                             (300, 500, 16, 20000), (0, 1, 16, 100)])
def test_compact(idx, B, hi, page, spare, in_place):
    pages = B * pages_of(hi, page) + spare
    table, lens, refs = pool(B, page, hi, pages, B + spare, shared=B // 3)
    caches = arrays(pages, 4, ((2, 16), (1, 48), (16,)) if pages > 5000 else ((16, 1024), (3, 16)))
    want, counted, rows, live = compact(caches, refs, table, lens, page)
    d, c = [x.cuda() for x in (refs, table, lens)], [x.cuda() for x in caches]
    out = outputs(in_place, *d)
    out.pop("lens_out")
    stats = idx.Stats()
    r, t, n = idx.idx_cache_compact(c, *d, page_size=page, stats=stats, **out)
    assert stats.read()["status"] == 0
    assert n.tolist() == [live] and torch.equal(r.cpu(), counted) and used(t, d[2], page) == rows
    for a, b in zip(c, want):
        assert torch.equal(a.cpu()[:live], b[:live])


def test_compact_keeps_pages_that_no_row_names(idx):
    """Pages that another table holds move too; counts below 0 are free; entries outside the pool stay."""
    table, lens, refs = pool(3, 16, 60, 30, 8)
    free = (refs == 0).nonzero()[:, 0]
    refs[free[-2:]], refs[free[0]] = 3, -4
    table[1, 0] = 777
    caches = arrays(30, 5)
    stats = idx.Stats()
    c = [x.cuda() for x in caches]
    r, t, n = idx.idx_cache_compact(c, refs.cuda(), table.cuda(), lens.cuda(), page_size=16, stats=stats)
    live = int((refs > 0).sum())
    assert stats.read()["status"] == 2 and n.tolist() == [live] and int(t[1, 0]) == 777
    assert (r[:live] > 0).all() and (r[live:] == 0).all() and sorted(r[:live].tolist()) == sorted(refs[refs > 0].tolist())


def test_forked_requests_grow_apart(idx):
    """The calls together: beams share their pages, write on, end, and the pool is compacted."""
    page, B, pages = 16, 4, 30
    g = torch.Generator().manual_seed(0)
    cache = torch.zeros(pages, page, 16, dtype=torch.uint8, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table, lens = torch.full((B, 8), -1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    said = [[] for _ in range(B)]
    for step in range(60):
        grow = [40 if step == 0 else 1] * B
        new = lens + torch.tensor(grow, dtype=torch.int32, device="cuda")
        out = dict(refs_out=refs, table_out=table, lens_out=lens)
        idx.idx_cache_resize([cache], refs, table, lens, new, page_size=page, **out)
        for b in range(B):
            for _ in range(grow[b]):
                token = int(torch.randint(1, 256, (1,), generator=g))
                cache[int(table[b, len(said[b]) // page]), len(said[b]) % page] = token
                said[b].append(token)
        if step % 3 == 1:
            parent = torch.randint(0, B, (B,), generator=g).to(torch.int32)
            idx.idx_cache_fork(refs, table, lens, parent.cuda(), page_size=page, **out)
            said = [list(said[p]) for p in parent.tolist()]
        if step % 7 == 2:
            out.pop("lens_out")
            live = idx.idx_cache_compact([cache], refs, table, lens, page_size=page, **out)[2]
            assert int(live) == int((refs > 0).sum()) == len({p for r in used(table, lens, page) for p in r})
        assert torch.equal(refs.cpu().clamp_min(0), counts(used(table, lens, page), pages))
        for b in range(B):
            have = [int(cache[p, i, 0]) for p in used(table, lens, page)[b] for i in range(page)][:len(said[b])]
            assert have == said[b], (step, b)
