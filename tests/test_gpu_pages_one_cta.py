"""idx_cache_resize and idx_cache_compact rank their pages with one CTA where a device does not place the cluster that many
pages or rows would take: the same results."""
import pytest
import torch

from _cache_ref import compact, counts, laid_out, pages_of, resize
from test_gpu_cache_pages import arrays, idx, lengths, outputs, pool, used  # noqa: F401

pytestmark = pytest.mark.gpu
ONE = {"row_split": -1}


@pytest.mark.parametrize("options", [ONE, None])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["step", "any"])
@pytest.mark.parametrize("B,hi,page,spare", [(5, 90, 16, 40), (700, 300, 16, 5000), (1100, 100, 16, 20000)])
def test_resize(idx, B, hi, page, spare, kind, in_place, options):
    pages = B * pages_of(hi, page) + spare
    table, lens, refs = pool(B, page, hi, pages, B, shared=B // 3, zeros=0.1)
    new, caches = lengths(lens, kind, hi, B).to(torch.int32), arrays(pages, B)
    want, rows, served, enough = resize(caches, table, lens, new, page, pages)
    d, c = [x.cuda() for x in (refs, table, lens)], [x.cuda() for x in caches]
    stats = idx.Stats()
    r, t, n = idx.idx_cache_resize(c, *d, new.cuda(), page_size=page, options=options, stats=stats, **outputs(in_place, *d))
    assert enough and stats.read()["status"] == 0 and torch.equal(n.cpu(), served) and used(t, n, page) == rows
    assert torch.equal(r.cpu().clamp_min(0), counts(rows, pages))
    assert all(torch.equal(a.cpu(), b) for a, b in zip(c, want))
    if not in_place:
        assert torch.equal(t.cpu(), laid_out(rows, table))


@pytest.mark.parametrize("options", [ONE, None])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,hi,page,spare", [(9, 200, 16, 50), (300, 500, 16, 20000), (0, 1, 16, 6000)])
def test_compact(idx, B, hi, page, spare, in_place, options):
    pages = B * pages_of(hi, page) + spare
    table, lens, refs = pool(B, page, hi, pages, B + spare, shared=B // 3)
    caches = arrays(pages, 4, ((1, 48), (16,)))
    want, counted, rows, live = compact(caches, refs, table, lens, page)
    d, c = [x.cuda() for x in (refs, table, lens)], [x.cuda() for x in caches]
    out = outputs(in_place, *d)
    out.pop("lens_out")
    stats = idx.Stats()
    r, t, n = idx.idx_cache_compact(c, *d, page_size=page, options=options, stats=stats, **out)
    assert stats.read()["status"] == 0 and n.tolist() == [live]
    assert torch.equal(r.cpu(), counted) and used(t, d[2], page) == rows
    assert all(torch.equal(a.cpu()[:live], b[:live]) for a, b in zip(c, want))
