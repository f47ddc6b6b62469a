"""idx_cache_resize reports a table entry that names no page, wherever in a row's length it lies, and keeps it."""
import pytest
import torch

from _cache_ref import counts, held, pages_of
from test_gpu_cache_pages import idx, outputs, pool  # noqa: F401

pytestmark = pytest.mark.gpu


def run(idx, table, lens, refs, new, in_place):
    d = [x.cuda() for x in (refs, table, lens)]
    stats = idx.Stats()
    r, t, n = idx.idx_cache_resize([], *d, new.cuda(), page_size=16, stats=stats, **outputs(in_place, *d))
    return r.cpu(), t.cpu(), n.cpu(), stats.read()["status"]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("wild", [-1, 40, 2 ** 31 - 1])
@pytest.mark.parametrize("old,new,slot", [(60, 60, 1), (60, 61, 0), (64, 65, 3), (60, 20, 1), (60, 20, 3), (60, 61, 3),
                                          (60, 0, 2), (64, 64, 0)])
@pytest.mark.parametrize("B", [3, 300])
def test_a_bad_entry_is_reported_and_kept(idx, B, old, new, slot, wild, in_place):
    """Kept, dropped and to be copied; with one CTA that ranks and with a cluster."""
    pages = 40 if B == 3 else 3000
    wild = pages if wild == 40 else wild
    table = torch.full((B, 6), -1, dtype=torch.int32)
    lens = torch.full((B,), 60 if B == 3 else 16, dtype=torch.int32)
    lens[1] = old
    at = 0
    for b in range(B):
        n = pages_of(int(lens[b]), 16)
        table[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    refs = counts(held(table, lens, 16), pages)
    refs[table[1, slot]] -= 1
    table[1, slot] = wild
    want = lens.clone()
    want[1] = new
    r, t, n, st = run(idx, table, lens, refs, want, in_place)
    assert st == 2 and torch.equal(n, want)
    kept = min(pages_of(old, 16), pages_of(new, 16))
    assert torch.equal(t[1, :kept], table[1, :kept])
    rows = held(t, n, 16)
    good = counts([[p for p in row if 0 <= p < pages] for row in rows], pages)
    assert torch.equal(r, good)


@pytest.mark.parametrize("in_place", [False, True])
def test_entries_past_a_rows_length_are_not_looked_at(idx, in_place):
    table, lens, refs = pool(5, 16, 60, 40, 3)
    for b, n in enumerate(lens.tolist()):
        table[b, pages_of(n, 16):] = 1000
    r, t, n, st = run(idx, table, lens, refs, lens, in_place)
    assert st == 0 and torch.equal(n, lens) and torch.equal(r, refs)
