"""The calls on pages refuse what their 32-bit page numbers would run past, before any CUDA call."""
import pytest

from test_cache_abi import BIG, EUNSUPPORTED, EWORKSPACE, compact, fork, idx, resize  # noqa: F401

MOST = 0x7fffff00                                # a step of 256 pages from below it stays below 2^31


@pytest.mark.parametrize("pages", [MOST + 1, BIG])
def test_more_pages_than_the_rankings_number(idx, pages):
    lib = idx.load()
    for f in (fork, resize, compact):
        assert f(lib, pages=pages) == EUNSUPPORTED
    assert lib.idx_cache_resize_workspace(3, pages, 2) == 0 and lib.idx_cache_compact_workspace(3, pages) == 0


def test_the_most_pages(idx):
    """Not refused for their number: the next check answers."""
    lib = idx.load()
    for f in (resize, compact):
        assert f(lib, pages=MOST, ws=None) == EWORKSPACE
    assert fork(lib, pages=MOST, table_out=1 << 20) == EWORKSPACE
    assert lib.idx_cache_resize_workspace(3, MOST, 2) > 0 and lib.idx_cache_compact_workspace(3, MOST) > 4 * MOST


def test_no_page_number_runs_over():
    """The loops of the rankings over the last warp's pages, as the kernels step them."""
    for ctas in (1, 16):
        groups = (MOST + 31) // 32
        per = -(-groups // (ctas * 32)) * 32
        for warp in (0, ctas * 32 - 1):
            first, end = min(warp * per, MOST), min((warp + 1) * per, MOST)
            last = first + (max(end - first, 1) - 1) // 256 * 256
            assert last + 7 * 32 + 31 <= BIG and last + 256 <= BIG
            last = first + (max(end - first, 1) - 1) // 32 * 32
            assert last + 31 + 32 <= BIG
