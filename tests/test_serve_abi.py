"""The serving operators' C entry points without a GPU: argument checks come before any
CUDA call, and the workspace sizes follow the sizes they are asked for."""
import ctypes

import pytest

OK, EINVAL, EALIGN, EWORKSPACE, EUNSUPPORTED = 0, 1, 2, 3, 4
BF16, FP8, FP16, FP32 = 1, 2, 4, 5


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_tiles_gb300 import build
    build.build()
    import sparse_attention_indexer_tiles_gb300 as pkg
    return pkg.load()


P = 1 << 20  # an aligned address that the checks never read
LL, F, SZ = ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t


def norm(lib, **kw):
    a = dict(x=P, x_stride=128, residual=None, weight=P, rows=4, N=128, eps=1e-6, group=0, dt=BF16, residual_out=None,
             out=P, scale=P)
    a.update(kw)
    return lib.idx_add_rmsnorm_quant(*a.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), EINVAL), (dict(N=0), EINVAL), (dict(x_stride=127), EINVAL), (dict(eps=-1.0), EINVAL),
    (dict(eps=float("nan")), EINVAL), (dict(group=16), EINVAL), (dict(group=-32), EINVAL),
    (dict(N=96, group=64), EINVAL), (dict(dt=FP8), EUNSUPPORTED), (dict(dt=9), EUNSUPPORTED),
    (dict(N=32769, x_stride=32769), EUNSUPPORTED), (dict(x=None), EINVAL), (dict(weight=None), EINVAL),
    (dict(out=None), EINVAL), (dict(scale=None), EINVAL), (dict(residual_out=P), EINVAL),
    (dict(x=P + 1), EALIGN), (dict(dt=FP32, x=P + 2), EALIGN), (dict(scale=P + 2), EALIGN),
    (dict(residual=P + 1), EALIGN), (dict(group=32, x=P + 2), EALIGN), (dict(group=32, x_stride=129), EALIGN),
    (dict(group=32, out=P + 4), EALIGN), (dict(rows=0, x=None), OK)])
def test_norm_checks(lib, kw, code):
    assert norm(lib, **kw) == code


def attention(lib, **kw):
    a = dict(q=P, k=P, v=P, prefix_table=P, table=P, lens=P, w=None, B=2, Q=1, Hq=8, Hkv=2, D=128, pages=10,
             page_size=64, prefix_len=100, table_stride=3, max_len=0, slots=0, scale=0.1, dt=BF16, out=P, lse=None,
             w_out=None, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    return lib.idx_prefix_attention(*a.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), EINVAL), (dict(Q=0), EINVAL), (dict(Q=17), EUNSUPPORTED), (dict(Hq=7), EINVAL), (dict(Hkv=0), EINVAL),
    (dict(Hq=258, Hkv=2), EUNSUPPORTED), (dict(D=96), EUNSUPPORTED), (dict(page_size=48), EUNSUPPORTED),
    (dict(page_size=8), EUNSUPPORTED), (dict(page_size=0), EUNSUPPORTED), (dict(prefix_len=-1), EINVAL),
    (dict(max_len=193), EINVAL), (dict(max_len=-1), EINVAL), (dict(table_stride=1 << 40), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(w=P), EINVAL), (dict(w_out=P), EINVAL),
    (dict(w=P, w_out=P, slots=191), EINVAL), (dict(dt=FP8), EUNSUPPORTED), (dict(dt=FP32), EUNSUPPORTED),
    (dict(B=40000), EUNSUPPORTED), (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(lens=None), EINVAL),
    (dict(prefix_table=None), EINVAL), (dict(table=None), EINVAL), (dict(out=None), EINVAL), (dict(q=P + 8), EALIGN),
    (dict(v=P + 8), EALIGN), (dict(lens=P + 2), EALIGN), (dict(ws=P + 128), EALIGN), (dict(ws=None), EWORKSPACE),
    (dict(ws_bytes=100), EWORKSPACE), (dict(B=0, q=None), OK)])
def test_attention_checks(lib, kw, code):
    assert attention(lib, **kw) == code


def evict(lib, **kw):
    a = dict(k=P, v=P, table=P, lens=P, w=P, positions=P, next_pos=P, B=2, Hkv=2, D=128, pages=10, page_size=64,
             table_stride=3, max_len=0, slots=192, budget=50, recent=10, sink=4, dt=BF16, lens_out=2 * P, w_out=P,
             positions_out=P, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    return lib.idx_cache_evict(*a.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), EINVAL), (dict(Hkv=0), EINVAL), (dict(budget=0), EINVAL), (dict(recent=-1), EINVAL),
    (dict(sink=-1), EINVAL), (dict(recent=47), EINVAL), (dict(recent=2 ** 31 - 1, sink=2 ** 31 - 1), EINVAL),
    (dict(D=32), EUNSUPPORTED), (dict(page_size=100), EUNSUPPORTED), (dict(dt=FP32), EUNSUPPORTED),
    (dict(slots=191), EINVAL), (dict(max_len=193), EINVAL), (dict(lens=None), EINVAL), (dict(lens_out=P), EINVAL),
    (dict(next_pos=None), EINVAL), (dict(w=None), EINVAL), (dict(positions_out=None), EINVAL), (dict(k=P + 4), EALIGN),
    (dict(w=P + 2), EALIGN), (dict(ws=None), EWORKSPACE), (dict(ws_bytes=8), EWORKSPACE), (dict(ws=P + 16), EALIGN),
    (dict(B=0, lens=None), OK)])
def test_evict_checks(lib, kw, code):
    assert evict(lib, **kw) == code


def test_workspaces(lib):
    ws = lib.idx_prefix_attention_workspace
    assert ws(0, 1, 8, 2, 128, 100, 100, 0) == 0 and ws(2, 1, 7, 2, 128, 100, 100, 0) == 0
    small, big = ws(2, 1, 8, 2, 128, 100, 100, 0), ws(2, 1, 8, 2, 128, 100, 100, 1)
    assert 0 < small < big and big - small >= 2 * 8 * 100 * 4
    assert ws(2, 1, 8, 2, 128, 0, 0, 0) == 0
    ev = lib.idx_cache_evict_workspace
    assert ev(2, 2, 100, 100) == 0 and ev(2, 2, 100, 50) == 0
    assert ev(2, 2, 100, 101) >= 2 * 2 * 2 * 4
    assert ev(2, 2, 100, 1 << 20) >= 2 * 2 * 2 * 100 * 4
