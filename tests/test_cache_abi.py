"""The C entry points of the cache in 4 bits and of its pages without a GPU: argument checks come before any CUDA
call, workspace sizes follow what they are asked for and grow with it, and the Python binding refuses what does not
fit."""
import ctypes
import itertools

import pytest
import torch

OK, EINVAL, EALIGN, EWORKSPACE, EUNSUPPORTED = 0, 1, 2, 3, 4
BF16, FP8, FP16, FP32 = 1, 2, 4, 5
P = 1 << 20  # an aligned address that the checks never read
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def idx():
    from sparse_attention_indexer_tiles_gb300 import build
    build.build()
    import sparse_attention_indexer_tiles_gb300 as pkg
    pkg.load()
    return pkg


def append(lib, **kw):
    a = dict(k=P, k_stride=256, v=P, v_stride=256, k_codes=P, k_sf=P, v_codes=P, v_sf=P, table=P, lens=P, q_start=P,
             B=2, T=4, Hkv=2, D=128, pages=10, page_size=64, table_stride=3, dt=BF16)
    a.update(kw)
    return lib.idx_cache_append_mxfp4(*a.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), EINVAL), (dict(T=-1), EINVAL), (dict(Hkv=0), EINVAL), (dict(pages=-1), EINVAL),
    (dict(table_stride=-1), EINVAL), (dict(k_stride=255), EINVAL), (dict(v_stride=0), EINVAL), (dict(D=96), EUNSUPPORTED),
    (dict(D=32, Hkv=1), EUNSUPPORTED), (dict(page_size=8), EUNSUPPORTED), (dict(page_size=0), EUNSUPPORTED),
    (dict(B=65536), EUNSUPPORTED), (dict(dt=FP32), EUNSUPPORTED), (dict(dt=FP8), EUNSUPPORTED),
    (dict(pages=1 << 24), EUNSUPPORTED), (dict(table_stride=1 << 40), EUNSUPPORTED), (dict(q_start=None, T=3), EINVAL),
    (dict(k=None), EINVAL), (dict(v_sf=None), EINVAL), (dict(table=None), EINVAL), (dict(lens=None), EINVAL),
    (dict(k=P + 1), EALIGN), (dict(k_codes=P + 8), EALIGN), (dict(v_sf=P + 4), EALIGN), (dict(lens=P + 2), EALIGN),
    (dict(q_start=P + 1), EALIGN), (dict(B=0, k=None), OK), (dict(T=0, k=None), OK)])
def test_append_checks(idx, kw, code):
    assert append(idx.load(), **kw) == code


def attention(lib, **kw):
    a = dict(q=P, q_stride=1024, k_codes=P, k_sf=P, v_codes=P, v_sf=P, table=P, lens=P, q_start=P, B=2, T=4, max_q=0,
             Hq=8, Hkv=2, D=128, pages=10, page_size=64, table_stride=3, max_len=0, window=0, sink=0, scale=0.1, dt=BF16,
             out=P, lse=None, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    return lib.idx_window_attention_mxfp4(*a.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), EINVAL), (dict(T=-1), EINVAL), (dict(max_q=-1), EINVAL), (dict(Hq=7), EINVAL), (dict(Hkv=0), EINVAL),
    (dict(window=-1), EINVAL), (dict(sink=-1), EINVAL), (dict(max_len=-1), EINVAL), (dict(max_len=193), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(q_stride=1023), EINVAL),
    (dict(q_start=None, T=3), EINVAL), (dict(q_start=None, max_q=1), EINVAL), (dict(Hq=258), EUNSUPPORTED),
    (dict(D=96), EUNSUPPORTED), (dict(page_size=48), EUNSUPPORTED), (dict(B=65536), EUNSUPPORTED),
    (dict(dt=FP32), EUNSUPPORTED), (dict(window=1 << 30), EUNSUPPORTED), (dict(sink=BIG), EUNSUPPORTED),
    (dict(T=BIG, q_stride=1024), EUNSUPPORTED), (dict(pages=1 << 25), EUNSUPPORTED), (dict(q=None), EINVAL),
    (dict(out=None), EINVAL), (dict(lens=None), EINVAL), (dict(table=None), EINVAL), (dict(k_codes=None), EINVAL),
    (dict(v_sf=None), EINVAL), (dict(pages=0), EINVAL), (dict(q=P + 8), EALIGN), (dict(q_stride=1028), EALIGN),
    (dict(out=P + 8), EALIGN), (dict(k_sf=P + 8), EALIGN), (dict(lse=P + 2), EALIGN), (dict(ws=P + 16), EALIGN),
    (dict(ws=None), EWORKSPACE), (dict(ws_bytes=100), EWORKSPACE), (dict(B=0, q=None), OK), (dict(T=0, q=None), OK)])
def test_attention_checks(idx, kw, code):
    assert attention(idx.load(), **kw) == code


SIZES = dict(B=[1, 7, 64], T=[1, 64, 5000], max_q=[1, 33, 5000], Hq=[4, 64], Hkv=[1, 4], D=[64, 128],
             max_len=[0, 1, 500, 40000], window=[1, 100, 5000, 0], sink=[0, 4, 1000])


def test_the_attentions_workspace_grows_with_its_arguments(idx):
    """One of the largest serves all: no size shrinks when an argument grows (a window of 0 is the largest)."""
    f = idx.load().idx_window_attention_mxfp4_workspace
    names = list(SIZES)
    at = {}
    for v in itertools.product(*SIZES.values()):
        at[v] = f(*v)
        assert 0 <= at[v] < 1 << 27
    for v in at:
        for i, n in enumerate(names):
            if n == "Hkv":
                continue  # fewer key heads make larger groups
            k = SIZES[n].index(v[i])
            if k:
                less = v[:i] + (SIZES[n][k - 1],) + v[i + 1:]
                assert at[less] <= at[v], (n, less, v)
    for bad in ((0, 4, 1, 8, 2, 128, 100, 0, 0), (1, 4, 1, 7, 2, 128, 100, 0, 0), (1, 4, 1, 8, 2, 96, 100, 0, 0),
                (1, 4, 1, 512, 2, 128, 100, 0, 0), (1, 4, 1, 8, 2, 128, -1, 0, 0), (1, 4, 1, 8, 0, 128, 1, 0, 0),
                (65536, 4, 1, 8, 2, 128, 100, 0, 0), (1, BIG, 1, 8, 2, 128, 100, 0, 0), (1, 4, 1, 8, 2, 128, BIG, 0, 0)):
        assert f(*bad) == 0, bad


def test_the_attentions_plan(idx):
    """What a call is cut into covers every key that a tile can see: sinks and the window's steps, which may begin and end
    inside one, in both paths."""
    plan = idx.idx_window_attention_mxfp4_plan
    for B, max_q, G, D, most, (window, sink) in itertools.product(
            [1, 16, 300], [1, 3, 500], [1, 5, 8, 128], [64, 128], [1, 100, 3000, 100000],
            [(0, 0), (1, 0), (1, 3), (64, 1), (1000, 100), (5000, 4000)]):
        p = plan(B, B * max_q, max_q, 2 * G, 2, D, most, window, sink)
        step = (80 if D == 128 else 96) if p["dense"] else 32
        tokens = min(max_q, max(1, -(-p["rows"] // G)) + 1)
        steps = -(-most // step)
        if window:
            steps = min(steps, -(-sink // step) + (window + tokens - 2) // step + 2)
        assert p["splits"] >= 1 and p["splits"] * p["keys"] >= steps * step, (p, B, max_q, G, D, most, window, sink)
        assert p["dense"] or p["rows"] in (8, 16)
    with pytest.raises(idx.IdxError):
        plan(1, 1, 1, 7, 2, 64, 100, 0, 0)
    assert idx.load().idx_window_attention_mxfp4_plan(1, 1, 1, 2, 2, 64, 100, 0, 0, None) == EINVAL


def two(*v):
    return (ctypes.c_void_p * 2)(*v), (ctypes.c_longlong * 2)(64, 48)


def resize(lib, **kw):
    caches, sizes = two(P, 2 * P)
    a = dict(caches=caches, sizes=sizes, n=2, refs=P, table=P, lens=P, new_lens=P, B=2, pages=10, page_size=64,
             table_stride=3, refs_out=P, table_out=P, lens_out=P, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    return lib.idx_cache_resize(*a.values(), None, None)


def fork(lib, **kw):
    a = dict(refs=P, table=P, lens=P, parent=P, B=2, pages=10, page_size=64, table_stride=3, refs_out=P, table_out=2 * P,
             lens_out=2 * P, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.idx_cache_fork(*a.values(), None, None)


def compact(lib, **kw):
    caches, sizes = two(P, 2 * P)
    a = dict(caches=caches, sizes=sizes, n=2, refs=P, table=P, lens=P, B=2, pages=10, page_size=64, table_stride=3,
             refs_out=P, table_out=P, live=P, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    return lib.idx_cache_compact(*a.values(), None, None)


COMMON = [(dict(B=-1), EINVAL), (dict(pages=-1), EINVAL), (dict(table_stride=-1), EINVAL), (dict(page_size=48), EUNSUPPORTED),
          (dict(B=1 << 25), EUNSUPPORTED), (dict(table_stride=1 << 26), EUNSUPPORTED), (dict(refs=None), EINVAL),
          (dict(refs_out=None), EINVAL), (dict(table=None), EINVAL), (dict(table_out=None), EINVAL), (dict(lens=None), EINVAL),
          (dict(refs=P + 2), EALIGN), (dict(table_out=P + 1), EALIGN), (dict(lens=P + 3), EALIGN)]
ARRAYS = [(dict(n=-1), EINVAL), (dict(n=9), EUNSUPPORTED), (dict(caches=None), EINVAL), (dict(sizes=None), EINVAL),
          (dict(caches=two(P, None)[0]), EINVAL), (dict(caches=two(P, P + 8)[0]), EALIGN),
          (dict(sizes=(ctypes.c_longlong * 2)(64, 40)), EALIGN), (dict(sizes=(ctypes.c_longlong * 2)(0, 16)), EINVAL)]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(parent=None), EINVAL), (dict(lens_out=None), EINVAL), (dict(parent=P + 2), EALIGN),
    (dict(table_out=P), EWORKSPACE), (dict(lens_out=P), EWORKSPACE), (dict(lens_out=P, ws=P, ws_bytes=8), EWORKSPACE),
    (dict(lens_out=P, ws=P + 4, ws_bytes=1 << 30), EALIGN), (dict(B=0, pages=0), OK)])
def test_fork_checks(idx, kw, code):
    assert fork(idx.load(), **kw) == code


def test_a_fork_does_not_write_its_parents(idx):
    assert fork(idx.load(), parent=P, lens=2 * P, lens_out=P) == EINVAL


@pytest.mark.parametrize("kw,code", COMMON + ARRAYS + [
    (dict(new_lens=None), EINVAL), (dict(lens_out=None), EINVAL), (dict(new_lens=P + 2), EALIGN), (dict(ws=None), EWORKSPACE),
    (dict(ws_bytes=8), EWORKSPACE), (dict(ws=P + 16), EALIGN), (dict(B=0, pages=0, n=0), OK)])
def test_resize_checks(idx, kw, code):
    assert resize(idx.load(), **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + ARRAYS + [
    (dict(live=None), EINVAL), (dict(live=P + 1), EALIGN), (dict(ws=None), EWORKSPACE), (dict(ws_bytes=8), EWORKSPACE),
    (dict(ws=P + 16), EALIGN)])
def test_compact_checks(idx, kw, code):
    assert compact(idx.load(), **kw) == code


def test_the_pages_workspaces(idx):
    lib = idx.load()
    assert lib.idx_cache_fork_workspace(0, 5) == 0 and lib.idx_cache_fork_workspace(3, -1) == 0
    assert lib.idx_cache_fork_workspace(3, 5) >= 4 * (3 + 15)
    assert lib.idx_cache_resize_workspace(-1, 5, 5) == 0 and lib.idx_cache_resize_workspace(3, 10, 2) >= 4 * (7 * 3 + 1 + 9)
    assert lib.idx_cache_resize_workspace(3, 1 << 30, 2) < 4096
    assert lib.idx_cache_compact_workspace(3, -1) == 0 and lib.idx_cache_compact_workspace(0, 100) >= 4 * (4 + 102 + 100)


def binding_calls(idx):
    codes, sf = torch.zeros(6, 2, 16, 32, dtype=torch.uint8), torch.zeros(6, 2, 16, 2, dtype=torch.uint8)
    table, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    k, q, refs = torch.zeros(2, 2, 64).bfloat16(), torch.zeros(2, 4, 64).bfloat16(), torch.zeros(6, dtype=torch.int32)
    return {
        "append": lambda x=k: idx.idx_cache_append_mxfp4(x, k, codes, sf, codes, sf, table, lens),
        "attention": lambda x=q: idx.idx_window_attention_mxfp4(x, codes, sf, codes, sf, table, lens),
        "fork": lambda x=refs: idx.idx_cache_fork(x, table, lens, lens, page_size=16),
        "resize": lambda x=refs: idx.idx_cache_resize([codes, sf], x, table, lens, lens, page_size=16),
        "compact": lambda x=refs: idx.idx_cache_compact([codes, sf], x, table, lens, page_size=16)}


@pytest.mark.parametrize("name", ["append", "attention", "fork", "resize", "compact"])
def test_the_binding_refuses_tensors_of_the_host(idx, name):
    with pytest.raises(ValueError, match="must live on a CUDA device"):
        binding_calls(idx)[name]()


@pytest.mark.parametrize("name", ["attention", "fork", "resize", "compact"])
def test_the_binding_refuses_wrong_ranks(idx, name):
    with pytest.raises(ValueError):
        binding_calls(idx)[name](torch.zeros(3, 3))


def test_the_module_checks_its_own_arguments(idx):
    m = idx._serve()
    for f in (m.cache_append_mxfp4, m.window_attention_mxfp4, m.cache_fork, m.cache_resize, m.cache_compact, m.bind_cache):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(ValueError, match="null"):
        m.bind_cache(0, 1, 2, 3, 4)
    with pytest.raises(ValueError, match="not a tensor"):
        m.cache_append_mxfp4(3, *[None] * 10)
    for f, n, what in ((m.cache_append_mxfp4, 11, "k_codes"), (m.window_attention_mxfp4, 18, "k_codes"),
                       (m.cache_fork, 11, "refs"), (m.cache_resize, 12, "refs"), (m.cache_compact, 11, "refs")):
        with pytest.raises(ValueError, match=what + " is missing"):
            f(*[None] * n)
