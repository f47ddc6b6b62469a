"""The attention's workspace query on sizes that the call refuses, in a process of its own: a
query that divides by zero would take this one down."""
import subprocess
import sys

import pytest

INT_MAX = 2 ** 31 - 1

# B, Q, Hq, Hkv, D, prefix_len, max_len, weights
REFUSED = [(1, 1, 129, 1, 128, 100, 64, 0), (1, 1, 256, 1, 128, 100, 64, 0), (2, 16, 258, 2, 64, 0, 64, 1),
           (1, 1, 256, 1, 64, 0, 640, 0), (1, 17, 8, 2, 128, 100, 64, 0), (1, INT_MAX, 8, 2, 128, 100, 64, 0),
           (1, 1, 8, 2, 96, 100, 64, 0), (1, 1, 8, 2, 0, 100, 64, 0), (1, 1, 8, 2, 256, 100, 64, 0),
           (1, 1, 8, 2, 128, INT_MAX, 64, 0), (1, 1, 8, 2, 128, 1 << 30, 64, 0), (1, 1, 8, 2, 128, 100, INT_MAX, 1),
           (1, 1, 8, 2, 128, 0, 1 << 30, 0), (40000, 1, 8, 2, 128, 100, 64, 0), (60000, 16, 4096, 1, 128, 0, 64, 0),
           (1, 1, INT_MAX, 1, 128, 100, 64, 0), (INT_MAX, 16, 128, 1, 64, 100, 64, 1)]
# the largest that it takes
TAKEN = [(1, 16, 128, 1, 128, 2 ** 30 - 1, 64, 0), (1, 1, 8, 2, 64, 100, 2 ** 30 - 1, 0), (65535, 1, 8, 1, 64, 0, 64, 0)]


def ask(sizes):
    code = ("import sparse_attention_indexer_tiles_gb300 as p; "
            f"print(p.load().idx_prefix_attention_workspace(*{sizes!r}))")
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_attention_indexer_tiles_gb300 import build
    build.build()


@pytest.mark.parametrize("sizes", [(1, 1, 256, 1, 128, 100, 64, 0), (1, 1, 129, 1, 128, 0, 64, 0)])
def test_a_group_that_is_too_wide_does_not_end_the_process(sizes):
    r = ask(sizes)
    assert r.returncode == 0 and int(r.stdout) == 0, (r.returncode, r.stderr)


def test_refused_sizes_need_nothing_and_the_largest_something():
    code = ("import sparse_attention_indexer_tiles_gb300 as p; f = p.load().idx_prefix_attention_workspace; "
            f"print([f(*s) for s in {REFUSED + TAKEN!r}])")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.returncode
    sizes = eval(r.stdout)
    assert sizes[:len(REFUSED)] == [0] * len(REFUSED)
    assert all(0 < n < 1 << 42 for n in sizes[len(REFUSED):]), sizes


def test_the_call_refuses_what_the_query_refuses():
    from sparse_attention_indexer_tiles_gb300 import load
    P = 1 << 20
    for B, Q, Hq, Hkv, D, prefix, most, weights in REFUSED:
        code = load().idx_prefix_attention(
            P, P, P, P, P, P, P if weights else None, B, Q, Hq, Hkv, D, 10, 64, prefix, 1 << 25, most, INT_MAX, 0.1, 1,
            P, None, P if weights else None, P, 1 << 60, None, None)
        assert code in (1, 4), (B, Q, Hq, Hkv, D, prefix, most)


def test_the_plan():
    import ctypes
    from sparse_attention_indexer_tiles_gb300 import IdxError, idx_prefix_attention_plan, load
    p = idx_prefix_attention_plan(8, 1, 64, 8, 128, 32768, 1024, True)
    assert p["prefix_parts"] * p["prefix_keys"] >= 32768 and p["private_parts"] * p["private_keys"] >= 1024
    assert (p["prefix_parts"] - 1) * p["prefix_keys"] < 32768 and not p["private_dense"]
    assert idx_prefix_attention_plan(8, 16, 16, 1, 64, 0, 4000, False)["private_dense"]
    for sizes in REFUSED:
        with pytest.raises(IdxError) as e:
            idx_prefix_attention_plan(*sizes)
        assert e.value.code == 4
    assert load().idx_prefix_attention_plan(1, 1, 8, 2, 128, 0, 64, 0, None) == 1
    assert load().idx_prefix_attention_plan(0, 1, 8, 2, 128, 0, 64, 0, (ctypes.c_int * 5)()) == 1
