"""The attention's workspace size does not shrink when an argument grows, so that a buffer for a
program's largest call serves all of its calls."""
import random

import pytest

P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_tiles_gb300 import build
    build.build()
    import sparse_attention_indexer_tiles_gb300 as pkg
    return pkg.load()


def size(lib, B, Q, G, Hkv, D, prefix, most, weights):
    return lib.idx_prefix_attention_workspace(B, Q, G * Hkv, Hkv, D, prefix, most, weights)


BASE = dict(B=32, Q=1, G=8, Hkv=8, D=128, prefix=32768, most=1024, weights=0)


@pytest.mark.parametrize("base", [{}, dict(Q=2, B=16, prefix=4096), dict(G=16, Hkv=1, D=64, weights=1),
                                  dict(B=3, most=60000), dict(B=60, prefix=512, most=8192, weights=1),
                                  dict(Q=16, G=16, Hkv=2), dict(prefix=0), dict(most=0)])
@pytest.mark.parametrize("name,values", [("B", range(1, 200)), ("Q", range(1, 17)), ("G", range(1, 129)),
                                         ("prefix", [*range(0, 3000, 37), *range(3000, 300000, 997)]),
                                         ("most", [*range(0, 3000, 37), *range(3000, 300000, 997)]),
                                         ("weights", (0, 1)), ("D", (64, 128))])
def test_along_one_argument(lib, base, name, values):
    sizes = [size(lib, **(BASE | base | {name: v})) for v in values]
    assert sizes == sorted(sizes)


def test_any_smaller_call_fits(lib):
    rng = random.Random(1)
    log = lambda most: int(most ** rng.random())  # noqa: E731
    for _ in range(3000):
        big = dict(B=log(300), Q=log(16), G=log(128), Hkv=rng.choice([1, 2, 8]), D=rng.choice([64, 128]),
                   prefix=log(200000), most=log(100000), weights=rng.randint(0, 1))
        small = {n: v if n == "Hkv" else rng.choice([64, v]) if n == "D" else rng.randint(0, v) if n in (
            "prefix", "most", "weights") else rng.randint(1, v) for n, v in big.items()}
        assert size(lib, **small) <= size(lib, **big), (small, big)


@pytest.mark.parametrize("B", [32, 33, 37])
def test_the_call_takes_the_largest_batchs_buffer(lib, B):
    """64 heads behind 32768 keys: 38 requests had needed less than 32.  (The address is refused next,
    as not aligned, so that nothing is launched.)"""
    have = size(lib, **(BASE | dict(B=38)))
    code = lib.idx_prefix_attention(P, P, P, P, P, P, None, B, 1, 64, 8, 128, 1000, 64, 32768, 16, 1024, 0, 0.1, 1, P,
                                    None, None, P + 128, have, None, None)
    assert code == 2
