"""The serving operators' Python binding without a GPU: what it refuses before it reaches the
library."""
import pytest
import torch


@pytest.fixture(scope="module")
def idx():
    from sparse_attention_indexer_tiles_gb300 import build
    build.build()
    import sparse_attention_indexer_tiles_gb300 as pkg
    pkg.load()
    return pkg


def calls(idx):
    x, w = torch.zeros(4, 128), torch.zeros(128)
    cache = torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16)
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    weights, pos = torch.zeros(2, 2, 48), torch.zeros(2, 2, 48, dtype=torch.int32)
    return {
        "norm": lambda **k: idx.idx_add_rmsnorm_quant(k.get("x", x), w, group=k.get("group", 0)),
        "attention": lambda **k: idx.idx_prefix_attention(k.get("x", q), cache, cache, table, lens),
        "evict": lambda **k: idx.idx_cache_evict(k.get("x", cache), cache, table, lens, weights, pos, lens,
                                                 k.get("group", 8)),
    }


@pytest.mark.parametrize("name", ["norm", "attention", "evict"])
def test_tensors_of_the_host_are_refused(idx, name):
    with pytest.raises(ValueError, match="must live on a CUDA device"):
        calls(idx)[name]()


@pytest.mark.parametrize("name", ["norm", "attention", "evict"])
def test_wrong_ranks_are_refused(idx, name):
    with pytest.raises(ValueError):
        calls(idx)[name](x=torch.zeros(3))


def test_the_module_checks_its_own_arguments(idx):
    m = idx._serve()
    for f in (m.add_rmsnorm_quant, m.prefix_attention, m.cache_evict, m.bind):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(ValueError, match="null"):
        m.bind(0, 1, 2)
    with pytest.raises(TypeError):
        m.bind("a", 1, 2)
    for bad in (3, "x", [1.0]):
        with pytest.raises(ValueError, match="not a tensor"):
            m.add_rmsnorm_quant(bad, None, None, None, 1e-6, 0, None, None, None, None)
    with pytest.raises(ValueError, match="q is missing"):
        m.prefix_attention(*[None] * 16)
    with pytest.raises(ValueError, match="k_cache is missing"):
        m.cache_evict(*[None] * 17)


def test_the_module_is_on_the_loaded_library(idx):
    assert idx._serve() is idx._serve()
