"""What a call allocates when it is given a stream, without a GPU: on that stream, with the
tensors it returns marked as used on the caller's.  Anything else is a race: a fill on the
caller's stream may run after the kernels, and a workspace of that stream's pool may be handed
out again while they run."""
import contextlib
import types

import pytest
import torch

import sparse_attention_indexer_tiles_gb300 as pkg

CUDA = torch.device("cuda", 0)


class FakeStream:
    def __init__(self, handle, device=CUDA):
        self.cuda_stream, self.device = handle, device


class FakeTensor:
    is_cuda, device, dtype = True, CUDA, torch.float32

    def __init__(self, shape, log, made_on=None):
        self.shape, self.log, self.made_on, self.used_on = tuple(shape), log, made_on, []

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256

    def numel(self):
        return 1 << 30

    def element_size(self):
        return 1

    def record_stream(self, s):
        self.used_on.append(s.cuda_stream)


class World:
    """torch's streams and allocations, as far as the wrappers use them."""

    def __init__(self, monkeypatch):
        self.now, self.made, self.launches = FakeStream(7), [], []

        @contextlib.contextmanager
        def on(s):
            was, self.now = self.now, s
            yield
            self.now = was

        def make(shape):
            t = FakeTensor(shape, self, self.now.cuda_stream)
            self.made.append(t)
            return t

        for name, f in (("empty", lambda *s, **k: make(s[0] if isinstance(s[0], tuple) else s)),
                        ("empty_like", lambda t: make(t.shape)), ("zeros_like", lambda t: make(t.shape)),
                        ("full_like", lambda t, v: make(t.shape))):
            monkeypatch.setattr(torch, name, f)
        cuda = types.SimpleNamespace(
            Stream=FakeStream, stream=on, device=lambda d: contextlib.nullcontext(),
            current_stream=lambda d=None: self.now, default_stream=lambda d: FakeStream(0),
            ExternalStream=lambda h, device: FakeStream(h, device))
        monkeypatch.setattr(torch, "cuda", cuda)
        launch = lambda *a: self.launches.append(a) or 0  # noqa: E731
        monkeypatch.setattr(pkg, "_serve", lambda: types.SimpleNamespace(
            add_rmsnorm_quant=launch, prefix_attention=launch, cache_evict=launch))
        for name in ("idx_prefix_attention_workspace", "idx_cache_evict_workspace"):
            monkeypatch.setattr(pkg, name, lambda *a: 4096)

    def t(self, *shape):
        return FakeTensor(shape, self)


def serving(w, **kw):
    cache, table, lens, slots = w.t(6, 2, 16, 64), w.t(2, 3), w.t(2), w.t(2, 2, 48)
    return {
        "norm": lambda: pkg.idx_add_rmsnorm_quant(w.t(4, 128), w.t(128), **kw),
        "attention": lambda: pkg.idx_prefix_attention(w.t(2, 1, 4, 64), cache, cache, table, lens, weights=slots, **kw),
        "evict": lambda: pkg.idx_cache_evict(cache, cache, table, lens, slots, slots, lens, 8, **kw)}


@pytest.mark.parametrize("stream", [FakeStream(42), 42, 0, 1])
@pytest.mark.parametrize("name,made", [("norm", 2), ("attention", 4), ("evict", 4)])
def test_on_the_launch_stream(monkeypatch, name, made, stream):
    w = World(monkeypatch)
    got = serving(w, stream=stream)[name]()
    handle = 42 if stream not in (0, 1) else 0
    assert [t.made_on for t in w.made] == [handle] * made
    assert w.now.cuda_stream == 7 and len(w.launches) == 1
    assert w.launches[0][-1] == (stream.cuda_stream if isinstance(stream, FakeStream) else stream)
    assert all(t.used_on == [7] for t in got)
    assert sum(t.used_on == [] for t in w.made) == made - len(got)  # the workspace


@pytest.mark.parametrize("stream", [None, FakeStream(7), 7])
@pytest.mark.parametrize("name,made", [("norm", 2), ("attention", 4), ("evict", 4)])
def test_on_the_callers_own_stream(monkeypatch, name, made, stream):
    w = World(monkeypatch)
    serving(w, stream=stream)[name]()
    assert [t.made_on for t in w.made] == [7] * made
    assert all(t.used_on == [] for t in w.made) and len(w.launches) == 1


@pytest.mark.parametrize("name", ["norm", "attention", "evict"])
def test_a_stream_of_another_device(monkeypatch, name):
    w = World(monkeypatch)
    with pytest.raises(ValueError, match="stream of cuda:1"):
        serving(w, stream=FakeStream(42, torch.device("cuda", 1)))[name]()
    assert not w.made and not w.launches


class FakeLibrary:
    """Every size query answers 4096, every call 0 (with its stream, the last argument, kept)."""

    def __init__(self, world):
        self.world = world

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            f = lambda *a: 4096  # noqa: E731
        else:
            f = lambda *a: self.world.launches.append(a) or 0  # noqa: E731
        return f


def scoring(w, **kw):
    def t(dtype, *shape):
        x = w.t(*shape)
        x.dtype = dtype
        return x

    q, k = t(torch.bfloat16, 4, 8, 64), t(torch.bfloat16, 100, 64)
    rest = [w.t(100), w.t(4, 8), w.t(4), w.t(4)]
    x, sf, kx, ksf = (t(torch.uint8, *s) for s in ((4, 8, 32), (4, 8, 2), (100, 32), (100, 2)))
    codes = (x, sf, kx, ksf)
    return {
        "topk": (lambda: pkg.idx_score_topk(q, k, *rest, 16, **kw), 1, 1),
        "from_scores": (lambda: pkg.idx_topk_from_scores(w.t(4, 100), None, rest[3], 16, **kw), 1, 1),
        "materialise": (lambda: pkg.idx_score_materialise(q, k, *rest, **kw), 1, 0),
        "expand": (lambda: pkg.idx_mxfp4_to_e4m3(x, sf, **kw), 1, 0),
        "topk_mxfp4": (lambda: pkg.idx_score_topk_mxfp4(*codes, *rest, 16, **kw), 1, 1),
        "materialise_mxfp4": (lambda: pkg.idx_score_materialise_mxfp4(*codes, *rest, **kw), 1, 1),
        "noalloc": (lambda: pkg.idx_score_topk_noalloc(q, k, *rest, 16, **kw), 1, 0),
        "routed": (lambda: pkg.idx_score_topk_routed(q, k, *rest, 16, **kw), 1, 1)}


@pytest.mark.parametrize("stream", [None, FakeStream(7), FakeStream(42), 42, 0])
@pytest.mark.parametrize("name", ["topk", "from_scores", "materialise", "expand", "topk_mxfp4", "materialise_mxfp4",
                                  "noalloc", "routed"])
def test_the_scoring_calls(monkeypatch, name, stream):
    w = World(monkeypatch)
    monkeypatch.setattr(pkg, "load", lambda: FakeLibrary(w))
    call, results, workspaces = scoring(w, stream=stream)[name]
    got = call()
    handle = {None: 7, 42: 42, 0: 0}[stream] if not isinstance(stream, FakeStream) else stream.cuda_stream
    assert [t.made_on for t in w.made] == [handle] * (results + workspaces)
    assert w.launches[-1][-1] == handle
    assert got.used_on == ([7] if handle != 7 else [])
    assert sum(t.used_on == [] for t in w.made) == workspaces + (results if handle == 7 else 0)
