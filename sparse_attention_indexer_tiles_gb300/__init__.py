"""Python binding of libidx, the GB300 (sm_103a) sparse-attention prefill indexer.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libidx.so`` (built from ``csrc/`` by ``build.py``).  PyTorch
provides device memory and the current stream.  There is no CPU path: when the
library is missing or the GPU is not an sm_103 part, the calls raise.

Entry points (same names as the C ABI in ``include/idx.h``):
  idx_score_topk            fused score + exact top-k (no [rows, keys] logits)
  idx_score_topk_host       the same on host-memory inputs and output (copies overlap the compute)
  idx_topk_from_scores      exact radix top-k of given fp32 scores
  idx_score_materialise     the two-pass baseline's score pass
  idx_score_topk_mxfp4, idx_score_materialise_mxfp4, idx_mxfp4_to_e4m3
                            the same on MXFP4 inputs (expanded exactly to e4m3)
  idx_score_topk_workspace, idx_topk_workspace, idx_status_string
  idx_add_rmsnorm_quant     residual add + RMS norm to e4m3 rows with scales (k and k_scale)
  idx_prefix_attention      decode attention over a shared prefix and private paged caches
  idx_cache_evict           keep a budget of cached slots by accumulated attention weight
  idx_cache_append_mxfp4    new keys and values into a paged cache in 4 bits
  idx_window_attention_mxfp4
                            attention over that cache: decode steps and prompts, window, sinks
  idx_cache_fork, idx_cache_resize, idx_cache_compact
                            which row of a page table holds which page of a cache
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

__all__ = [
    "IdxError", "Options", "Stats", "load", "idx_score_topk", "idx_score_topk_workspace",
    "idx_score_topk_host", "idx_score_topk_host_workspace",
    "idx_topk_from_scores", "idx_topk_workspace", "idx_score_materialise",
    "idx_status_string", "DTYPES", "STAT_FIELDS", "StageEvents", "idx_launch_count",
    "idx_score_topk_noalloc", "idx_page_table_transform", "idx_route_fused",
    "idx_score_topk_routed", "idx_score_topk_routed_workspace", "idx_mxfp4_to_e4m3",
    "idx_score_topk_mxfp4", "idx_score_materialise_mxfp4", "idx_add_rmsnorm_quant",
    "idx_prefix_attention", "idx_prefix_attention_workspace", "idx_prefix_attention_plan",
    "idx_cache_evict", "idx_cache_evict_workspace", "idx_cache_append_mxfp4",
    "idx_window_attention_mxfp4", "idx_window_attention_mxfp4_workspace",
    "idx_window_attention_mxfp4_plan", "idx_cache_fork",
    "idx_cache_fork_workspace", "idx_cache_resize", "idx_cache_resize_workspace",
    "idx_cache_compact", "idx_cache_compact_workspace",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libidx.so")

IDX_BF16, IDX_FP8_E4M3, IDX_MXFP4 = 1, 2, 3
DTYPES = {torch.bfloat16: IDX_BF16, torch.float8_e4m3fn: IDX_FP8_E4M3}
IDX_FP16, IDX_FP32 = 4, 5  # the serving operators' further types
STAT_FIELDS = ("emit_all_rows", "overflow_rows", "short_rows", "fallback_rows", "max_count",
               "split_rows", "tie_rescan_rows", "reserved")


class IdxError(RuntimeError):
    def __init__(self, fn: str, code: int, text: str):
        super().__init__(f"{fn} failed: {text} (status {code})")
        self.code = code


class Options(ctypes.Structure):
    """Mirror of idx_options."""
    _fields_ = [("cap_factor", ctypes.c_float), ("target_factor", ctypes.c_float),
                ("sample_stride", ctypes.c_int), ("row_split", ctypes.c_int),
                ("d_status", ctypes.c_void_p), ("d_stats", ctypes.c_void_p),
                ("relative_rows", ctypes.c_int), ("test_stall_us", ctypes.c_int),
                ("stage_events", ctypes.c_void_p)]


class Stats:
    """Device counters (idx_stats) plus the device status word."""

    def __init__(self, device=None):
        dev = device or torch.device("cuda", torch.cuda.current_device())
        self.buf = torch.zeros(len(STAT_FIELDS) + 1, dtype=torch.int32, device=dev)

    def reset(self):
        self.buf.zero_()

    @property
    def stats_ptr(self) -> int:
        return self.buf.data_ptr()

    @property
    def status_ptr(self) -> int:
        return self.buf.data_ptr() + 4 * len(STAT_FIELDS)

    def read(self) -> dict:
        v = self.buf.cpu().tolist()
        d = dict(zip(STAT_FIELDS, v[:len(STAT_FIELDS)]))
        d["status"] = v[-1]
        return d


_lib = None


def load(path: str | None = None):
    """Load libidx.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"libidx.so not found at {p}; run "
                          "`python -c 'import __graft_entry__ as g; g.build()'` first")
    lib = ctypes.CDLL(p)
    P, I, LL, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
    lib.idx_score_topk_workspace.argtypes = [I, LL, LL, I, I, I, I, P]
    lib.idx_score_topk_workspace.restype = SZ
    lib.idx_score_topk.argtypes = [P, P, P, P, P, P, I, LL, LL, I, I, I, I, P, P, SZ, P, P]
    lib.idx_score_topk.restype = I
    lib.idx_score_topk_host_workspace.argtypes = [I, LL, LL, I, I, I, I, P]
    lib.idx_score_topk_host_workspace.restype = SZ
    lib.idx_score_topk_host.argtypes = [P, P, P, P, P, P, I, LL, LL, I, I, I, I, P, P, SZ, P, P]
    lib.idx_score_topk_host.restype = I
    lib.idx_topk_workspace.argtypes = [I, LL, I, P]
    lib.idx_topk_workspace.restype = SZ
    lib.idx_topk_from_scores.argtypes = [P, LL, P, P, I, I, P, P, SZ, P, P]
    lib.idx_topk_from_scores.restype = I
    lib.idx_score_materialise.argtypes = [P, P, P, P, P, P, I, LL, I, I, I, P, LL, P, P]
    lib.idx_score_materialise.restype = I
    lib.idx_route_fused.argtypes = [I, LL, I]
    lib.idx_route_fused.restype = I
    lib.idx_score_topk_routed_workspace.argtypes = [I, LL, LL, I, I, I, I, P]
    lib.idx_score_topk_routed_workspace.restype = SZ
    lib.idx_score_topk_routed.argtypes = [P, P, P, P, P, P, I, LL, LL, I, I, I, I, P, P, SZ, P,
                                          P]
    lib.idx_score_topk_routed.restype = I
    lib.idx_page_table_transform.argtypes = [P, I, I, P, I, LL, P, I, P, P]
    lib.idx_page_table_transform.restype = I
    lib.idx_mxfp4_to_e4m3.argtypes = [P, P, LL, I, P, P, P]
    lib.idx_mxfp4_to_e4m3.restype = I
    lib.idx_score_topk_mxfp4_workspace.argtypes = [I, LL, LL, I, I, I, P]
    lib.idx_score_topk_mxfp4_workspace.restype = SZ
    lib.idx_score_topk_mxfp4.argtypes = [P, P, P, P, P, P, P, P, I, LL, LL, I, I, I, P, P, SZ,
                                         P, P]
    lib.idx_score_topk_mxfp4.restype = I
    lib.idx_score_materialise_mxfp4_workspace.argtypes = [I, LL, I, I]
    lib.idx_score_materialise_mxfp4_workspace.restype = SZ
    lib.idx_score_materialise_mxfp4.argtypes = [P, P, P, P, P, P, P, P, I, LL, I, I, P, LL, P,
                                                SZ, P, P]
    lib.idx_score_materialise_mxfp4.restype = I
    F = ctypes.c_float
    lib.idx_add_rmsnorm_quant.argtypes = [P, LL, P, P, I, I, F, I, I, P, P, P, P, P]
    lib.idx_add_rmsnorm_quant.restype = I
    lib.idx_prefix_attention_workspace.argtypes = [I] * 8
    lib.idx_prefix_attention_workspace.restype = SZ
    lib.idx_prefix_attention_plan.argtypes = [I] * 8 + [P]
    lib.idx_prefix_attention_plan.restype = I
    lib.idx_prefix_attention.argtypes = [P] * 7 + [I] * 8 + [LL, I, LL, F, I, P, P, P, P, SZ, P, P]
    lib.idx_prefix_attention.restype = I
    lib.idx_cache_evict_workspace.argtypes = [I] * 4
    lib.idx_cache_evict_workspace.restype = SZ
    lib.idx_cache_evict.argtypes = [P] * 7 + [I] * 5 + [LL, I, LL, I, I, I, I, P, P, P, P, SZ, P, P]
    lib.idx_cache_evict.restype = I
    lib.idx_cache_append_mxfp4.argtypes = [P, LL, P, LL] + [P] * 7 + [I] * 6 + [LL, I, P, P]
    lib.idx_cache_append_mxfp4.restype = I
    lib.idx_window_attention_mxfp4_workspace.argtypes = [I] * 9
    lib.idx_window_attention_mxfp4_workspace.restype = SZ
    lib.idx_window_attention_mxfp4_plan.argtypes = [I] * 9 + [P]
    lib.idx_window_attention_mxfp4_plan.restype = I
    lib.idx_window_attention_mxfp4.argtypes = [P, LL] + [P] * 7 + [I] * 8 + [LL, I, I, I, F, I, P, P, P, SZ, P, P]
    lib.idx_window_attention_mxfp4.restype = I
    lib.idx_cache_fork_workspace.argtypes = [I, LL]
    lib.idx_cache_fork_workspace.restype = SZ
    lib.idx_cache_fork.argtypes = [P] * 4 + [I] * 3 + [LL, P, P, P, P, SZ, P, P]
    lib.idx_cache_fork.restype = I
    lib.idx_cache_resize_workspace.argtypes = [I, I, LL]
    lib.idx_cache_resize_workspace.restype = SZ
    lib.idx_cache_resize.argtypes = [P, P, I] + [P] * 4 + [I] * 3 + [LL, P, P, P, P, SZ, P, P]
    lib.idx_cache_resize.restype = I
    lib.idx_cache_compact_workspace.argtypes = [I, I]
    lib.idx_cache_compact_workspace.restype = SZ
    lib.idx_cache_compact.argtypes = [P, P, I] + [P] * 3 + [I] * 3 + [LL, P, P, P, P, SZ, P, P]
    lib.idx_cache_compact.restype = I
    lib.idx_status_string.argtypes = [I]
    lib.idx_status_string.restype = ctypes.c_char_p
    lib.idx_version.argtypes = []
    lib.idx_version.restype = I
    lib.idx_last_cuda_error.argtypes = []
    lib.idx_last_cuda_error.restype = ctypes.c_char_p
    lib.idx_launch_count.argtypes = []
    lib.idx_launch_count.restype = ctypes.c_ulonglong
    _lib = lib
    return lib


def idx_launch_count() -> int:
    """Kernels launched by libidx in this process so far."""
    return int(load().idx_launch_count())


class StageEvents:
    """CUDA events the library records at its stage boundaries
    (options.stage_events); elapsed(i, j) in ms after a synchronize."""

    def __init__(self, n: int = 5):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(n)]
        for e in self.events:
            e.record()  # torch creates its events lazily, on the first record
        self._arr = (ctypes.c_void_p * n)(*[e.cuda_event for e in self.events])

    @property
    def ptr(self) -> int:
        return ctypes.cast(self._arr, ctypes.c_void_p).value

    def elapsed(self, i: int, j: int) -> float:
        return self.events[i].elapsed_time(self.events[j])


def idx_status_string(code: int) -> str:
    return load().idx_status_string(int(code)).decode()


def _check(fn: str, code: int):
    if code != 0:
        text = idx_status_string(code)
        cuda = load().idx_last_cuda_error().decode() if code in (4, 5) else ""
        raise IdxError(fn, code, f"{text} ({cuda})" if cuda else text)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


class _Launch:
    """The context in which a call on `device` makes what the caller did not bring.  When the call
    was given a stream, that stream is current in it: fills are ordered with the kernels, and the
    memory of what the call drops on return (its workspace) is not handed out again before they
    have ended.  `result` marks a tensor that is returned as used on the caller's stream too."""

    __slots__ = ("context", "caller")

    def __init__(self, stream, device):
        self.caller = self.context = None
        if stream is None:
            return
        if device.type != "cuda":
            raise ValueError("idx: every tensor must live on a CUDA device")
        if not isinstance(stream, torch.cuda.Stream):
            # 0 and 1 are handles of the default stream, which torch keeps as one of its own
            stream = torch.cuda.default_stream(device) if int(stream) in (0, 1) else \
                torch.cuda.ExternalStream(int(stream), device=device)
        if device.index is not None and stream.device != device:
            raise ValueError(f"idx: a stream of {stream.device} for tensors on {device}")
        caller = torch.cuda.current_stream(device)
        if caller.cuda_stream != stream.cuda_stream:
            self.caller, self.context = caller, torch.cuda.stream(stream)

    def __enter__(self):
        if self.context is not None:
            self.context.__enter__()
        return self

    def __exit__(self, *exc):
        if self.context is not None:
            self.context.__exit__(*exc)

    def result(self, t):
        if self.caller is not None:
            t.record_stream(self.caller)
        return t


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _dev(*ts):
    """Check that every tensor is a contiguous CUDA tensor and that all of them
    live on one device; returns that device."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("idx: every tensor must live on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("idx: tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"idx: tensors on different devices ({dev} and {t.device})")
    return dev


def make_options(options: Options | dict | None, stats: Stats | None = None) -> Options | None:
    if options is None and stats is None:
        return None
    o = options if isinstance(options, Options) else Options(**(options or {}))
    if stats is not None:
        o.d_stats = stats.stats_ptr
        o.d_status = stats.status_ptr
    return o


def _opt_ref(o: Options | None):
    return None if o is None else ctypes.byref(o)


def idx_score_topk_workspace(rows: int, keys: int, max_len: int, H: int, D: int, topk: int,
                             dtype, options=None) -> int:
    dt = DTYPES[dtype] if not isinstance(dtype, int) else dtype
    o = make_options(options)
    return int(load().idx_score_topk_workspace(rows, keys, max_len, H, D, topk, dt, _opt_ref(o)))


def idx_score_topk(q, k, k_scale, w, ks, ke, topk: int, *, max_len: int = 0, out=None, ws=None,
                   options=None, stats: Stats | None = None, stream=None):
    """Exact top-k indices [rows, topk] int32 (ascending, -1 padded)."""
    dev = _dev(q, k, k_scale, w, ks, ke, out, ws)
    with torch.cuda.device(dev), _Launch(stream, dev) as on:
        rows, H, D = q.shape
        keys = k.shape[0]
        dt = DTYPES[q.dtype]
        o = make_options(options, stats)
        need = idx_score_topk_workspace(rows, keys, max_len, H, D, topk, dt, o)
        if out is None:
            out = on.result(torch.empty(rows, topk, dtype=torch.int32, device=q.device))
        if ws is None:
            ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
        _check("idx_score_topk", load().idx_score_topk(
            _ptr(q), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(ks), _ptr(ke), rows, keys, max_len, H, D,
            topk, dt, _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _opt_ref(o),
            _stream(stream)))
        return out


def idx_score_topk_host_workspace(rows: int, keys: int, max_len: int, H: int, D: int, topk: int,
                                  dtype, options=None) -> int:
    dt = DTYPES[dtype] if not isinstance(dtype, int) else dtype
    return int(load().idx_score_topk_host_workspace(rows, keys, max_len, H, D, topk, dt,
                                                    _opt_ref(make_options(options))))


def idx_score_topk_host(q, k, k_scale, w, ks, ke, topk: int, *, max_len: int = 0, out=None,
                        ws=None, device=None, options=None, stats: Stats | None = None,
                        stream=None):
    """idx_score_topk on inputs in host memory (CPU tensors; pinned ones let the
    copies overlap the compute): returns the indices [rows, topk] int32 in host
    memory, complete once `stream` is synchronised.  ws is a device uint8
    tensor (allocated on `device`, default the current one, when None)."""
    for t in (q, k, k_scale, w, ks, ke, out):
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise ValueError("idx_score_topk_host: inputs and out are contiguous CPU tensors")
    dev = ws.device if ws is not None else torch.device("cuda", torch.cuda.current_device()) \
        if device is None else torch.device(device)
    if not dev.type == "cuda":
        raise ValueError("idx_score_topk_host: the workspace lives on a CUDA device")
    with torch.cuda.device(dev), _Launch(stream, dev):
        rows, H, D = q.shape
        keys = k.shape[0]
        dt = DTYPES[q.dtype]
        o = make_options(options, stats)
        need = idx_score_topk_host_workspace(rows, keys, max_len, H, D, topk, dt, o)
        if out is None:
            out = torch.empty(rows, topk, dtype=torch.int32, pin_memory=True)
        if ws is None:
            ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        _check("idx_score_topk_host", load().idx_score_topk_host(
            _ptr(q), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(ks), _ptr(ke), rows, keys, max_len, H,
            D, topk, dt, _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _opt_ref(o),
            _stream(stream)))
        return out


def idx_topk_workspace(rows: int, row_stride: int, topk: int, options=None) -> int:
    return int(load().idx_topk_workspace(rows, row_stride, topk, _opt_ref(make_options(options))))


def idx_topk_from_scores(scores, ks, ke, topk: int, *, out=None, ws=None, options=None,
                         stats: Stats | None = None, stream=None):
    """Exact top-k of fp32 scores [rows, row_stride]; ks may be None."""
    dev = _dev(scores, ks, ke, out, ws)
    with torch.cuda.device(dev), _Launch(stream, dev) as on:
        if scores.dtype != torch.float32:
            raise ValueError("idx_topk_from_scores: scores must be float32")
        rows, stride = scores.shape
        o = make_options(options, stats)
        need = int(load().idx_topk_workspace(rows, stride, topk, _opt_ref(o)))
        if out is None:
            out = on.result(torch.empty(rows, topk, dtype=torch.int32, device=scores.device))
        if ws is None and need:
            ws = torch.empty(need, dtype=torch.uint8, device=scores.device)
        nbytes = 0 if ws is None else ws.numel() * ws.element_size()
        _check("idx_topk_from_scores", load().idx_topk_from_scores(
            _ptr(scores), stride, _ptr(ks), _ptr(ke), rows, topk, _ptr(out), _ptr(ws), nbytes,
            _opt_ref(o), _stream(stream)))
        return out


def idx_score_materialise(q, k, k_scale, w, ks, ke, *, out=None, row_stride: int | None = None,
                          options=None, stats: Stats | None = None, stream=None):
    """fp32 scores [rows, row_stride]; row r's key j at column j - ks[r]."""
    dev = _dev(q, k, k_scale, w, ks, ke, out)
    with torch.cuda.device(dev), _Launch(stream, dev) as on:
        rows, H, D = q.shape
        keys = k.shape[0]
        if out is None:
            stride = row_stride or keys
            out = on.result(torch.empty(rows, stride, dtype=torch.float32, device=q.device))
        stride = out.shape[1]
        o = make_options(options, stats)
        _check("idx_score_materialise", load().idx_score_materialise(
            _ptr(q), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(ks), _ptr(ke), rows, keys, H, D,
            DTYPES[q.dtype], _ptr(out), stride, _opt_ref(o), _stream(stream)))
        return out


def _mx_shapes(q, q_sf, k, k_sf):
    """rows, H, D of MXFP4 q [rows, H, D/2] uint8 with q_sf [rows, H, D/32] and k
    [keys, D/2] with k_sf [keys, D/32]."""
    for t in (q, q_sf, k, k_sf):
        if t.dtype != torch.uint8:
            raise ValueError("MXFP4 elements and scales are uint8 tensors")
    rows, H, half = q.shape
    D = 2 * half
    if q_sf.shape != (rows, H, D // 32) or k.shape[1] != half or \
            k_sf.shape != (k.shape[0], D // 32):
        raise ValueError("inconsistent MXFP4 shapes")
    return rows, H, D


def idx_mxfp4_to_e4m3(x, sf, *, out=None, options=None, stats: Stats | None = None,
                      stream=None):
    """MXFP4 rows x [n, D/2] + sf [n, D/32] -> e4m3 [n, D] (exact within the
    e4m3 range, else IDX_DEV_RANGE)."""
    dev = _dev(x, sf, out)
    with torch.cuda.device(dev), _Launch(stream, dev) as on:
        n, half = x.shape[0], x.shape[-1]
        D = 2 * half
        if out is None:
            out = on.result(torch.empty(*x.shape[:-1], D, dtype=torch.float8_e4m3fn,
                                        device=x.device))
        o = make_options(options, stats)
        _check("idx_mxfp4_to_e4m3", load().idx_mxfp4_to_e4m3(
            _ptr(x), _ptr(sf), x.numel() // half, D, _ptr(out), _opt_ref(o), _stream(stream)))
        return out


def idx_score_topk_mxfp4(q, q_sf, k, k_sf, k_scale, w, ks, ke, topk: int, *, max_len: int = 0,
                         out=None, ws=None, options=None, stats: Stats | None = None,
                         stream=None):
    """idx_score_topk on MXFP4 q/k (with their e8m0 block scales)."""
    dev = _dev(q, q_sf, k, k_sf, k_scale, w, ks, ke, out, ws)
    with torch.cuda.device(dev), _Launch(stream, dev) as on:
        rows, H, D = _mx_shapes(q, q_sf, k, k_sf)
        keys = k.shape[0]
        o = make_options(options, stats)
        need = int(load().idx_score_topk_mxfp4_workspace(rows, keys, max_len, H, D, topk,
                                                         _opt_ref(o)))
        if out is None:
            out = on.result(torch.empty(rows, topk, dtype=torch.int32, device=q.device))
        if ws is None:
            ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
        _check("idx_score_topk_mxfp4", load().idx_score_topk_mxfp4(
            _ptr(q), _ptr(q_sf), _ptr(k), _ptr(k_sf), _ptr(k_scale), _ptr(w), _ptr(ks), _ptr(ke),
            rows, keys, max_len, H, D, topk, _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
            _opt_ref(o), _stream(stream)))
        return out


def idx_score_materialise_mxfp4(q, q_sf, k, k_sf, k_scale, w, ks, ke, *, out=None,
                                row_stride: int | None = None, ws=None, options=None,
                                stats: Stats | None = None, stream=None):
    """idx_score_materialise on MXFP4 q/k (with their e8m0 block scales)."""
    dev = _dev(q, q_sf, k, k_sf, k_scale, w, ks, ke, out, ws)
    with torch.cuda.device(dev), _Launch(stream, dev) as on:
        rows, H, D = _mx_shapes(q, q_sf, k, k_sf)
        keys = k.shape[0]
        if out is None:
            out = on.result(torch.empty(rows, row_stride or keys, dtype=torch.float32,
                                        device=q.device))
        need = int(load().idx_score_materialise_mxfp4_workspace(rows, keys, H, D))
        if ws is None:
            ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
        o = make_options(options, stats)
        _check("idx_score_materialise_mxfp4", load().idx_score_materialise_mxfp4(
            _ptr(q), _ptr(q_sf), _ptr(k), _ptr(k_sf), _ptr(k_scale), _ptr(w), _ptr(ks), _ptr(ke),
            rows, keys, H, D, _ptr(out), out.shape[1], _ptr(ws), ws.numel() * ws.element_size(),
            _opt_ref(o), _stream(stream)))
        return out


def idx_score_topk_noalloc(q, k, k_scale, w, ks, ke, topk: int, *, max_len: int = 0, out=None,
                           options=None, stats: Stats | None = None, stream=None):
    """idx_score_topk on the library's built-in scratch array (no workspace,
    no allocation by the library; out is allocated here when not given)."""
    dev = _dev(q, k, k_scale, w, ks, ke, out)
    with torch.cuda.device(dev), _Launch(stream, dev) as on:
        lib = load()
        fn = lib.idx_score_topk_noalloc
        P, I, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
        fn.argtypes = [P, P, P, P, P, P, I, LL, LL, I, I, I, I, P, P, P]
        fn.restype = I
        rows, H, D = q.shape
        if out is None:
            out = on.result(torch.empty(rows, topk, dtype=torch.int32, device=q.device))
        o = make_options(options, stats)
        _check("idx_score_topk_noalloc", fn(
            _ptr(q), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(ks), _ptr(ke), rows, k.shape[0], max_len,
            H, D, topk, DTYPES[q.dtype], _ptr(out), _opt_ref(o), _stream(stream)))
        return out


def idx_page_table_transform(idx, table, page_size: int = 64, *, row_map=None, options=None,
                             stats: Stats | None = None, stream=None):
    """In place: every position p >= 0 of idx [rows, topk] int32 becomes
    table[t, p // page_size] * page_size + p % page_size (t = row_map[r] or r);
    -1 entries stay.  Returns idx."""
    dev = _dev(idx, table, row_map)
    with torch.cuda.device(dev):
        if idx.dtype != torch.int32 or table.dtype != torch.int32:
            raise ValueError("idx_page_table_transform: idx and table must be int32")
        if row_map is not None and row_map.dtype != torch.int32:
            raise ValueError("idx_page_table_transform: row_map must be int32")
        rows, topk = idx.shape
        o = make_options(options, stats)
        _check("idx_page_table_transform", load().idx_page_table_transform(
            _ptr(idx), rows, topk, _ptr(table), table.shape[0], table.shape[1], _ptr(row_map),
            page_size, _opt_ref(o), _stream(stream)))
        return idx


def idx_route_fused(rows: int, max_len: int, topk: int) -> bool:
    """The routing gate: True when a call of `rows` rows whose longest row sees
    max_len keys takes the fused path."""
    return bool(load().idx_route_fused(rows, max_len, topk))


def idx_score_topk_routed_workspace(rows: int, keys: int, max_len: int, H: int, D: int,
                                    topk: int, dtype, options=None) -> int:
    dt = DTYPES[dtype] if not isinstance(dtype, int) else dtype
    o = make_options(options)
    return int(load().idx_score_topk_routed_workspace(rows, keys, max_len, H, D, topk, dt,
                                                      _opt_ref(o)))


def idx_score_topk_routed(q, k, k_scale, w, ks, ke, topk: int, *, max_len: int = 0, out=None,
                          ws=None, options=None, stats: Stats | None = None, stream=None):
    """idx_score_topk by the faster path for the longest row (fused, or the
    logits then their top-k); the same indices either way."""
    dev = _dev(q, k, k_scale, w, ks, ke, out, ws)
    with torch.cuda.device(dev), _Launch(stream, dev) as on:
        rows, H, D = q.shape
        keys = k.shape[0]
        dt = DTYPES[q.dtype]
        o = make_options(options, stats)
        need = int(load().idx_score_topk_routed_workspace(rows, keys, max_len, H, D, topk, dt,
                                                          _opt_ref(o)))
        if out is None:
            out = on.result(torch.empty(rows, topk, dtype=torch.int32, device=q.device))
        if ws is None:
            ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
        _check("idx_score_topk_routed", load().idx_score_topk_routed(
            _ptr(q), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(ks), _ptr(ke), rows, keys, max_len, H, D,
            topk, dt, _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _opt_ref(o),
            _stream(stream)))
        return out


# The serving operators are called per layer and token, so the checks of their tensors and the
# calls themselves are a small C++ module (csrc/serve_binding.cpp); what is left here is the
# allocation of the outputs that the caller did not bring.
_serve_module = None


def _serve():
    """The binding module, on the functions of the loaded libidx."""
    global _serve_module
    if _serve_module is None:
        lib = load()
        p = os.path.join(_HERE, "_build", "_serve.so")
        if not os.path.exists(p):
            raise ImportError(f"_serve.so not found at {p}; run "
                              "`python -c 'import __graft_entry__ as g; g.build()'` first")
        loader = importlib.machinery.ExtensionFileLoader("_serve", p)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_serve", loader))
        loader.exec_module(module)
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.idx_add_rmsnorm_quant, lib.idx_prefix_attention, lib.idx_cache_evict)))
        module.bind_cache(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.idx_cache_append_mxfp4, lib.idx_window_attention_mxfp4, lib.idx_cache_fork,
            lib.idx_cache_resize, lib.idx_cache_compact)))
        _serve_module = module
    return _serve_module


def _serve_call(fn: str, f, args, options, stats, stream):
    o = None
    if options is not None or stats is not None:
        o = make_options(options, stats)
    if isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    code = f(*args, None if o is None else ctypes.addressof(o), stream)
    if code:
        _check(fn, code)


def idx_add_rmsnorm_quant(x, weight, *, residual=None, residual_out=None, eps: float = 1e-6,
                          group: int = 0, out=None, scale=None, options=None,
                          stats: Stats | None = None, stream=None):
    """RMS norm of x (+ residual) [rows, N] to e4m3: (out [rows, N] e4m3, scale fp32
    [rows] or, with group 32, 64 or 128, [rows, N // group]).  x may be a column
    slice of a wider tensor.  residual_out receives x + residual in x's type."""
    fn = "idx_add_rmsnorm_quant"
    if out is None or scale is None:
        if x.dim() != 2:
            raise ValueError(f"{fn}: x must be [rows, N] with adjacent columns")
        rows, N = x.shape
        with _Launch(stream, x.device) as on:
            if out is None:
                out = on.result(torch.empty(rows, N, dtype=torch.float8_e4m3fn, device=x.device))
            if scale is None:
                scale = on.result(torch.empty((rows, N // group) if group > 0 else (rows,),
                                              dtype=torch.float32, device=x.device))
    _serve_call(fn, _serve().add_rmsnorm_quant, (
        x, weight, residual, residual_out, eps, group, out, scale), options, stats, stream)
    return out, scale


def idx_prefix_attention_workspace(B: int, Q: int, Hq: int, Hkv: int, D: int, prefix_len: int,
                                   max_len: int, weights: bool) -> int:
    return int(load().idx_prefix_attention_workspace(B, Q, Hq, Hkv, D, prefix_len, max_len,
                                                     int(bool(weights))))


def idx_prefix_attention_plan(B: int, Q: int, Hq: int, Hkv: int, D: int, prefix_len: int,
                              max_len: int, weights: bool) -> dict:
    """The parts that such a call is cut into: prefix_parts of prefix_keys keys each, private_parts
    of private_keys, and whether the private ones take the tensor cores' dense path."""
    plan = (ctypes.c_int * 5)()
    _check("idx_prefix_attention_plan", load().idx_prefix_attention_plan(
        B, Q, Hq, Hkv, D, prefix_len, max_len, int(bool(weights)), plan))
    return dict(prefix_parts=plan[0], prefix_keys=plan[1], private_parts=plan[2],
                private_keys=plan[3], private_dense=bool(plan[4]))


def idx_prefix_attention(q, k_cache, v_cache, table, lens, *, prefix_table=None,
                         prefix_len: int = 0, max_len: int = 0, scale: float | None = None,
                         weights=None, weights_out=None, out=None, lse=None, ws=None,
                         options=None, stats: Stats | None = None, stream=None):
    """Decode attention of q [B, Q, Hq, D] over a shared prefix (prefix_table) and each
    request's own pages (table [B, P], lens [B]) of k_cache, v_cache
    [pages, Hkv, page_size, D]: (out, lse [B, Q, Hq]), and weights_out when weights
    [B, Hkv, slots] (what each private slot has gathered) is given."""
    fn = "idx_prefix_attention"
    if out is None or lse is None or ws is None:
        if q.dim() != 4 or k_cache.dim() != 4 or table.dim() != 2:
            raise ValueError(f"{fn}: q [B, Q, Hq, D], caches [pages, Hkv, page_size, D], "
                             "table [B, P]")
        B, Q, Hq, D = q.shape
        with _Launch(stream, q.device) as on:
            if out is None:
                out = on.result(torch.empty_like(q))
            if lse is None:
                lse = on.result(torch.empty(B, Q, Hq, dtype=torch.float32, device=q.device))
            if ws is None:
                Hkv, page_size = k_cache.shape[1:3]
                need = idx_prefix_attention_workspace(
                    B, Q, Hq, Hkv, D, prefix_len, max_len or table.shape[1] * page_size,
                    weights is not None) if Hkv and Hq % Hkv == 0 else 0
                ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    if weights is not None and weights_out is None:
        with _Launch(stream, q.device) as on:
            weights_out = on.result(torch.zeros_like(weights))
    _serve_call(fn, _serve().prefix_attention, (
        q, k_cache, v_cache, table, lens, prefix_table, prefix_len, max_len, scale, weights,
        weights_out, out, lse, ws), options, stats, stream)
    return (out, lse) if weights is None else (out, lse, weights_out)


def idx_cache_evict_workspace(B: int, Hkv: int, budget: int, max_len: int) -> int:
    return int(load().idx_cache_evict_workspace(B, Hkv, budget, max_len))


def idx_cache_evict(k_cache, v_cache, table, lens, weights, positions, next_pos, budget: int, *,
                    recent: int = 0, sink: int = 0, max_len: int = 0, lens_out=None,
                    weights_out=None, positions_out=None, ws=None, options=None,
                    stats: Stats | None = None, stream=None):
    """Keep the `budget` best slots of every (request, key head) by weights
    [B, Hkv, slots], protecting positions < sink and >= next_pos - recent; the K/V rows
    that move do so in place.  Returns (lens_out, weights_out, positions_out);
    weights_out and positions_out may be the inputs themselves."""
    fn = "idx_cache_evict"
    if lens_out is None or weights_out is None or positions_out is None or ws is None:
        if k_cache.dim() != 4 or table.dim() != 2:
            raise ValueError(f"{fn}: caches [pages, Hkv, page_size, D], table [B, P], weights "
                             "[B, Hkv, slots]")
        with _Launch(stream, lens.device) as on:
            if lens_out is None:
                lens_out = on.result(torch.empty_like(lens))
            if weights_out is None:
                weights_out = on.result(torch.zeros_like(weights))
            if positions_out is None:
                positions_out = on.result(torch.full_like(positions, -1))
            if ws is None:
                need = idx_cache_evict_workspace(table.shape[0], k_cache.shape[1], budget,
                                                 max_len or table.shape[1] * k_cache.shape[2])
                ws = torch.empty(max(256, need), dtype=torch.uint8, device=lens.device)
    _serve_call(fn, _serve().cache_evict, (
        k_cache, v_cache, table, lens, weights, positions, next_pos, budget, recent, sink, max_len,
        lens_out, weights_out, positions_out, ws), options, stats, stream)
    return lens_out, weights_out, positions_out


def idx_cache_append_mxfp4(k, v, k_codes, k_sf, v_codes, v_sf, table, lens, *, q_start=None,
                           options=None, stats: Stats | None = None, stream=None) -> None:
    """Write the new tokens' k, v [T, Hkv, D] (slices of a wider projection may be given) into a
    paged MXFP4 cache: codes [pages, Hkv, page_size, D // 2] and scales [..., D // 32] uint8.
    lens [B] counts the new tokens, whose slots they take whatever those hold; q_start [B + 1] says
    which are whose (None: T / B each)."""
    _serve_call("idx_cache_append_mxfp4", _serve().cache_append_mxfp4, (
        k, v, k_codes, k_sf, v_codes, v_sf, table, lens, q_start), options, stats, stream)


def idx_window_attention_mxfp4_workspace(B: int, T: int, max_q: int, Hq: int, Hkv: int, D: int,
                                         max_len: int, window: int, sink: int) -> int:
    return int(load().idx_window_attention_mxfp4_workspace(B, T, max_q, Hq, Hkv, D, max_len,
                                                           window, sink))


def idx_window_attention_mxfp4_plan(B: int, T: int, max_q: int, Hq: int, Hkv: int, D: int,
                                    max_len: int, window: int, sink: int) -> dict:
    """How such a call is cut: splits of the keys that a tile of rows sees, keys each, whether the
    rows take the tensor cores' dense path, and the most rows of a tile."""
    plan = (ctypes.c_int * 4)()
    _check("idx_window_attention_mxfp4_plan", load().idx_window_attention_mxfp4_plan(
        B, T, max_q, Hq, Hkv, D, max_len, window, sink, plan))
    return dict(splits=plan[0], keys=plan[1], dense=bool(plan[2]), rows=plan[3])


def idx_window_attention_mxfp4(q, k_codes, k_sf, v_codes, v_sf, table, lens, *, q_start=None,
                               max_q: int = 0, max_len: int = 0, window: int = 0, sink: int = 0,
                               scale: float | None = None, out=None, lse=None, ws=None,
                               options=None, stats: Stats | None = None, stream=None):
    """Causal attention of the new tokens' q [T, Hq, D] over each request's slots of a paged MXFP4
    cache: (out [T, Hq, D], lse [T, Hq]).  With a window, a token sees the `window` newest slots
    up to its own and the first `sink` ones.  max_q bounds a request's new tokens, max_len its
    slots.  An out that is allocated here is 0 for tokens outside every request."""
    fn = "idx_window_attention_mxfp4"
    if out is None or lse is None or ws is None:
        if q.dim() != 3 or k_codes.dim() != 4 or table.dim() != 2:
            raise ValueError(f"{fn}: q [T, Hq, D], codes [pages, Hkv, page_size, D // 2], "
                             "table [B, P]")
        T, Hq, D = q.shape
        make = torch.empty if q_start is None else torch.zeros
        with _Launch(stream, q.device) as on:
            if out is None:
                out = on.result(make(T, Hq, D, dtype=q.dtype, device=q.device))
            if lse is None:
                lse = on.result(make(T, Hq, dtype=torch.float32, device=q.device))
            if ws is None:
                need = idx_window_attention_mxfp4_workspace(
                    table.shape[0], T, max_q, Hq, k_codes.shape[1], D,
                    max_len or min(table.shape[1] * k_codes.shape[2], 0x7fffffff), window, sink)
                ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _serve_call(fn, _serve().window_attention_mxfp4, (
        q, k_codes, k_sf, v_codes, v_sf, table, lens, q_start, max_q, max_len, window, sink, scale,
        out, lse, ws), options, stats, stream)
    return out, lse


def idx_cache_fork_workspace(B: int, width: int) -> int:
    return int(load().idx_cache_fork_workspace(B, width))


def idx_cache_fork(refs, table, lens, parent, *, page_size: int, refs_out=None, table_out=None,
                   lens_out=None, ws=None, options=None, stats: Stats | None = None, stream=None):
    """Row i of the page table takes over the pages and the length of row parent[i] (i: stays, -1:
    ends), all rows at once; refs [pages] counts the entries that name a page.  Returns
    (refs_out, table_out, lens_out), each of which may be its input: a call in place takes a
    workspace."""
    fn = "idx_cache_fork"
    in_place = ws is None and (table_out is table or lens_out is lens)
    if in_place or refs_out is None or table_out is None or lens_out is None:
        with _Launch(stream, refs.device) as on:
            refs_out, table_out, lens_out = _page_results(on, fn, refs, refs_out, table, table_out,
                                                          lens, lens_out)
            if in_place:
                ws = torch.empty(max(256, idx_cache_fork_workspace(*table.shape)),
                                 dtype=torch.uint8, device=refs.device)
    _serve_call(fn, _serve().cache_fork, (
        refs, table, lens, parent, page_size, refs_out, table_out, lens_out, ws), options, stats,
        stream)
    return refs_out, table_out, lens_out


def _page_results(on, fn, refs, refs_out, table, table_out, lens, lens_out):
    """What a call on pages writes, where the caller did not bring it."""
    if refs.dim() != 1 or table.dim() != 2:
        raise ValueError(f"{fn}: refs [pages], table [B, P]")
    if refs_out is None:
        refs_out = on.result(torch.empty_like(refs))
    if table_out is None:
        table_out = on.result(torch.full_like(table, -1))
    if lens_out is None:
        lens_out = on.result(torch.empty_like(lens))
    return refs_out, table_out, lens_out


def idx_cache_resize_workspace(B: int, pages: int, width: int) -> int:
    return int(load().idx_cache_resize_workspace(B, pages, width))


def idx_cache_resize(caches, refs, table, lens, new_lens, *, page_size: int, refs_out=None,
                     table_out=None, lens_out=None, ws=None, options=None,
                     stats: Stats | None = None, stream=None):
    """Rows of the page table go from lens to new_lens slots: they give pages back and take free
    ones (refs 0, lowest first), and a row that grows into a page which others hold too takes a
    copy of it in every one of `caches` ([pages, ...] tensors).  Returns (refs_out, table_out,
    lens_out), each of which may be its input; lens_out tells where the pages did not suffice.  An
    append after it takes torch.where(lens_out == new_lens, lens_out, 0): a row that was not served
    has no slots for its new tokens."""
    fn = "idx_cache_resize"
    if refs_out is None or table_out is None or lens_out is None or ws is None:
        with _Launch(stream, refs.device) as on:
            refs_out, table_out, lens_out = _page_results(on, fn, refs, refs_out, table, table_out,
                                                          lens, lens_out)
            if ws is None:
                need = idx_cache_resize_workspace(table.shape[0], refs.shape[0], table.shape[1])
                ws = torch.empty(max(256, need), dtype=torch.uint8, device=refs.device)
    _serve_call(fn, _serve().cache_resize, (
        caches, refs, table, lens, new_lens, page_size, refs_out, table_out, lens_out, ws), options,
        stats, stream)
    return refs_out, table_out, lens_out


def idx_cache_compact_workspace(B: int, pages: int) -> int:
    return int(load().idx_cache_compact_workspace(B, pages))


def idx_cache_compact(caches, refs, table, lens, *, page_size: int, refs_out=None, table_out=None,
                      live=None, ws=None, options=None, stats: Stats | None = None, stream=None):
    """Move the live pages (refs above 0) of `caches` ([pages, ...] tensors) to the front, in
    place; returns (refs_out, table_out, live [1]), the first two may be their inputs."""
    fn = "idx_cache_compact"
    if refs_out is None or table_out is None or live is None or ws is None:
        with _Launch(stream, refs.device) as on:
            refs_out, table_out, _ = _page_results(on, fn, refs, refs_out, table, table_out, lens,
                                                   lens)
            if live is None:
                live = on.result(torch.empty(1, dtype=torch.int32, device=refs.device))
            if ws is None:
                need = idx_cache_compact_workspace(table.shape[0], refs.shape[0])
                ws = torch.empty(max(256, need), dtype=torch.uint8, device=refs.device)
    _serve_call(fn, _serve().cache_compact, (
        caches, refs, table, lens, page_size, refs_out, table_out, live, ws), options, stats,
        stream)
    return refs_out, table_out, live
