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
"""
from __future__ import annotations

import ctypes
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
    "idx_prefix_attention", "idx_prefix_attention_workspace", "idx_cache_evict",
    "idx_cache_evict_workspace",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libidx.so")

IDX_BF16, IDX_FP8_E4M3, IDX_MXFP4 = 1, 2, 3
DTYPES = {torch.bfloat16: IDX_BF16, torch.float8_e4m3fn: IDX_FP8_E4M3}
IDX_FP16, IDX_FP32 = 4, 5
# the serving operators' types (the indexer's own are DTYPES)
SERVE_DTYPES = {torch.bfloat16: IDX_BF16, torch.float16: IDX_FP16, torch.float32: IDX_FP32}
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
    lib.idx_prefix_attention.argtypes = [P] * 7 + [I] * 8 + [LL, I, LL, F, I, P, P, P, P, SZ, P, P]
    lib.idx_prefix_attention.restype = I
    lib.idx_cache_evict_workspace.argtypes = [I] * 4
    lib.idx_cache_evict_workspace.restype = SZ
    lib.idx_cache_evict.argtypes = [P] * 7 + [I] * 5 + [LL, I, LL, I, I, I, I, P, P, P, P, SZ, P, P]
    lib.idx_cache_evict.restype = I
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
    with torch.cuda.device(dev):
        rows, H, D = q.shape
        keys = k.shape[0]
        dt = DTYPES[q.dtype]
        o = make_options(options, stats)
        need = idx_score_topk_workspace(rows, keys, max_len, H, D, topk, dt, o)
        if out is None:
            out = torch.empty(rows, topk, dtype=torch.int32, device=q.device)
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
    with torch.cuda.device(dev):
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
    with torch.cuda.device(dev):
        if scores.dtype != torch.float32:
            raise ValueError("idx_topk_from_scores: scores must be float32")
        rows, stride = scores.shape
        o = make_options(options, stats)
        need = int(load().idx_topk_workspace(rows, stride, topk, _opt_ref(o)))
        if out is None:
            out = torch.empty(rows, topk, dtype=torch.int32, device=scores.device)
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
    with torch.cuda.device(dev):
        rows, H, D = q.shape
        keys = k.shape[0]
        if out is None:
            stride = row_stride or keys
            out = torch.empty(rows, stride, dtype=torch.float32, device=q.device)
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
    with torch.cuda.device(dev):
        n, half = x.shape[0], x.shape[-1]
        D = 2 * half
        if out is None:
            out = torch.empty(*x.shape[:-1], D, dtype=torch.float8_e4m3fn, device=x.device)
        o = make_options(options, stats)
        _check("idx_mxfp4_to_e4m3", load().idx_mxfp4_to_e4m3(
            _ptr(x), _ptr(sf), x.numel() // half, D, _ptr(out), _opt_ref(o), _stream(stream)))
        return out


def idx_score_topk_mxfp4(q, q_sf, k, k_sf, k_scale, w, ks, ke, topk: int, *, max_len: int = 0,
                         out=None, ws=None, options=None, stats: Stats | None = None,
                         stream=None):
    """idx_score_topk on MXFP4 q/k (with their e8m0 block scales)."""
    dev = _dev(q, q_sf, k, k_sf, k_scale, w, ks, ke, out, ws)
    with torch.cuda.device(dev):
        rows, H, D = _mx_shapes(q, q_sf, k, k_sf)
        keys = k.shape[0]
        o = make_options(options, stats)
        need = int(load().idx_score_topk_mxfp4_workspace(rows, keys, max_len, H, D, topk,
                                                         _opt_ref(o)))
        if out is None:
            out = torch.empty(rows, topk, dtype=torch.int32, device=q.device)
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
    with torch.cuda.device(dev):
        rows, H, D = _mx_shapes(q, q_sf, k, k_sf)
        keys = k.shape[0]
        if out is None:
            out = torch.empty(rows, row_stride or keys, dtype=torch.float32, device=q.device)
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
    with torch.cuda.device(dev):
        lib = load()
        fn = lib.idx_score_topk_noalloc
        P, I, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
        fn.argtypes = [P, P, P, P, P, P, I, LL, LL, I, I, I, I, P, P, P]
        fn.restype = I
        rows, H, D = q.shape
        if out is None:
            out = torch.empty(rows, topk, dtype=torch.int32, device=q.device)
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
    with torch.cuda.device(dev):
        rows, H, D = q.shape
        keys = k.shape[0]
        dt = DTYPES[q.dtype]
        o = make_options(options, stats)
        need = int(load().idx_score_topk_routed_workspace(rows, keys, max_len, H, D, topk, dt,
                                                          _opt_ref(o)))
        if out is None:
            out = torch.empty(rows, topk, dtype=torch.int32, device=q.device)
        if ws is None:
            ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
        _check("idx_score_topk_routed", load().idx_score_topk_routed(
            _ptr(q), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(ks), _ptr(ke), rows, keys, max_len, H, D,
            topk, dt, _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _opt_ref(o),
            _stream(stream)))
        return out


# The serving operators are called per layer and token, so their bindings keep the host's
# part short: one pass over the tensors, and the device switched only when it differs.

# the current stream's handle without a Stream object (a microsecond less), where torch has it
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _raw_stream(stream, index: int) -> int:
    if stream is None:
        return _current_handle(index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _serve_device(fn: str, *ts) -> int:
    """The index of the one CUDA device that every tensor (all contiguous) lives on."""
    index = None
    for t in ts:
        if t is None:
            continue
        i = t.get_device()
        if i == index:
            if t.is_contiguous():
                continue
        else:
            if i < 0:
                raise ValueError(f"{fn}: every tensor must live on a CUDA device")
            if index is not None:
                raise ValueError(f"{fn}: tensors on different devices (cuda:{index} and cuda:{i})")
            index = i
        if not t.is_contiguous():
            raise ValueError(f"{fn}: tensors must be contiguous")
    return index


def _serve_call(fn: str, f, index: int, args, options, stats, stream):
    """f(*args, options, stream) with the tensors' device current."""
    o = None
    if options is not None or stats is not None:
        o = _opt_ref(make_options(options, stats))
    if torch.cuda.current_device() == index:
        code = f(*args, o, _raw_stream(stream, index))
    else:
        with torch.cuda.device(index):
            code = f(*args, o, _raw_stream(stream, index))
    if code:
        _check(fn, code)


def _serve_dtype(fn: str, *ts):
    """The one element type of the tensors, as the C ABI names it."""
    dtype = ts[0].dtype
    for t in ts:
        if t is not None and t.dtype is not dtype:
            raise ValueError(f"{fn}: {t.dtype} and {dtype} tensors where one type is needed")
    if dtype not in SERVE_DTYPES:
        raise ValueError(f"{fn}: unsupported type {dtype}")
    return SERVE_DTYPES[dtype]


def _expect(fn: str, name: str, t, dtype, shape):
    if t is not None and (t.dtype is not dtype or t.shape != shape):
        raise ValueError(f"{fn}: {name} must be {dtype} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")


def idx_add_rmsnorm_quant(x, weight, *, residual=None, residual_out=None, eps: float = 1e-6,
                          group: int = 0, out=None, scale=None, options=None,
                          stats: Stats | None = None, stream=None):
    """RMS norm of x (+ residual) [rows, N] to e4m3: (out [rows, N] e4m3, scale fp32
    [rows] or, with group 32, 64 or 128, [rows, N // group]).  x may be a column
    slice of a wider tensor.  residual_out receives x + residual in x's type."""
    fn = "idx_add_rmsnorm_quant"
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError(f"{fn}: x must be [rows, N] with adjacent columns")
    rows, N = x.shape
    x_stride = x.stride(0) if rows > 1 else max(N, x.stride(0))
    index = _serve_device(fn, weight, residual, residual_out, out, scale)
    if x.get_device() != index:
        raise ValueError(f"{fn}: x is not on cuda:{index}, the other tensors' device")
    dt = _serve_dtype(fn, x, weight, residual, residual_out)
    _expect(fn, "weight", weight, x.dtype, (N,))
    _expect(fn, "residual", residual, x.dtype, (rows, N))
    _expect(fn, "residual_out", residual_out, x.dtype, (rows, N))
    if group < 0 or (group and N % group):
        raise ValueError(f"{fn}: {N} columns are not whole groups of {group}")
    scales = (rows, N // group) if group else (rows,)
    if out is None:
        out = torch.empty(rows, N, dtype=torch.float8_e4m3fn, device=x.device)
    else:
        _expect(fn, "out", out, torch.float8_e4m3fn, (rows, N))
    if scale is None:
        scale = torch.empty(scales, dtype=torch.float32, device=x.device)
    else:
        _expect(fn, "scale", scale, torch.float32, scales)
    _serve_call(fn, load().idx_add_rmsnorm_quant, index, (
        x.data_ptr(), x_stride, _ptr(residual), weight.data_ptr(), rows, N, eps, group, dt,
        _ptr(residual_out), out.data_ptr(), scale.data_ptr()), options, stats, stream)
    return out, scale


def idx_prefix_attention_workspace(B: int, Q: int, Hq: int, Hkv: int, D: int, prefix_len: int,
                                   max_len: int, weights: bool) -> int:
    return int(load().idx_prefix_attention_workspace(B, Q, Hq, Hkv, D, prefix_len, max_len,
                                                     int(bool(weights))))


def idx_prefix_attention(q, k_cache, v_cache, table, lens, *, prefix_table=None,
                         prefix_len: int = 0, max_len: int = 0, scale: float | None = None,
                         weights=None, weights_out=None, out=None, lse=None, ws=None,
                         options=None, stats: Stats | None = None, stream=None):
    """Decode attention of q [B, Q, Hq, D] over a shared prefix (prefix_table) and each
    request's own pages (table [B, P], lens [B]) of k_cache, v_cache
    [pages, Hkv, page_size, D]: (out, lse [B, Q, Hq]), and weights_out when weights
    [B, Hkv, slots] (what each private slot has gathered) is given."""
    fn = "idx_prefix_attention"
    index = _serve_device(fn, q, k_cache, v_cache, table, lens, prefix_table, weights,
                          weights_out, out, lse, ws)
    dt = _serve_dtype(fn, q, k_cache, v_cache)
    cache = k_cache.shape
    if q.dim() != 4 or len(cache) != 4 or cache != v_cache.shape or table.dim() != 2:
        raise ValueError(f"{fn}: q [B, Q, Hq, D], caches [pages, Hkv, page_size, D], table [B, P]")
    B, Q, Hq, D = q.shape
    pages, Hkv, page_size, cache_d = cache
    if cache_d != D:
        raise ValueError(f"{fn}: q has {D} dimensions, the caches {cache_d}")
    width = table.shape[1]
    _expect(fn, "table", table, torch.int32, (B, width))
    _expect(fn, "lens", lens, torch.int32, (B,))
    if prefix_len > 0 and (prefix_table is None or prefix_table.dtype is not torch.int32 or
                           prefix_table.numel() * page_size < prefix_len):
        raise ValueError(f"{fn}: prefix_table must be int32 and cover prefix_len")
    slots = 0
    if weights is not None:
        if weights.dim() != 3 or weights.dtype is not torch.float32 or \
                weights.shape[:2] != (B, Hkv):
            raise ValueError(f"{fn}: weights must be float32 [B, Hkv, slots]")
        slots = weights.shape[2]
        if weights_out is None:
            weights_out = torch.zeros_like(weights)
        else:
            _expect(fn, "weights_out", weights_out, torch.float32, (B, Hkv, slots))
    elif weights_out is not None:
        raise ValueError(f"{fn}: weights_out without weights")
    if out is None:
        out = torch.empty_like(q)
    else:
        _expect(fn, "out", out, q.dtype, q.shape)
    if lse is None:
        lse = torch.empty(B, Q, Hq, dtype=torch.float32, device=q.device)
    else:
        _expect(fn, "lse", lse, torch.float32, (B, Q, Hq))
    if ws is None:
        need = idx_prefix_attention_workspace(
            B, Q, Hq, Hkv, D, prefix_len, max_len or width * page_size,
            weights is not None) if Hq % Hkv == 0 else 0
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _serve_call(fn, load().idx_prefix_attention, index, (
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _ptr(prefix_table),
        table.data_ptr(), lens.data_ptr(), _ptr(weights), B, Q, Hq, Hkv, D, pages, page_size,
        prefix_len, width, max_len, slots, D ** -0.5 if scale is None else scale, dt,
        out.data_ptr(), lse.data_ptr(), _ptr(weights_out), ws.data_ptr(), ws.nbytes),
        options, stats, stream)
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
    index = _serve_device(fn, k_cache, v_cache, table, lens, weights, positions, next_pos,
                          lens_out, weights_out, positions_out, ws)
    dt = _serve_dtype(fn, k_cache, v_cache)
    cache = k_cache.shape
    if len(cache) != 4 or cache != v_cache.shape or table.dim() != 2 or weights.dim() != 3:
        raise ValueError(f"{fn}: caches [pages, Hkv, page_size, D], table [B, P], weights "
                         "[B, Hkv, slots]")
    pages, Hkv, page_size, D = cache
    B, width = table.shape
    shape = (B, Hkv, weights.shape[2])
    _expect(fn, "table", table, torch.int32, (B, width))
    _expect(fn, "lens", lens, torch.int32, (B,))
    _expect(fn, "next_pos", next_pos, torch.int32, (B,))
    _expect(fn, "weights", weights, torch.float32, shape)
    _expect(fn, "positions", positions, torch.int32, shape)
    if lens_out is None:
        lens_out = torch.empty_like(lens)
    else:
        _expect(fn, "lens_out", lens_out, torch.int32, (B,))
    if weights_out is None:
        weights_out = torch.zeros_like(weights)
    else:
        _expect(fn, "weights_out", weights_out, torch.float32, shape)
    if positions_out is None:
        positions_out = torch.full_like(positions, -1)
    else:
        _expect(fn, "positions_out", positions_out, torch.int32, shape)
    if ws is None:
        ws = torch.empty(max(256, idx_cache_evict_workspace(B, Hkv, budget,
                                                            max_len or width * page_size)),
                         dtype=torch.uint8, device=lens.device)
    _serve_call(fn, load().idx_cache_evict, index, (
        k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), lens.data_ptr(),
        weights.data_ptr(), positions.data_ptr(), next_pos.data_ptr(), B, Hkv, D, pages,
        page_size, width, max_len, shape[2], budget, recent, sink, dt, lens_out.data_ptr(),
        weights_out.data_ptr(), positions_out.data_ptr(), ws.data_ptr(), ws.nbytes),
        options, stats, stream)
    return lens_out, weights_out, positions_out
