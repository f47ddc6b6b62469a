// Python binding of the serving operators (idx_add_rmsnorm_quant, idx_prefix_attention,
// idx_cache_evict, and those of the cache in 4 bits and of its pages): their tensors' checks
// and the calls into libidx.  A serving loop makes
// these calls per layer and token, and through Python-side checks and ctypes the small ones
// cost more on the host (8 to 17 us) than on the GPU.  Each function takes the tensors as the
// package's wrapper has them, raises ValueError for one that does not fit, and returns
// libidx's status.  libidx is the one that the package loaded: bind() and bind_cache()
// take its functions' addresses.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <initializer_list>
#include <sstream>
#include <string>

#include "idx.h"

namespace {

decltype(&idx_add_rmsnorm_quant) norm_fn;
decltype(&idx_prefix_attention) attention_fn;
decltype(&idx_cache_evict) evict_fn;
decltype(&idx_cache_append_mxfp4) append_fn;
decltype(&idx_window_attention_mxfp4) window_fn;
decltype(&idx_cache_fork) fork_fn;
decltype(&idx_cache_resize) resize_fn;
decltype(&idx_cache_compact) compact_fn;

struct Bad {
    std::string text;
};

// The checks of one call; every tensor has to live on the first one's device.
struct Checks {
    const char* fn;
    PyObject* const* last;  // the options' address and the stream
    int device = -1;

    [[noreturn]] void bad(const std::string& what) const { throw Bad{std::string(fn) + ": " + what}; }

    // A CUDA tensor; None gives null.
    const at::Tensor* get(PyObject* o, const char* name) {
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) bad(std::string(name) + " is not a tensor");
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda()) bad("every tensor must live on a CUDA device");
        const int d = t.get_device();
        if (device >= 0 && d != device)
            bad("tensors on different devices (cuda:" + std::to_string(device) + " and cuda:" +
                std::to_string(d) + ")");
        device = d;
        return &t;
    }
    // A contiguous one.
    const at::Tensor* dense(PyObject* o, const char* name) {
        const at::Tensor* t = get(o, name);
        if (t && !t->is_contiguous()) bad("tensors must be contiguous");
        return t;
    }
    const at::Tensor& need(PyObject* o, const char* name) {
        const at::Tensor* t = dense(o, name);
        if (!t) bad(std::string(name) + " is missing");
        return *t;
    }
    void expect(const at::Tensor* t, const char* name, at::ScalarType type,
                std::initializer_list<int64_t> shape) const {
        if (!t || (t->scalar_type() == type && t->sizes() == at::IntArrayRef(shape))) return;
        std::ostringstream s;
        s << name << " must be " << type << " " << at::IntArrayRef(shape) << ", got "
          << t->scalar_type() << " " << t->sizes();
        bad(s.str());
    }
    // The one element type of the tensors, as libidx names it.
    idx_dtype type(std::initializer_list<const at::Tensor*> ts) const {
        const at::ScalarType first = (*ts.begin())->scalar_type();
        for (const at::Tensor* t : ts)
            if (t && t->scalar_type() != first) {
                std::ostringstream s;
                s << t->scalar_type() << " and " << first << " tensors where one type is needed";
                bad(s.str());
            }
        if (first == at::kBFloat16) return IDX_BF16;
        if (first == at::kHalf) return IDX_FP16;
        if (first == at::kFloat) return IDX_FP32;
        std::ostringstream s;
        s << "unsupported type " << first;
        bad(s.str());
    }
    int whole(PyObject* o, const char* name) const {
        return fits(PyLong_AsLongLong(o), name);
    }
    int fits(long long v, const char* name) const {
        if (v == -1 && PyErr_Occurred()) throw Bad{""};
        if (v < INT_MIN || v > INT_MAX) bad(std::string(name) + " does not fit an int");
        return (int)v;
    }
    float real(PyObject* o) const {
        const double v = PyFloat_AsDouble(o);
        if (v == -1.0 && PyErr_Occurred()) throw Bad{""};
        return (float)v;
    }
};

template <typename T = void> T* data(const at::Tensor* t) {
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
// f(args..., options, stream) with the tensors' device current and the interpreter released;
// no stream (None): the device's current one.
template <typename F, typename... A> long launch(const Checks& c, F* f, A... args) {
    const auto address = [](PyObject* o) { return o == Py_None ? nullptr : PyLong_AsVoidPtr(o); };
    auto* options = static_cast<idx_options*>(address(c.last[0]));
    void* stream = c.last[1] == Py_None ? c10::cuda::getCurrentCUDAStream(c.device).stream()
                                        : address(c.last[1]);
    if (PyErr_Occurred()) throw Bad{""};
    const c10::cuda::CUDAGuard guard(c.device);
    long status;
    Py_BEGIN_ALLOW_THREADS
    status = f(args..., options, stream);
    Py_END_ALLOW_THREADS
    return status;
}

// One call of `count` arguments, the last two the options' address and the stream.
template <typename F>
PyObject* run(const char* fn, PyObject* const* a, Py_ssize_t have, Py_ssize_t count, F&& call) {
    if (have != count) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", fn, count, have);
        return nullptr;
    }
    try {
        Checks c{fn, a + count - 2};
        return PyLong_FromLong(call(c));
    } catch (const Bad& b) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, b.text.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (x, weight, residual, residual_out, eps, group, out, scale, options, stream)
PyObject* add_rmsnorm_quant(PyObject*, PyObject* const* a, Py_ssize_t have) {
    return run("idx_add_rmsnorm_quant", a, have, 10, [&](Checks& c) -> long {
        const at::Tensor* x = c.get(a[0], "x");
        if (!x || x->dim() != 2 || (x->size(1) > 1 && x->stride(1) != 1))
            c.bad("x must be [rows, N] with adjacent columns");
        const int rows = c.fits(x->size(0), "rows"), n = c.fits(x->size(1), "N");
        const long long stride = rows > 1 ? x->stride(0) : std::max<int64_t>(n, x->stride(0));
        const at::Tensor& weight = c.need(a[1], "weight");
        const at::Tensor* residual = c.dense(a[2], "residual");
        const at::Tensor* residual_out = c.dense(a[3], "residual_out");
        const at::Tensor& out = c.need(a[6], "out");
        const at::Tensor& scale = c.need(a[7], "scale");
        const int group = c.whole(a[5], "group");
        const idx_dtype dt = c.type({x, &weight, residual, residual_out});
        c.expect(&weight, "weight", x->scalar_type(), {n});
        c.expect(residual, "residual", x->scalar_type(), {rows, n});
        c.expect(residual_out, "residual_out", x->scalar_type(), {rows, n});
        c.expect(&out, "out", at::kFloat8_e4m3fn, {rows, n});
        if (group < 0 || (group && n % group))
            c.bad(std::to_string(n) + " columns are not whole groups of " + std::to_string(group));
        if (group)
            c.expect(&scale, "scale", at::kFloat, {rows, n / group});
        else
            c.expect(&scale, "scale", at::kFloat, {rows});
        return launch(c, norm_fn, data(x), stride, data(residual), data(&weight), rows, n,
                      c.real(a[4]), group, dt, data(residual_out), data<uint8_t>(&out),
                      data<float>(&scale));
    });
}

// (q, k_cache, v_cache, table, lens, prefix_table, prefix_len, max_len, scale, weights,
//  weights_out, out, lse, ws, options, stream); scale None: D^-1/2
PyObject* prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t have) {
    return run("idx_prefix_attention", a, have, 16, [&](Checks& c) -> long {
        const at::Tensor& q = c.need(a[0], "q");
        const at::Tensor& k = c.need(a[1], "k_cache");
        const at::Tensor& v = c.need(a[2], "v_cache");
        const at::Tensor& table = c.need(a[3], "table");
        const at::Tensor& lens = c.need(a[4], "lens");
        const at::Tensor* prefix_table = c.dense(a[5], "prefix_table");
        const at::Tensor* w = c.dense(a[9], "weights");
        const at::Tensor* w_out = c.dense(a[10], "weights_out");
        const at::Tensor& out = c.need(a[11], "out");
        const at::Tensor& lse = c.need(a[12], "lse");
        const at::Tensor& ws = c.need(a[13], "ws");
        const int prefix_len = c.whole(a[6], "prefix_len"), max_len = c.whole(a[7], "max_len");
        const idx_dtype dt = c.type({&q, &k, &v});
        if (q.dim() != 4 || k.dim() != 4 || k.sizes() != v.sizes() || table.dim() != 2)
            c.bad("q [B, Q, Hq, D], caches [pages, Hkv, page_size, D], table [B, P]");
        const int B = c.fits(q.size(0), "B"), Q = c.fits(q.size(1), "Q"), Hq = c.fits(q.size(2), "Hq");
        const int D = c.fits(q.size(3), "D"), pages = c.fits(k.size(0), "pages");
        const int Hkv = c.fits(k.size(1), "Hkv"), page_size = c.fits(k.size(2), "page_size");
        if (k.size(3) != D)
            c.bad("q has " + std::to_string(D) + " dimensions, the caches " + std::to_string(k.size(3)));
        c.expect(&table, "table", at::kInt, {B, table.size(1)});
        c.expect(&lens, "lens", at::kInt, {B});
        if (prefix_len > 0 && (!prefix_table || prefix_table->scalar_type() != at::kInt ||
                               prefix_table->numel() * page_size < prefix_len))
            c.bad("prefix_table must be int32 and cover prefix_len");
        long long slots = 0;
        if (w) {
            if (w->dim() != 3 || w->scalar_type() != at::kFloat || w->size(0) != B || w->size(1) != Hkv)
                c.bad("weights must be float32 [B, Hkv, slots]");
            slots = w->size(2);
            if (!w_out) c.bad("weights without weights_out");
            c.expect(w_out, "weights_out", at::kFloat, {B, Hkv, slots});
        } else if (w_out) {
            c.bad("weights_out without weights");
        }
        c.expect(&out, "out", q.scalar_type(), {B, Q, Hq, D});
        c.expect(&lse, "lse", at::kFloat, {B, Q, Hq});
        const float scale = a[8] == Py_None ? (float)(1. / std::sqrt((double)D)) : c.real(a[8]);
        return launch(c, attention_fn, data(&q), data(&k), data(&v), data<int>(prefix_table),
                      data<int>(&table), data<int>(&lens), data<float>(w), B, Q, Hq, Hkv, D, pages,
                      page_size, prefix_len, table.size(1), max_len, slots, scale, dt, data(&out),
                      data<float>(&lse), data<float>(w_out), data(&ws), ws.nbytes());
    });
}

// (k_cache, v_cache, table, lens, weights, positions, next_pos, budget, recent, sink, max_len,
//  lens_out, weights_out, positions_out, ws, options, stream)
PyObject* cache_evict(PyObject*, PyObject* const* a, Py_ssize_t have) {
    return run("idx_cache_evict", a, have, 17, [&](Checks& c) -> long {
        const at::Tensor& k = c.need(a[0], "k_cache");
        const at::Tensor& v = c.need(a[1], "v_cache");
        const at::Tensor& table = c.need(a[2], "table");
        const at::Tensor& lens = c.need(a[3], "lens");
        const at::Tensor& w = c.need(a[4], "weights");
        const at::Tensor& pos = c.need(a[5], "positions");
        const at::Tensor& next_pos = c.need(a[6], "next_pos");
        const at::Tensor& lens_out = c.need(a[11], "lens_out");
        const at::Tensor& w_out = c.need(a[12], "weights_out");
        const at::Tensor& pos_out = c.need(a[13], "positions_out");
        const at::Tensor& ws = c.need(a[14], "ws");
        const idx_dtype dt = c.type({&k, &v});
        if (k.dim() != 4 || k.sizes() != v.sizes() || table.dim() != 2 || w.dim() != 3)
            c.bad("caches [pages, Hkv, page_size, D], table [B, P], weights [B, Hkv, slots]");
        const int pages = c.fits(k.size(0), "pages"), Hkv = c.fits(k.size(1), "Hkv");
        const int page_size = c.fits(k.size(2), "page_size"), D = c.fits(k.size(3), "D");
        const int B = c.fits(table.size(0), "B");
        const int64_t slots = w.size(2);
        c.expect(&table, "table", at::kInt, {B, table.size(1)});
        c.expect(&lens, "lens", at::kInt, {B});
        c.expect(&next_pos, "next_pos", at::kInt, {B});
        c.expect(&w, "weights", at::kFloat, {B, Hkv, slots});
        c.expect(&pos, "positions", at::kInt, {B, Hkv, slots});
        c.expect(&lens_out, "lens_out", at::kInt, {B});
        c.expect(&w_out, "weights_out", at::kFloat, {B, Hkv, slots});
        c.expect(&pos_out, "positions_out", at::kInt, {B, Hkv, slots});
        return launch(c, evict_fn, data(&k), data(&v), data<int>(&table), data<int>(&lens),
                      data<float>(&w), data<int>(&pos), data<int>(&next_pos), B, Hkv, D, pages,
                      page_size, table.size(1), c.whole(a[10], "max_len"), slots,
                      c.whole(a[7], "budget"), c.whole(a[8], "recent"), c.whole(a[9], "sink"), dt,
                      data<int>(&lens_out), data<float>(&w_out), data<int>(&pos_out), data(&ws),
                      ws.nbytes());
    });
}

// The cache in 4 bits as its calls take it, and whose tokens are new.
struct Mxfp4Cache {
    const at::Tensor *k_codes, *k_sf, *v_codes, *v_sf, *table, *lens, *q_start;
    int B, pages, Hkv, page_size, D;
};
// a: k_codes, k_sf, v_codes, v_sf, table, lens, q_start
Mxfp4Cache mxfp4_cache(Checks& c, PyObject* const* a) {
    Mxfp4Cache m;
    m.k_codes = &c.need(a[0], "k_codes");
    m.k_sf = &c.need(a[1], "k_sf");
    m.v_codes = &c.need(a[2], "v_codes");
    m.v_sf = &c.need(a[3], "v_sf");
    m.table = &c.need(a[4], "table");
    m.lens = &c.need(a[5], "lens");
    m.q_start = c.dense(a[6], "q_start");
    if (m.k_codes->dim() != 4 || m.table->dim() != 2)
        c.bad("codes [pages, Hkv, page_size, D / 2], table [B, P]");
    m.pages = c.fits(m.k_codes->size(0), "pages");
    m.Hkv = c.fits(m.k_codes->size(1), "Hkv");
    m.page_size = c.fits(m.k_codes->size(2), "page_size");
    m.D = c.fits(m.k_codes->size(3) * 2, "D");
    m.B = c.fits(m.table->size(0), "B");
    c.expect(m.k_codes, "k_codes", at::kByte, {m.pages, m.Hkv, m.page_size, m.D / 2});
    c.expect(m.v_codes, "v_codes", at::kByte, {m.pages, m.Hkv, m.page_size, m.D / 2});
    c.expect(m.k_sf, "k_sf", at::kByte, {m.pages, m.Hkv, m.page_size, m.D / 32});
    c.expect(m.v_sf, "v_sf", at::kByte, {m.pages, m.Hkv, m.page_size, m.D / 32});
    c.expect(m.table, "table", at::kInt, {m.B, m.table->size(1)});
    c.expect(m.lens, "lens", at::kInt, {m.B});
    c.expect(m.q_start, "q_start", at::kInt, {m.B + 1});
    return m;
}
// Rows [T, heads, D] of tokens that may lie apart: the elements from one token to the next.
long long token_stride(const Checks& c, const at::Tensor* t, const char* name, int64_t heads, int64_t D) {
    if (!t || t->dim() != 3 || t->size(1) != heads || t->size(2) != D || (D > 1 && t->stride(2) != 1) ||
        (heads > 1 && t->stride(1) != D))
        c.bad(std::string(name) + " must be [T, " + std::to_string(heads) + ", " + std::to_string(D) +
              "] with every token's rows adjacent");
    return t->size(0) > 1 ? t->stride(0) : std::max<int64_t>(heads * D, t->stride(0));
}

// (k, v, k_codes, k_sf, v_codes, v_sf, table, lens, q_start, options, stream)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t have) {
    return run("idx_cache_append_mxfp4", a, have, 11, [&](Checks& c) -> long {
        const at::Tensor *k = c.get(a[0], "k"), *v = c.get(a[1], "v");
        const Mxfp4Cache m = mxfp4_cache(c, a + 2);
        const long long ks = token_stride(c, k, "k", m.Hkv, m.D), vs = token_stride(c, v, "v", m.Hkv, m.D);
        const idx_dtype dt = c.type({k, v});
        const int T = c.fits(k->size(0), "T");
        if (v->size(0) != T) c.bad("k and v have different numbers of tokens");
        return launch(c, append_fn, data(k), ks, data(v), vs, data<uint8_t>(m.k_codes), data<uint8_t>(m.k_sf),
                      data<uint8_t>(m.v_codes), data<uint8_t>(m.v_sf), data<int>(m.table), data<int>(m.lens),
                      data<int>(m.q_start), m.B, T, m.Hkv, m.D, m.pages, m.page_size, m.table->size(1), dt);
    });
}

// (q, k_codes, k_sf, v_codes, v_sf, table, lens, q_start, max_q, max_len, window, sink, scale, out, lse,
//  ws, options, stream); scale None: D^-1/2
PyObject* window_attention(PyObject*, PyObject* const* a, Py_ssize_t have) {
    return run("idx_window_attention_mxfp4", a, have, 18, [&](Checks& c) -> long {
        const at::Tensor* q = c.get(a[0], "q");
        const Mxfp4Cache m = mxfp4_cache(c, a + 1);
        if (!q || q->dim() != 3) c.bad("q must be [T, Hq, D]");
        const int T = c.fits(q->size(0), "T"), Hq = c.fits(q->size(1), "Hq");
        const long long qs = token_stride(c, q, "q", Hq, m.D);
        const idx_dtype dt = c.type({q});
        const at::Tensor& out = c.need(a[13], "out");
        const at::Tensor& lse = c.need(a[14], "lse");
        const at::Tensor& ws = c.need(a[15], "ws");
        c.expect(&out, "out", q->scalar_type(), {T, Hq, m.D});
        c.expect(&lse, "lse", at::kFloat, {T, Hq});
        const float scale = a[12] == Py_None ? (float)(1. / std::sqrt((double)m.D)) : c.real(a[12]);
        return launch(c, window_fn, data(q), qs, data<uint8_t>(m.k_codes), data<uint8_t>(m.k_sf),
                      data<uint8_t>(m.v_codes), data<uint8_t>(m.v_sf), data<int>(m.table), data<int>(m.lens),
                      data<int>(m.q_start), m.B, T, c.whole(a[8], "max_q"), Hq, m.Hkv, m.D, m.pages, m.page_size,
                      m.table->size(1), c.whole(a[9], "max_len"), c.whole(a[10], "window"), c.whole(a[11], "sink"),
                      scale, dt, data(&out), data<float>(&lse), data(&ws), ws.nbytes());
    });
}

// A page table, its rows' lengths and its pages' counts, before and after a call.
struct Pages {
    const at::Tensor *refs, *table, *lens, *refs_out, *table_out;
    int B, pages;
};
Pages pages_of(Checks& c, PyObject* refs, PyObject* table, PyObject* lens, PyObject* refs_out, PyObject* table_out) {
    Pages p;
    p.refs = &c.need(refs, "refs");
    p.table = &c.need(table, "table");
    p.lens = &c.need(lens, "lens");
    p.refs_out = &c.need(refs_out, "refs_out");
    p.table_out = &c.need(table_out, "table_out");
    if (p.refs->dim() != 1 || p.table->dim() != 2) c.bad("refs [pages], table [B, P]");
    p.pages = c.fits(p.refs->size(0), "pages");
    p.B = c.fits(p.table->size(0), "B");
    c.expect(p.refs, "refs", at::kInt, {p.pages});
    c.expect(p.refs_out, "refs_out", at::kInt, {p.pages});
    c.expect(p.table, "table", at::kInt, {p.B, p.table->size(1)});
    c.expect(p.table_out, "table_out", at::kInt, {p.B, p.table->size(1)});
    c.expect(p.lens, "lens", at::kInt, {p.B});
    return p;
}
// The arrays [pages, ...] whose pages move: a sequence of tensors.
struct Caches {
    void* p[8];
    long long bytes[8];
    int n = 0;
};
Caches caches_of(Checks& c, PyObject* list, int pages) {
    Caches r;
    PyObject* seq = PySequence_Fast(list, "caches must be a sequence of tensors");
    if (!seq) throw Bad{""};
    struct Release {
        PyObject* o;
        ~Release() { Py_DECREF(o); }
    } release{seq};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    if (n > 8) c.bad("at most 8 caches");
    for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor& t = c.need(PySequence_Fast_GET_ITEM(seq, i), "a cache");
        if (t.dim() < 1 || t.size(0) != pages) c.bad("caches must be [pages, ...]");
        if (pages > 0 && t.numel() == 0) c.bad("a cache has empty pages");
        r.p[i] = t.data_ptr();
        r.bytes[i] = pages > 0 ? (long long)(t.nbytes() / pages) : 16;
        ++r.n;
    }
    return r;
}

// (refs, table, lens, parent, page_size, refs_out, table_out, lens_out, ws, options, stream); ws may be None
PyObject* cache_fork(PyObject*, PyObject* const* a, Py_ssize_t have) {
    return run("idx_cache_fork", a, have, 11, [&](Checks& c) -> long {
        const Pages p = pages_of(c, a[0], a[1], a[2], a[5], a[6]);
        const at::Tensor& parent = c.need(a[3], "parent");
        const at::Tensor& lens_out = c.need(a[7], "lens_out");
        const at::Tensor* ws = c.dense(a[8], "ws");
        c.expect(&parent, "parent", at::kInt, {p.B});
        c.expect(&lens_out, "lens_out", at::kInt, {p.B});
        return launch(c, fork_fn, data<int>(p.refs), data<int>(p.table), data<int>(p.lens), data<int>(&parent), p.B,
                      p.pages, c.whole(a[4], "page_size"), p.table->size(1), data<int>(p.refs_out),
                      data<int>(p.table_out), data<int>(&lens_out), data(ws), ws ? ws->nbytes() : 0);
    });
}

// (caches, refs, table, lens, new_lens, page_size, refs_out, table_out, lens_out, ws, options, stream)
PyObject* cache_resize(PyObject*, PyObject* const* a, Py_ssize_t have) {
    return run("idx_cache_resize", a, have, 12, [&](Checks& c) -> long {
        const Pages p = pages_of(c, a[1], a[2], a[3], a[6], a[7]);
        const Caches caches = caches_of(c, a[0], p.pages);
        const at::Tensor& new_lens = c.need(a[4], "new_lens");
        const at::Tensor& lens_out = c.need(a[8], "lens_out");
        const at::Tensor& ws = c.need(a[9], "ws");
        c.expect(&new_lens, "new_lens", at::kInt, {p.B});
        c.expect(&lens_out, "lens_out", at::kInt, {p.B});
        return launch(c, resize_fn, caches.p, caches.bytes, caches.n, data<int>(p.refs), data<int>(p.table),
                      data<int>(p.lens), data<int>(&new_lens), p.B, p.pages, c.whole(a[5], "page_size"),
                      p.table->size(1), data<int>(p.refs_out), data<int>(p.table_out), data<int>(&lens_out), data(&ws),
                      ws.nbytes());
    });
}

// (caches, refs, table, lens, page_size, refs_out, table_out, live, ws, options, stream)
PyObject* cache_compact(PyObject*, PyObject* const* a, Py_ssize_t have) {
    return run("idx_cache_compact", a, have, 11, [&](Checks& c) -> long {
        const Pages p = pages_of(c, a[1], a[2], a[3], a[5], a[6]);
        const Caches caches = caches_of(c, a[0], p.pages);
        const at::Tensor& live = c.need(a[7], "live");
        const at::Tensor& ws = c.need(a[8], "ws");
        c.expect(&live, "live", at::kInt, {1});
        return launch(c, compact_fn, caches.p, caches.bytes, caches.n, data<int>(p.refs), data<int>(p.table),
                      data<int>(p.lens), p.B, p.pages, c.whole(a[4], "page_size"), p.table->size(1),
                      data<int>(p.refs_out), data<int>(p.table_out), data<int>(&live), data(&ws), ws.nbytes());
    });
}

// Addresses of functions, or an exception.
bool addresses(PyObject* const* a, int n, void** f) {
    for (int i = 0; i < n; ++i)
        if (!(f[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
            return false;
        }
    return true;
}

// bind(idx_add_rmsnorm_quant, idx_prefix_attention, idx_cache_evict): the functions' addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t have) {
    if (have != 3) {
        PyErr_SetString(PyExc_TypeError, "bind takes three addresses");
        return nullptr;
    }
    void* f[3];
    if (!addresses(a, 3, f)) return nullptr;
    norm_fn = reinterpret_cast<decltype(norm_fn)>(f[0]);
    attention_fn = reinterpret_cast<decltype(attention_fn)>(f[1]);
    evict_fn = reinterpret_cast<decltype(evict_fn)>(f[2]);
    Py_RETURN_NONE;
}

// bind_cache(idx_cache_append_mxfp4, idx_window_attention_mxfp4, idx_cache_fork, idx_cache_resize,
// idx_cache_compact): the same
PyObject* bind_cache(PyObject*, PyObject* const* a, Py_ssize_t have) {
    if (have != 5) {
        PyErr_SetString(PyExc_TypeError, "bind_cache takes five addresses");
        return nullptr;
    }
    void* f[5];
    if (!addresses(a, 5, f)) return nullptr;
    append_fn = reinterpret_cast<decltype(append_fn)>(f[0]);
    window_fn = reinterpret_cast<decltype(window_fn)>(f[1]);
    fork_fn = reinterpret_cast<decltype(fork_fn)>(f[2]);
    resize_fn = reinterpret_cast<decltype(resize_fn)>(f[3]);
    compact_fn = reinterpret_cast<decltype(compact_fn)>(f[4]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    {"add_rmsnorm_quant", (PyCFunction)(void (*)(void))add_rmsnorm_quant, METH_FASTCALL, nullptr},
    {"prefix_attention", (PyCFunction)(void (*)(void))prefix_attention, METH_FASTCALL, nullptr},
    {"cache_evict", (PyCFunction)(void (*)(void))cache_evict, METH_FASTCALL, nullptr},
    {"bind_cache", (PyCFunction)(void (*)(void))bind_cache, METH_FASTCALL, nullptr},
    {"cache_append_mxfp4", (PyCFunction)(void (*)(void))cache_append, METH_FASTCALL, nullptr},
    {"window_attention_mxfp4", (PyCFunction)(void (*)(void))window_attention, METH_FASTCALL, nullptr},
    {"cache_fork", (PyCFunction)(void (*)(void))cache_fork, METH_FASTCALL, nullptr},
    {"cache_resize", (PyCFunction)(void (*)(void))cache_resize, METH_FASTCALL, nullptr},
    {"cache_compact", (PyCFunction)(void (*)(void))cache_compact, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, methods,
                      nullptr,               nullptr,  nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve(void) { return PyModule_Create(&module); }
