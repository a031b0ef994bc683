// Python marshalling of the calls around the decode step: tensors are checked,
// turned into the C ABI's descriptors and passed on.  No computation.
//
// A small extension module instead of ctypes because these calls are a few
// microseconds of GPU time each and take up to fifteen tensors: reading shapes,
// strides and types through Python attributes cost 9 to 14 us a call, more than
// the kernels; here it is well under one.
//
// Every function takes its arguments by position, raises ValueError or
// TypeError for arguments the descriptors cannot express, and returns the C
// call's status.  C++ exceptions stop at the boundary.
#include <Python.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <stdexcept>
#include <string>

#include "../../include/tree_attn.h"

namespace {

struct BadType : std::runtime_error {
    using std::runtime_error::runtime_error;
};
using BadValue = std::invalid_argument;

decltype(&tree_attn_norm_rope) p_norm_rope;
decltype(&tree_attn_cache_write) p_cache_write;
decltype(&tree_attn_cache_read) p_cache_read;
decltype(&tree_attn_page_bounds) p_page_bounds;
decltype(&tree_attn_select_workspace_bytes) p_select_workspace_bytes;
decltype(&tree_attn_select_pages) p_select_pages;
decltype(&tree_attn_decode_selected) p_decode_selected;
decltype(&tree_attn_cache_write_int4) p_cache_write_int4;
decltype(&tree_attn_cache_read_int4) p_cache_read_int4;
decltype(&tree_attn_window_workspace_bytes) p_window_workspace_bytes;
decltype(&tree_attn_decode_window) p_decode_window;
decltype(&tree_attn_decode_int4) p_decode_int4;

using Tensor = at::Tensor;

// The tensor argument `o` (null for None).
const Tensor* opt(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw BadType(std::string(name) + " must be a tensor");
    const Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided) throw BadType(std::string(name) + " must be a dense tensor");
    return &t;
}
const Tensor& need(PyObject* o, const char* name) {
    const Tensor* t = opt(o, name);
    if (!t) throw BadValue(std::string(name) + " is needed");
    return *t;
}
long long integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw BadType("");  // (the Python error is already set)
    return v;
}
int int32(PyObject* o, const char* name) {
    const long long v = integer(o);
    if (v > 0x7fffffff || v < -0x7fffffffLL - 1) throw BadValue(std::string(name) + " is out of range");
    return static_cast<int>(v);
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw BadType("");
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw BadType("");
    return v != 0;
}

int dtype_code(const Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return TA_F32;
        case at::kBFloat16: return TA_BF16;
        case at::ScalarType::Float8_e4m3fn: return TA_E4M3;
        default: throw BadType("unsupported dtype; use float32, bfloat16 or float8_e4m3fn (caches)");
    }
}
int vec_dtype(const Tensor& t) {
    const int c = dtype_code(t);
    if (c == TA_E4M3) throw BadType("head vectors must be bfloat16 or float32");
    return c;
}
int32_t size32(int64_t v, const char* what) {
    if (v > 0x7fffffff) throw BadValue(std::string(what) + " has too many entries");
    return static_cast<int32_t>(v);
}

// All tensors of a call: on one CUDA device, the current one.
struct Device {
    int index = -1;
    void add(const Tensor* t) {
        if (!t) return;
        if (!t->is_cuda()) throw BadValue("tensors must live on a CUDA device");
        const int d = t->get_device();
        if (index >= 0 && d != index) throw BadValue("tensors must live on one CUDA device");
        index = d;
    }
    // The stream of the call: an integer handle, or None for the current one.
    void* stream(PyObject* s) const {
        const int cur = c10::cuda::current_device();
        if (cur != index)
            throw BadValue("the tensors are on cuda:" + std::to_string(index) + " and the current device is cuda:" +
                           std::to_string(cur) + ": make theirs the current one");
        if (s != Py_None) {
            const unsigned long long h = PyLong_AsUnsignedLongLong(s);
            if (PyErr_Occurred()) throw BadType("");
            return reinterpret_cast<void*>(h);
        }
        return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
    }
};

// Whether vectors of d elements, one for each (i, j) in [0, n) x [0, m) at i a + j b, overlap: two of them do
// where |x a + y b| < d for some steps |x| < n, |y| < m, not both 0.
bool overlapping(int64_t n, int64_t a, int64_t m, int64_t b, int64_t d) {
    if (n <= 1) a = 0, n = 1;
    if (m <= 1) b = 0, m = 1;
    if (a < b) std::swap(a, b), std::swap(n, m);
    // the usual layouts: the smaller step keeps vectors apart, and the larger one its whole runs
    if ((m == 1 || b >= d) && (n == 1 || a >= (m - 1) * b + d)) return false;
    if ((m > 1 && b < d) || (n > 1 && a < d)) return true;
    for (int64_t y = 1; y < m && y * b < (n - 1) * a + d; ++y) {  // (x and y of opposite signs; the x on either side of y b / a)
        const int64_t x = y * b / a;
        if ((x < n && y * b - x * a < d) || (x + 1 < n && (x + 1) * a - y * b < d)) return true;
    }
    return false;
}

// Head vectors [tokens, heads, head_dim]; `output`: they must not share memory.
ta_heads heads(const Tensor& t, const char* name, bool output = false) {
    if (t.dim() != 3 || (t.stride(2) != 1 && t.size(2) > 1))
        throw BadValue(std::string(name) + " must be [tokens, heads, head_dim] with contiguous channels");
    ta_heads h;
    h.data = t.data_ptr();
    h.stride_t = t.size(0) > 1 ? t.stride(0) : 0;
    h.stride_h = t.size(1) > 1 ? t.stride(1) : 0;
    if (output && overlapping(t.size(0), h.stride_t, t.size(1), h.stride_h, t.size(2)))
        throw BadValue(std::string(name) + " is written to: its vectors must not share memory");
    return h;
}

const int32_t* ints(const Tensor* t, const char* name, int64_t n) {
    if (!t) return nullptr;
    if (t->scalar_type() != at::kInt || t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
        throw BadValue(std::string(name) + " must be a contiguous int32 tensor of " + std::to_string(n) + " entries");
    return t->const_data_ptr<int32_t>();
}

const float* scales(const Tensor* t, const char* name, int64_t n) {
    if (!t) return nullptr;
    if (t->scalar_type() != at::kFloat || t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
        throw BadValue(std::string(name) + " must be a contiguous float32 tensor [num_kv_heads]");
    return t->const_data_ptr<float>();
}

ta_rope rope_of(int64_t d, const Tensor* inv_freq, const Tensor* qw, const Tensor* kw, bool norm, double eps, bool interleaved) {
    ta_rope r;
    std::memset(&r, 0, sizeof r);
    if (inv_freq) {
        if (inv_freq->scalar_type() != at::kFloat || inv_freq->dim() != 1 || !inv_freq->is_contiguous())
            throw BadValue("inv_freq must be a contiguous float32 tensor [rot_dim / 2]");
        r.inv_freq = inv_freq->const_data_ptr<float>();
        r.rot_dim = size32(2 * inv_freq->size(0), "inv_freq");
    }
    r.weight_dtype = TA_F32;
    if (qw && kw && qw->scalar_type() != kw->scalar_type()) throw BadValue("q_weight and k_weight must have one type");
    for (const Tensor* w : {qw, kw}) {
        if (!w) continue;
        if (!norm) throw BadValue("norm weights need norm=True");
        if ((w->scalar_type() != at::kBFloat16 && w->scalar_type() != at::kFloat) || w->dim() != 1 || w->size(0) != d || !w->is_contiguous())
            throw BadValue("norm weights must be contiguous [head_dim] tensors, bfloat16 or float32");
        r.weight_dtype = dtype_code(*w);
    }
    r.q_weight = qw ? qw->data_ptr() : nullptr;
    r.k_weight = kw ? kw->data_ptr() : nullptr;
    r.norm = norm;
    r.eps = static_cast<float>(eps);
    r.interleaved = interleaved;
    return r;
}

// A stride of a cache axis; an axis of one entry may carry any, so it gets a valid one.  (Strides
// of 0 on every axis would mean a dense cache to the C call, whatever memory is behind the view.)
int64_t cache_stride(const Tensor& t, int axis) {
    if (t.size(axis) <= 1) return 128;
    if (t.stride(axis) == 0) throw BadValue("a cache's entries must not share memory: an axis of several has stride 0");
    return t.stride(axis);
}

void check_table(const Tensor& bt) {
    if (bt.scalar_type() != at::kInt || bt.dim() != 2 || !bt.is_contiguous())
        throw BadValue("block_table must be a contiguous int32 [B, max_pages] tensor");
}

// Rows, pages and lengths of pools [pages, page, Hkv, ..].
void pool_places(const Tensor& k, const Tensor& bt, PyObject* max_seqlen, ta_shape* s, ta_paged_kv* pg) {
    check_table(bt);
    s->batch = size32(bt.size(0), "block_table");
    s->num_kv_heads = size32(k.size(2), "a cache");
    pg->block_table = bt.const_data_ptr<int32_t>();
    pg->max_pages_per_seq = size32(bt.size(1), "block_table");
    pg->page_size = size32(k.size(1), "a page");
    pg->num_pages = size32(k.size(0), "a pool");
    const int64_t all = bt.size(1) * k.size(1);
    s->max_seqlen = max_seqlen == Py_None ? static_cast<int32_t>(std::min<int64_t>(all, 0x7fffffff)) : int32(max_seqlen, "max_seqlen");
}
// The same of dense caches [B, Hkv, S, ..].
void dense_places(const Tensor& k, PyObject* max_seqlen, ta_shape* s) {
    s->batch = size32(k.size(0), "a cache");
    s->num_kv_heads = size32(k.size(1), "a cache");
    s->max_seqlen = size32(k.size(2), "a cache");
    if (max_seqlen != Py_None) {
        const int most = int32(max_seqlen, "max_seqlen");
        if (most < 1 || most > s->max_seqlen) throw BadValue("max_seqlen must be at least 1 and at most the cache's tokens");
        s->max_seqlen = most;
    }
}

// [pages, page, Hkv, d] pools
void pool_shape(const Tensor& k, const Tensor& bt, PyObject* max_seqlen, ta_shape* s, ta_paged_kv* pg) {
    if (k.dim() != 4 || k.stride(3) != 1) throw BadValue("page pools must be [num_pages, page_size, Hkv, d] with contiguous channels");
    pool_places(k, bt, max_seqlen, s, pg);
    s->head_dim = size32(k.size(3), "a cache");
    s->kv_dtype = dtype_code(k);
    s->kv_stride_b = cache_stride(k, 0);
    s->kv_stride_t = cache_stride(k, 1);
    s->kv_stride_h = cache_stride(k, 2);
}

// [B, Hkv, S, d] caches
void dense_shape(const Tensor& k, PyObject* max_seqlen, ta_shape* s) {
    if (k.dim() != 4 || k.stride(3) != 1) throw BadValue("dense caches must be [B, Hkv, S, d] with contiguous channels");
    dense_places(k, max_seqlen, s);
    s->head_dim = size32(k.size(3), "a cache");
    s->kv_dtype = dtype_code(k);
    s->kv_stride_b = cache_stride(k, 0);
    s->kv_stride_h = cache_stride(k, 1);
    s->kv_stride_t = cache_stride(k, 2);
}

void same_cache(const Tensor& k, const Tensor& v) {
    if (!v.sizes().equals(k.sizes()) || !v.strides().equals(k.strides()) || v.scalar_type() != k.scalar_type())
        throw BadValue("the key and value caches must agree on shape, strides and type");
}

// The token list of a cache write or read of head vectors like `vec`, and their type.
void tokens_of(const Tensor& pos, const Tensor* rows, const Tensor& vec, ta_shape* shape, ta_tokens* tokens) {
    shape->num_q_heads = shape->num_kv_heads;
    shape->q_dtype = vec_dtype(vec);
    if (pos.dim() != 1) throw BadValue("positions must be a contiguous int32 tensor [tokens]");
    tokens->num_tokens = size32(pos.size(0), "positions");
    tokens->positions = ints(&pos, "positions", pos.size(0));
    tokens->rows = ints(rows, "rows", pos.size(0));
    if (vec.dim() != 3 || vec.size(0) != pos.size(0) || vec.size(1) != shape->num_kv_heads || vec.size(2) != shape->head_dim)
        throw BadValue("head vectors must be [tokens, num_kv_heads, head_dim] of the cache and the positions");
}

// A 4-bit cache: codes [.., d / 2] and steps [.., d / 16] over the axes of the other caches.
struct Int4Cache {
    ta_shape shape;
    ta_paged_kv paged;
    ta_int4_kv cache;
    const ta_paged_kv* pages = nullptr;
    Int4Cache(const Tensor& kc, const Tensor& vc, const Tensor& kst, const Tensor& vst, const Tensor* bt, PyObject* max_seqlen, const Tensor* ks,
              const Tensor* vs) {
        std::memset(&shape, 0, sizeof shape);
        std::memset(&paged, 0, sizeof paged);
        std::memset(&cache, 0, sizeof cache);
        same_cache(kc, vc);
        same_cache(kst, vst);
        if (kc.scalar_type() != at::kByte || kst.scalar_type() != at::ScalarType::Float8_e4m3fn)
            throw BadType("4-bit caches are uint8 codes and float8_e4m3fn steps");
        if (kc.dim() != 4 || kst.dim() != 4 || kc.stride(3) != 1 || kst.stride(3) != 1)
            throw BadValue("4-bit caches must be 4-D, with contiguous codes [.., d / 2] and steps [.., d / 16]");
        for (int i = 0; i < 3; ++i)
            if (kc.size(i) != kst.size(i)) throw BadValue("codes and steps must agree on pages or rows, tokens and heads");
        if (kc.size(3) != 8 * kst.size(3)) throw BadValue("there must be a step for every eight bytes of codes");
        if (bt) {
            pool_places(kc, *bt, max_seqlen, &shape, &paged);
            pages = &paged;
        } else {
            dense_places(kc, max_seqlen, &shape);
        }
        shape.head_dim = size32(2 * kc.size(3), "a cache");
        shape.kv_dtype = TA_INT4;
        const int h = bt ? 2 : 1, t = bt ? 1 : 2;
        cache.k_codes = kc.data_ptr();
        cache.v_codes = vc.data_ptr();
        cache.k_steps = kst.data_ptr();
        cache.v_steps = vst.data_ptr();
        cache.code_stride_b = cache_stride(kc, 0);
        cache.code_stride_h = cache_stride(kc, h);
        cache.code_stride_t = cache_stride(kc, t);
        cache.step_stride_b = cache_stride(kst, 0);
        cache.step_stride_h = cache_stride(kst, h);
        cache.step_stride_t = cache_stride(kst, t);
        if (!ks != !vs) throw BadValue("k_scale and v_scale go together");
        cache.k_scale = scales(ks, "k_scale", shape.num_kv_heads);
        cache.v_scale = scales(vs, "v_scale", shape.num_kv_heads);
    }
};

// Shape, pages and tokens of a cache write or read of head vectors like `vec`.
struct CacheCall {
    ta_shape shape;
    ta_paged_kv paged;
    ta_tokens tokens;
    const ta_paged_kv* pages = nullptr;
    CacheCall(const Tensor& kc, const Tensor& vc, const Tensor& pos, const Tensor* rows, const Tensor* bt, PyObject* max_seqlen, const Tensor& vec) {
        std::memset(&shape, 0, sizeof shape);
        std::memset(&paged, 0, sizeof paged);
        std::memset(&tokens, 0, sizeof tokens);
        same_cache(kc, vc);
        if (bt) {
            pool_shape(kc, *bt, max_seqlen, &shape, &paged);
            pages = &paged;
        } else {
            dense_shape(kc, max_seqlen, &shape);
        }
        tokens_of(pos, rows, vec, &shape, &tokens);
    }
};

void like(const Tensor& a, const Tensor& b, const char* what) {
    if (!a.sizes().equals(b.sizes()) || a.scalar_type() != b.scalar_type()) throw BadValue(std::string(what) + " must agree on shape and type");
}

// torch.OutOfMemoryError (the class itself is not among libtorch_python's exported symbols).
void set_out_of_memory(const char* what) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, what);
    Py_XDECREF(type);
    Py_XDECREF(torch);
}

template <typename Fn>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, Fn&& fn) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    if (!p_norm_rope) {
        PyErr_SetString(PyExc_RuntimeError, "the library is not loaded");
        return nullptr;
    }
    try {
        return PyLong_FromLong(fn());
    } catch (const BadValue& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const BadType& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const c10::OutOfMemoryError& e) {  // (a workspace that torch's allocator could not provide)
        if (!PyErr_Occurred()) set_out_of_memory(e.what_without_backtrace());
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// The GIL is not held while the C call enqueues.
template <typename Fn>
int enqueue(Fn&& fn) {
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn();
    Py_END_ALLOW_THREADS
    return rc;
}

// q, k, positions, inv_freq, q_weight, k_weight, norm, eps, interleaved, q_out, k_out, stream
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        const Tensor *q = opt(a[0], "q"), *k = opt(a[1], "k"), *f = opt(a[3], "inv_freq"), *qw = opt(a[4], "q_weight"),
                     *kw = opt(a[5], "k_weight"), *qo = opt(a[9], "q_out"), *ko = opt(a[10], "k_out");
        const Tensor& pos = need(a[2], "positions");
        const bool norm = truth(a[6]);
        if (!q && !k) throw BadValue("q or k is needed");
        if (!q != !qo || !k != !ko) throw BadValue("an output without its input, or the other way round");
        if (!norm && !f) throw BadValue("nothing to do: no norm and no inv_freq");
        const Tensor& x = q ? *q : *k;
        ta_heads h[4];
        std::memset(h, 0, sizeof h);
        if (q) h[0] = heads(*q, "q"), h[1] = heads(*qo, "q_out", true), like(*q, *qo, "q and q_out");
        if (k) h[2] = heads(*k, "k"), h[3] = heads(*ko, "k_out", true), like(*k, *ko, "k and k_out");
        if (q && k && (q->size(0) != k->size(0) || q->size(2) != k->size(2) || q->scalar_type() != k->scalar_type()))
            throw BadValue("q and k must agree on tokens, head_dim and type");
        ta_shape s;
        std::memset(&s, 0, sizeof s);
        s.batch = s.max_seqlen = 1;
        s.num_q_heads = q ? size32(q->size(1), "q") : 0;
        s.num_kv_heads = k ? size32(k->size(1), "k") : 0;
        s.head_dim = size32(x.size(2), "a vector");
        s.q_dtype = vec_dtype(x);
        ta_tokens tok;
        std::memset(&tok, 0, sizeof tok);
        tok.num_tokens = size32(x.size(0), "the token list");
        tok.positions = ints(&pos, "positions", x.size(0));
        const ta_rope r = rope_of(x.size(2), f, qw, kw, norm, real(a[7]), truth(a[8]));
        Device dev;
        for (const Tensor* t : {q, k, &pos, f, qw, kw, qo, ko}) dev.add(t);
        void* st = dev.stream(a[11]);
        return enqueue([&] {
            return p_norm_rope(&s, &tok, &r, q ? &h[0] : nullptr, q ? &h[1] : nullptr, k ? &h[2] : nullptr, k ? &h[3] : nullptr, st);
        });
    });
}

// Vectors, norm and rotation of a cache write: what the writes of both kinds of caches share.
struct Written {
    ta_heads hk, hv, hq, hqo;
    ta_rope rope;
    bool turned;
    const Tensor* q;
    // k, v, q, q_out, inv_freq, q_weight, k_weight, norm, eps, interleaved
    Written(const Tensor& k, const Tensor& v, const Tensor* q_, const Tensor* qo, const Tensor* f, const Tensor* qw, const Tensor* kw, PyObject* norm_,
            PyObject* eps, PyObject* interleaved, ta_shape* shape)
        : q(q_) {
        const bool norm = truth(norm_);
        turned = norm || f;
        if (!q != !qo) throw BadValue("q and q_out go together");
        if (q && !turned) throw BadValue("q needs a norm or a rotation");
        if (!norm && (qw || kw)) throw BadValue("norm weights need norm=True");
        hk = heads(k, "k");
        hv = heads(v, "v");
        if (q) {
            like(*q, *qo, "q and q_out");
            hq = heads(*q, "q");
            hqo = heads(*qo, "q_out", true);
            if (q->size(0) != k.size(0) || q->size(2) != k.size(2) || q->scalar_type() != k.scalar_type())
                throw BadValue("q and k must agree on tokens, head_dim and type");
            shape->num_q_heads = size32(q->size(1), "q");
        }
        if (turned) rope = rope_of(k.size(2), f, qw, kw, norm, real(eps), truth(interleaved));
    }
};

// k, v, k_cache, v_cache, positions, rows, block_table, k_scale, v_scale, q, q_out, inv_freq, q_weight, k_weight, norm, eps,
// interleaved, max_seqlen, stream
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 19, [&] {
        const Tensor &k = need(a[0], "k"), &v = need(a[1], "v"), &kc = need(a[2], "k_cache"), &vc = need(a[3], "v_cache"),
                     &pos = need(a[4], "positions");
        const Tensor *rows = opt(a[5], "rows"), *bt = opt(a[6], "block_table"), *ks = opt(a[7], "k_scale"), *vs = opt(a[8], "v_scale"),
                     *q = opt(a[9], "q"), *qo = opt(a[10], "q_out"), *f = opt(a[11], "inv_freq"), *qw = opt(a[12], "q_weight"),
                     *kw = opt(a[13], "k_weight");
        like(k, v, "k and v");
        CacheCall c(kc, vc, pos, rows, bt, a[17], k);
        const Written w(k, v, q, qo, f, qw, kw, a[14], a[15], a[16], &c.shape);
        const float *pks = scales(ks, "k_scale", c.shape.num_kv_heads), *pvs = scales(vs, "v_scale", c.shape.num_kv_heads);
        Device dev;
        for (const Tensor* t : {&k, &v, &kc, &vc, &pos, rows, bt, ks, vs, q, qo, f, qw, kw}) dev.add(t);
        void* st = dev.stream(a[18]);
        return enqueue([&] {
            return p_cache_write(&c.shape, c.pages, &c.tokens, w.turned ? &w.rope : nullptr, q ? &w.hq : nullptr, q ? &w.hqo : nullptr, &w.hk, &w.hv,
                                 kc.data_ptr(), vc.data_ptr(), pks, pvs, st);
        });
    });
}

// k, v, k_codes, v_codes, k_steps, v_steps, positions, rows, block_table, k_scale, v_scale, q, q_out, inv_freq, q_weight, k_weight,
// norm, eps, interleaved, max_seqlen, stream
PyObject* cache_write_int4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 21, [&] {
        const Tensor &k = need(a[0], "k"), &v = need(a[1], "v"), &kc = need(a[2], "k_codes"), &vc = need(a[3], "v_codes"),
                     &kst = need(a[4], "k_steps"), &vst = need(a[5], "v_steps"), &pos = need(a[6], "positions");
        const Tensor *rows = opt(a[7], "rows"), *bt = opt(a[8], "block_table"), *ks = opt(a[9], "k_scale"), *vs = opt(a[10], "v_scale"),
                     *q = opt(a[11], "q"), *qo = opt(a[12], "q_out"), *f = opt(a[13], "inv_freq"), *qw = opt(a[14], "q_weight"),
                     *kw = opt(a[15], "k_weight");
        like(k, v, "k and v");
        Int4Cache c(kc, vc, kst, vst, bt, a[19], ks, vs);
        ta_tokens tokens;
        std::memset(&tokens, 0, sizeof tokens);
        tokens_of(pos, rows, k, &c.shape, &tokens);
        const Written w(k, v, q, qo, f, qw, kw, a[16], a[17], a[18], &c.shape);
        Device dev;
        for (const Tensor* t : {&k, &v, &kc, &vc, &kst, &vst, &pos, rows, bt, ks, vs, q, qo, f, qw, kw}) dev.add(t);
        void* st = dev.stream(a[20]);
        return enqueue([&] {
            return p_cache_write_int4(&c.shape, c.pages, &tokens, w.turned ? &w.rope : nullptr, q ? &w.hq : nullptr, q ? &w.hqo : nullptr, &w.hk,
                                      &w.hv, &c.cache, st);
        });
    });
}

// k_codes, v_codes, k_steps, v_steps, positions, rows, block_table, k_scale, v_scale, k_out, v_out, max_seqlen, stream
PyObject* cache_read_int4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        const Tensor &kc = need(a[0], "k_codes"), &vc = need(a[1], "v_codes"), &kst = need(a[2], "k_steps"), &vst = need(a[3], "v_steps"),
                     &pos = need(a[4], "positions"), &ko = need(a[9], "k_out"), &vo = need(a[10], "v_out");
        const Tensor *rows = opt(a[5], "rows"), *bt = opt(a[6], "block_table"), *ks = opt(a[7], "k_scale"), *vs = opt(a[8], "v_scale");
        like(ko, vo, "k_out and v_out");
        Int4Cache c(kc, vc, kst, vst, bt, a[11], ks, vs);
        ta_tokens tokens;
        std::memset(&tokens, 0, sizeof tokens);
        tokens_of(pos, rows, ko, &c.shape, &tokens);
        const ta_heads hk = heads(ko, "k_out", true), hv = heads(vo, "v_out", true);
        Device dev;
        for (const Tensor* t : {&kc, &vc, &kst, &vst, &pos, &ko, &vo, rows, bt, ks, vs}) dev.add(t);
        void* st = dev.stream(a[12]);
        return enqueue([&] { return p_cache_read_int4(&c.shape, c.pages, &tokens, &c.cache, &hk, &hv, st); });
    });
}

// k_cache, v_cache, positions, rows, block_table, k_scale, v_scale, k_out, v_out, max_seqlen, stream
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const Tensor &kc = need(a[0], "k_cache"), &vc = need(a[1], "v_cache"), &pos = need(a[2], "positions"), &ko = need(a[7], "k_out"),
                     &vo = need(a[8], "v_out");
        const Tensor *rows = opt(a[3], "rows"), *bt = opt(a[4], "block_table"), *ks = opt(a[5], "k_scale"), *vs = opt(a[6], "v_scale");
        like(ko, vo, "k_out and v_out");
        CacheCall c(kc, vc, pos, rows, bt, a[9], ko);
        const ta_heads hk = heads(ko, "k_out", true), hv = heads(vo, "v_out", true);
        const float *pks = scales(ks, "k_scale", c.shape.num_kv_heads), *pvs = scales(vs, "v_scale", c.shape.num_kv_heads);
        Device dev;
        for (const Tensor* t : {&kc, &vc, &pos, &ko, &vo, rows, bt, ks, vs}) dev.add(t);
        void* st = dev.stream(a[10]);
        return enqueue([&] { return p_cache_read(&c.shape, c.pages, &c.tokens, kc.data_ptr(), vc.data_ptr(), &hk, &hv, pks, pvs, st); });
    });
}

void check_bounds(const Tensor& b, int64_t pages, int64_t hkv, int64_t d, bool f32) {
    if (b.dim() != 4 || b.size(0) != pages || b.size(1) != hkv || b.size(2) != 2 || b.size(3) != d || !b.is_contiguous() ||
        b.scalar_type() != (f32 ? at::kFloat : at::kBFloat16))
        throw BadValue("bounds must be a contiguous [num_pages, Hkv, 2, d] tensor, float32 for FP32 caches, else bfloat16");
}

// k_pages, block_table, seqlens, bounds, new_tokens, max_seqlen, stream
PyObject* page_bounds(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&] {
        const Tensor &k = need(a[0], "k_pages"), &bt = need(a[1], "block_table"), &len = need(a[2], "seqlens"), &b = need(a[3], "bounds");
        ta_shape s;
        ta_paged_kv pg;
        std::memset(&s, 0, sizeof s);
        std::memset(&pg, 0, sizeof pg);
        pool_shape(k, bt, a[5], &s, &pg);
        s.num_q_heads = s.num_kv_heads;
        check_bounds(b, pg.num_pages, s.num_kv_heads, s.head_dim, s.kv_dtype == TA_F32);
        const int32_t* pl = ints(&len, "seqlens", s.batch);
        const int nt = static_cast<int>(std::min<long long>(std::max<long long>(integer(a[4]), 0), 0x7fffffff));
        Device dev;
        for (const Tensor* t : {&k, &bt, &len, &b}) dev.add(t);
        void* st = dev.stream(a[6]);
        return enqueue([&] { return p_page_bounds(&s, &pg, k.data_ptr(), pl, nt, b.data_ptr(), st); });
    });
}

void check_query(const Tensor& q, const ta_shape& s) {
    if (q.dim() != 3 || q.size(0) != s.batch || q.size(2) != s.head_dim || !q.is_contiguous())
        throw BadValue("q must be a contiguous [B, Hq, d] tensor that agrees with the pages and block_table");
}

// Shape and pages of a selection over `bounds` [num_pages, Hkv, 2, d].
void select_shape(const Tensor& b, const Tensor& bt, PyObject* page, PyObject* max_seqlen, ta_shape* s, ta_paged_kv* pg) {
    if (b.dim() != 4 || (b.scalar_type() != at::kFloat && b.scalar_type() != at::kBFloat16))
        throw BadValue("bounds must be a contiguous [num_pages, Hkv, 2, d] tensor, float32 or bfloat16");
    check_bounds(b, b.size(0), b.size(1), b.size(3), b.scalar_type() == at::kFloat);
    check_table(bt);
    std::memset(s, 0, sizeof *s);
    std::memset(pg, 0, sizeof *pg);
    s->batch = size32(bt.size(0), "block_table");
    s->num_q_heads = s->num_kv_heads = size32(b.size(1), "bounds");
    s->head_dim = size32(b.size(3), "bounds");
    s->kv_dtype = dtype_code(b);
    pg->block_table = bt.const_data_ptr<int32_t>();
    pg->max_pages_per_seq = size32(bt.size(1), "block_table");
    pg->page_size = int32(page, "page_size");
    pg->num_pages = size32(b.size(0), "bounds");
    const int64_t all = bt.size(1) * std::max(0, pg->page_size);
    s->max_seqlen = max_seqlen == Py_None ? static_cast<int32_t>(std::min<int64_t>(all, 0x7fffffff)) : int32(max_seqlen, "max_seqlen");
}

// bounds, block_table, page_size, max_seqlen
PyObject* select_workspace_bytes(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 4, [&] {
        ta_shape s;
        ta_paged_kv pg;
        select_shape(need(a[0], "bounds"), need(a[1], "block_table"), a[2], a[3], &s, &pg);
        return static_cast<long>(p_select_workspace_bytes(&s, &pg));
    });
}

// q, bounds, block_table, seqlens, page_size, num_select, first_pages, last_pages, selected, workspace, max_seqlen, stream
PyObject* select_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        const Tensor &q = need(a[0], "q"), &b = need(a[1], "bounds"), &bt = need(a[2], "block_table"), &len = need(a[3], "seqlens"),
                     &sel = need(a[8], "selected");
        const Tensor* given = opt(a[9], "workspace");
        Device dev;
        for (const Tensor* t : {&q, &b, &bt, &len, &sel, given}) dev.add(t);
        ta_shape s;
        ta_paged_kv pg;
        select_shape(b, bt, a[4], a[10], &s, &pg);
        check_query(q, s);
        s.num_q_heads = size32(q.size(1), "q");
        s.q_dtype = vec_dtype(q);
        const int ns = int32(a[5], "num_select"), first = int32(a[6], "first_pages"), last = int32(a[7], "last_pages");
        if (sel.scalar_type() != at::kInt || sel.dim() != 3 || sel.size(0) != s.batch || sel.size(1) != s.num_kv_heads || sel.size(2) != ns ||
            !sel.is_contiguous())
            throw BadValue("selected must be a contiguous int32 [B, Hkv, num_select] tensor");
        const int32_t* pl = ints(&len, "seqlens", s.batch);
        void* st = dev.stream(a[11]);
        if (given && !given->is_contiguous()) throw BadValue("workspace must be contiguous");
        if (!given && a[11] != Py_None) throw BadValue("a workspace is needed with a stream");
        // (from torch's allocator for the current stream, which the call runs on)
        const Tensor ws = given ? *given
                                : at::empty({static_cast<int64_t>(std::max<size_t>(16, p_select_workspace_bytes(&s, &pg)))},
                                            q.options().dtype(at::kByte));
        return enqueue([&] {
            return p_select_pages(&s, &pg, q.data_ptr(), b.data_ptr(), pl, ns, first, last, static_cast<int32_t*>(sel.data_ptr()), ws.data_ptr(),
                                  ws.nbytes(), st);
        });
    });
}

// q, k_pages, v_pages, block_table, seqlens, selected, out, lse, scale, max_seqlen, k_scale, v_scale, stream
PyObject* decode_selected(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        const Tensor &q = need(a[0], "q"), &k = need(a[1], "k_pages"), &v = need(a[2], "v_pages"), &bt = need(a[3], "block_table"),
                     &len = need(a[4], "seqlens"), &sel = need(a[5], "selected"), &out = need(a[6], "out");
        const Tensor *lse = opt(a[7], "lse"), *ks = opt(a[10], "k_scale"), *vs = opt(a[11], "v_scale");
        ta_shape s;
        ta_paged_kv pg;
        std::memset(&s, 0, sizeof s);
        std::memset(&pg, 0, sizeof pg);
        same_cache(k, v);
        pool_shape(k, bt, a[9], &s, &pg);
        check_query(q, s);
        s.num_q_heads = size32(q.size(1), "q");
        s.q_dtype = vec_dtype(q);
        s.scale = a[8] == Py_None ? 0.f : static_cast<float>(real(a[8]));
        if (sel.scalar_type() != at::kInt || sel.dim() != 3 || sel.size(0) != s.batch || sel.size(1) != s.num_kv_heads || !sel.is_contiguous())
            throw BadValue("selected must be a contiguous int32 [B, Hkv, num_select] tensor");
        if (out.scalar_type() != at::kFloat || !out.sizes().equals(q.sizes()) || !out.is_contiguous())
            throw BadValue("out must be a contiguous float32 [B, Hq, d] tensor");
        if (lse && (lse->scalar_type() != at::kFloat || lse->dim() != 2 || lse->size(0) != q.size(0) || lse->size(1) != q.size(1) ||
                    !lse->is_contiguous()))
            throw BadValue("lse must be a contiguous float32 [B, Hq] tensor");
        const float *pks = scales(ks, "k_scale", s.num_kv_heads), *pvs = scales(vs, "v_scale", s.num_kv_heads);
        const int32_t* pl = ints(&len, "seqlens", s.batch);
        const int ns = size32(sel.size(2), "selected");
        Device dev;
        for (const Tensor* t : {&q, &k, &v, &bt, &len, &sel, &out, lse, ks, vs}) dev.add(t);
        void* st = dev.stream(a[12]);
        return enqueue([&] {
            return p_decode_selected(&s, &pg, q.data_ptr(), k.data_ptr(), v.data_ptr(), pl, sel.const_data_ptr<int32_t>(), ns,
                                     out.data_ptr<float>(), lse ? lse->data_ptr<float>() : nullptr, pks, pvs, st);
        });
    });
}

// Queries [B, Hq, d] or [B, Hq, queries, d], outputs, lengths and window of a call over a row's first and last tokens.
struct Windowed {
    int queries = 1, window, sinks;
    const int32_t* lengths;
    // q, seqlens, window, sinks, out, lse, scale
    Windowed(const Tensor& q, const Tensor& len, PyObject* window_, PyObject* sinks_, const Tensor& out, const Tensor* lse, PyObject* scale, ta_shape* s) {
        const int64_t d = q.dim();
        if ((d != 3 && d != 4) || q.size(0) != s->batch || q.size(d - 1) != s->head_dim || !q.is_contiguous())
            throw BadValue("q must be a contiguous [B, Hq, d] or [B, Hq, queries, d] tensor that agrees with the cache");
        s->num_q_heads = size32(q.size(1), "q");
        s->q_dtype = vec_dtype(q);
        if (d == 4) queries = size32(q.size(2), "q");
        s->scale = scale == Py_None ? 0.f : static_cast<float>(real(scale));
        window = window_ == Py_None ? 0x7fffffff : int32(window_, "window");
        sinks = int32(sinks_, "sinks");
        lengths = ints(&len, "seqlens", s->batch);
        if (out.scalar_type() != at::kFloat || !out.sizes().equals(q.sizes()) || !out.is_contiguous())
            throw BadValue("out must be a contiguous float32 tensor of q's shape");
        if (lse && (lse->scalar_type() != at::kFloat || lse->dim() != d - 1 || !lse->sizes().equals(q.sizes().slice(0, d - 1)) || !lse->is_contiguous()))
            throw BadValue("lse must be a contiguous float32 tensor of q's shape without the channels");
    }
};

// The workspace of a windowed call: the given one, or one from torch's allocator for the current stream.
Tensor window_workspace(const Tensor* given, PyObject* stream, const ta_shape& s, const ta_paged_kv* pages, const Windowed& w, const Tensor& q) {
    if (given) {
        if (!given->is_contiguous()) throw BadValue("workspace must be contiguous");
        return *given;
    }
    const size_t need = p_window_workspace_bytes(&s, pages, w.queries, w.window, w.sinks);
    if (need && stream != Py_None) throw BadValue("a workspace is needed with a stream");
    return need ? at::empty({static_cast<int64_t>(need)}, q.options().dtype(at::kByte)) : Tensor();
}

// cache shape: k_cache or k_codes, block_table, q, window, sinks, max_seqlen; bytes of workspace that the call needs
PyObject* window_workspace_bytes(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const Tensor &k = need(a[0], "the cache"), &q = need(a[2], "q");
        const Tensor* bt = opt(a[1], "block_table");
        ta_shape s;
        ta_paged_kv pg;
        std::memset(&s, 0, sizeof s);
        std::memset(&pg, 0, sizeof pg);
        if (k.dim() != 4 || q.dim() < 3 || q.dim() > 4) throw BadValue("caches must be 4-D, and q 3-D or 4-D");
        if (bt)
            pool_places(k, *bt, a[5], &s, &pg);
        else
            dense_places(k, a[5], &s);
        const bool codes = k.scalar_type() == at::kByte;
        s.head_dim = size32(q.size(q.dim() - 1), "q");
        s.kv_dtype = codes ? static_cast<int>(TA_INT4) : dtype_code(k);
        s.num_q_heads = size32(q.size(1), "q");
        s.q_dtype = vec_dtype(q);
        return static_cast<long>(p_window_workspace_bytes(&s, bt ? &pg : nullptr, q.dim() == 4 ? size32(q.size(2), "q") : 1,
                                                          a[3] == Py_None ? 0x7fffffff : int32(a[3], "window"), int32(a[4], "sinks")));
    });
}

// q, k_cache, v_cache, seqlens, window, sinks, block_table, out, lse, scale, max_seqlen, k_scale, v_scale, workspace, stream
PyObject* decode_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        const Tensor &q = need(a[0], "q"), &k = need(a[1], "k_cache"), &v = need(a[2], "v_cache"), &len = need(a[3], "seqlens"), &out = need(a[7], "out");
        const Tensor *bt = opt(a[6], "block_table"), *lse = opt(a[8], "lse"), *ks = opt(a[11], "k_scale"), *vs = opt(a[12], "v_scale"),
                     *given = opt(a[13], "workspace");
        ta_shape s;
        ta_paged_kv pg;
        std::memset(&s, 0, sizeof s);
        std::memset(&pg, 0, sizeof pg);
        same_cache(k, v);
        if (bt)
            pool_shape(k, *bt, a[10], &s, &pg);
        else
            dense_shape(k, a[10], &s);
        const Windowed w(q, len, a[4], a[5], out, lse, a[9], &s);
        const float *pks = scales(ks, "k_scale", s.num_kv_heads), *pvs = scales(vs, "v_scale", s.num_kv_heads);
        Device dev;
        for (const Tensor* t : {&q, &k, &v, bt, &len, &out, lse, ks, vs, given}) dev.add(t);
        void* st = dev.stream(a[14]);
        const Tensor ws = window_workspace(given, a[14], s, bt ? &pg : nullptr, w, q);
        return enqueue([&] {
            return p_decode_window(&s, bt ? &pg : nullptr, w.queries, w.window, w.sinks, q.data_ptr(), k.data_ptr(), v.data_ptr(), w.lengths,
                                   out.data_ptr<float>(), lse ? lse->data_ptr<float>() : nullptr, pks, pvs, ws.defined() ? ws.data_ptr() : nullptr,
                                   ws.defined() ? ws.nbytes() : 0, st);
        });
    });
}

// q, k_codes, v_codes, k_steps, v_steps, seqlens, window, sinks, block_table, out, lse, scale, max_seqlen, k_scale, v_scale, workspace, stream
PyObject* decode_int4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 17, [&] {
        const Tensor &q = need(a[0], "q"), &kc = need(a[1], "k_codes"), &vc = need(a[2], "v_codes"), &kst = need(a[3], "k_steps"),
                     &vst = need(a[4], "v_steps"), &len = need(a[5], "seqlens"), &out = need(a[9], "out");
        const Tensor *bt = opt(a[8], "block_table"), *lse = opt(a[10], "lse"), *ks = opt(a[13], "k_scale"), *vs = opt(a[14], "v_scale"),
                     *given = opt(a[15], "workspace");
        Int4Cache c(kc, vc, kst, vst, bt, a[12], ks, vs);
        const Windowed w(q, len, a[6], a[7], out, lse, a[11], &c.shape);
        Device dev;
        for (const Tensor* t : {&q, &kc, &vc, &kst, &vst, bt, &len, &out, lse, ks, vs, given}) dev.add(t);
        void* st = dev.stream(a[16]);
        const Tensor ws = window_workspace(given, a[16], c.shape, c.pages, w, q);
        return enqueue([&] {
            return p_decode_int4(&c.shape, c.pages, w.queries, w.window, w.sinks, q.data_ptr(), &c.cache, w.lengths, out.data_ptr<float>(),
                                 lse ? lse->data_ptr<float>() : nullptr, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, st);
        });
    });
}

template <typename F>
bool resolve(void* lib, const char* name, F* f) {
    *f = reinterpret_cast<F>(dlsym(lib, name));
    return *f != nullptr;
}

// Resolve the C entry points of the library at `path` (already loaded by the binding).
PyObject* init(PyObject*, PyObject* path) {
    const char* p = PyUnicode_AsUTF8(path);
    if (!p) return nullptr;
    void* lib = dlopen(p, RTLD_NOW);
    if (!lib || !resolve(lib, "tree_attn_cache_write", &p_cache_write) || !resolve(lib, "tree_attn_cache_read", &p_cache_read) ||
        !resolve(lib, "tree_attn_page_bounds", &p_page_bounds) ||
        !resolve(lib, "tree_attn_select_workspace_bytes", &p_select_workspace_bytes) ||
        !resolve(lib, "tree_attn_select_pages", &p_select_pages) || !resolve(lib, "tree_attn_decode_selected", &p_decode_selected) ||
        !resolve(lib, "tree_attn_cache_write_int4", &p_cache_write_int4) || !resolve(lib, "tree_attn_cache_read_int4", &p_cache_read_int4) ||
        !resolve(lib, "tree_attn_window_workspace_bytes", &p_window_workspace_bytes) ||
        !resolve(lib, "tree_attn_decode_window", &p_decode_window) || !resolve(lib, "tree_attn_decode_int4", &p_decode_int4) ||
        !resolve(lib, "tree_attn_norm_rope", &p_norm_rope)) {
        PyErr_Format(PyExc_RuntimeError, "%s lacks the serving entry points: build it again", p);
        return nullptr;
    }
    Py_RETURN_NONE;
}

#define TA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {{"init", init, METH_O, nullptr},
                           TA_METHOD(norm_rope),
                           TA_METHOD(cache_write),
                           TA_METHOD(cache_read),
                           TA_METHOD(page_bounds),
                           TA_METHOD(select_workspace_bytes),
                           TA_METHOD(select_pages),
                           TA_METHOD(decode_selected),
                           TA_METHOD(cache_write_int4),
                           TA_METHOD(cache_read_int4),
                           TA_METHOD(window_workspace_bytes),
                           TA_METHOD(decode_window),
                           TA_METHOD(decode_int4),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving_calls() { return PyModule_Create(&g_module); }
