// Python extension module of the serving operators: torch tensors to the C ABI
// of include/fusedlin.h.
//
// A decode step issues these calls back to back, and each runs for a few
// microseconds on the GPU, so the host side has to stay near the launch's own
// time (2.2 us on the Grace host). Through ctypes the same checks and argument
// blocks took 10 to 17 us a call, more than the kernels of a decode step. Argument
// marshalling only: every step of the computation is in libfusedlin.so.
//
// Every function takes its arguments by position (the package's Python
// functions, which hold the documentation, pass them on) and raises TypeError
// or ValueError for tensors that do not fit, FusedLinError for a status of the
// library.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <exception>

#include "../../include/fusedlin.h"

namespace {

struct Raised {};  // a Python error is set

PyObject* g_error = nullptr;  // FusedLinError

[[noreturn]] void raise(PyObject* type, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(type, fmt, ap);
    va_end(ap);
    throw Raised{};
}

void check(fl_status st) {
    if (st == FL_OK) return;
    PyObject* v = Py_BuildValue("(is)", (int)st, fl_last_error());
    if (v != nullptr) {
        PyErr_SetObject(g_error, v);
        Py_DECREF(v);
    }
    throw Raised{};
}

std::string shape_of(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

// A tensor argument, or null for None where that is allowed.
const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
    return &THPVariable_Unpack(o);
}

int integer(PyObject* o, const char* name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v != (int)v) raise(PyExc_ValueError, "%s out of range: %ld", name, v);
    return (int)v;
}

float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)v;
}

// The device that the call runs on: the current one, whose stream it is issued on.
struct Call {
    int device;
    void* stream;
    explicit Call(PyObject* s) : device(c10::cuda::current_device()) {
        if (s == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
        } else {
            stream = PyLong_AsVoidPtr(s);
            if (PyErr_Occurred()) throw Raised{};
        }
    }
    // t is on the device, of the dtype and, unless told otherwise, contiguous
    void fits(const at::Tensor* t, const char* name, at::ScalarType dtype, bool contiguous = true) const {
        if (t == nullptr) return;
        if (!t->is_cuda()) raise(PyExc_ValueError, "%s must be a CUDA tensor", name);
        if (t->get_device() != device)
            raise(PyExc_ValueError, "%s is on device %d, the current device is %d", name, (int)t->get_device(), device);
        if (t->scalar_type() != dtype)
            raise(PyExc_TypeError, "%s has dtype %s, expected %s", name, c10::toString(t->scalar_type()), c10::toString(dtype));
        if (contiguous && !t->is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous (row-major)", name);
    }
    at::Tensor empty(at::IntArrayRef sizes, at::ScalarType dtype) const {
        return at::detail::empty_cuda(sizes, dtype, c10::Device(c10::kCUDA, (c10::DeviceIndex)device), std::nullopt);
    }
};

void shaped(const at::Tensor* t, const char* name, at::IntArrayRef shape) {
    if (t != nullptr && t->sizes() != shape)
        raise(PyExc_ValueError, "%s has shape %s, expected %s", name, shape_of(t->sizes()).c_str(), shape_of(shape).c_str());
}

fl_dtype dtype_of(const at::Tensor& t) {
    if (t.scalar_type() == at::kHalf) return FL_F16;
    if (t.scalar_type() == at::kBFloat16) return FL_BF16;
    raise(PyExc_TypeError, "libfusedlin computes on fp16 or bf16 tensors, got %s", c10::toString(t.scalar_type()));
}

int size32(int64_t v, const char* name) {
    if (v != (int)v) raise(PyExc_ValueError, "%s is too large: %lld", name, (long long)v);
    return (int)v;
}

void matrix(const at::Tensor& t, const char* name) {
    if (t.dim() != 2) raise(PyExc_ValueError, "%s has shape %s, expected two axes", name, shape_of(t.sizes()).c_str());
}

void* addr(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

// The tensor an argument holds, or a new one in `own`.
const at::Tensor* given_or_new(const Call& c, PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dtype,
                               at::Tensor& own) {
    if (o == Py_None) {
        own = c.empty(shape, dtype);
        return &own;
    }
    const at::Tensor* t = tensor(o, name);
    c.fits(t, name, dtype);
    shaped(t, name, shape);
    return t;
}

PyObject* as_result(PyObject* o, const at::Tensor& own) {
    if (own.defined()) return THPVariable_Wrap(own);
    Py_INCREF(o);
    return o;
}

PyObject* pair_of(PyObject* a, PyObject* b) {
    PyObject* r = a != nullptr && b != nullptr ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
}

// The workspace given, or one made here.
struct Workspace {
    void* p = nullptr;
    size_t bytes = 0;
    at::Tensor own;
    Workspace(const Call& c, PyObject* o, size_t need) {
        if (o != Py_None) {
            const at::Tensor* t = tensor(o, "workspace");
            if (!t->is_cuda() || !t->is_contiguous())
                raise(PyExc_ValueError, "workspace must be a contiguous CUDA tensor");
            c.fits(t, "workspace", t->scalar_type());
            p = t->data_ptr();
            bytes = t->nbytes();
        } else if (need > 0) {
            own = c.empty({(int64_t)need}, at::kByte);
            p = own.data_ptr();
            bytes = need;
        }
    }
};

// ---------------------------------------------------------------------------
// 4-bit weights
// ---------------------------------------------------------------------------
// w4_quantize(W, group, q, scales, stream) -> (q, scales)
PyObject* w4_quantize(PyObject* const* a) {
    const Call c(a[4]);
    const at::Tensor* W = tensor(a[0], "W");
    matrix(*W, "W");
    const int64_t N = W->size(0), K = W->size(1);
    const int group = integer(a[1], "group");
    if ((group != 32 && group != 64 && group != 128) || K % group != 0)
        raise(PyExc_ValueError, "group must be 32, 64 or 128 and divide K (group %d, K %lld)", group, (long long)K);
    const fl_dtype dt = dtype_of(*W);
    c.fits(W, "W", W->scalar_type());
    at::Tensor own_q, own_s;
    const at::Tensor* q = given_or_new(c, a[2], "q", {N, K / 2}, at::kByte, own_q);
    const at::Tensor* s = given_or_new(c, a[3], "scales", {N, K / group}, W->scalar_type(), own_s);
    check(fl_w4_quantize(W->data_ptr(), q->data_ptr(), s->data_ptr(), size32(N, "N"), size32(K, "K"), group, dt, c.stream));
    return pair_of(as_result(a[2], own_q), as_result(a[3], own_s));
}

// A 4-bit weight with K columns; its row count in N.
fl_w4_weight weight(const Call& c, const char* name, const at::Tensor* q, const at::Tensor* s, const at::Tensor* z,
                    int64_t K, at::ScalarType dtype, int64_t& N) {
    if (q->dim() != 2 || q->size(1) * 2 != K)
        raise(PyExc_ValueError, "%s: q has shape %s, expected [N, %lld]", name, shape_of(q->sizes()).c_str(), (long long)(K / 2));
    N = q->size(0);
    if (s->dim() != 2 || s->size(0) != N || s->size(1) < 1 || K % s->size(1) != 0)
        raise(PyExc_ValueError, "%s: scales has shape %s, expected [%lld, K / group]", name, shape_of(s->sizes()).c_str(), (long long)N);
    c.fits(q, name, at::kByte);
    c.fits(s, name, dtype);
    c.fits(z, name, at::kByte);
    shaped(z, name, s->sizes());
    return fl_w4_weight{q->data_ptr(), s->data_ptr(), addr(z), size32(K / s->size(1), "group")};
}

fl_w4_weight weight_tuple(const Call& c, const char* name, PyObject* o, int64_t K, at::ScalarType dtype, int64_t& N) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) < 2 || PyTuple_GET_SIZE(o) > 3)
        raise(PyExc_TypeError, "%s must be a tuple (q, scales) or (q, scales, zeros)", name);
    const at::Tensor* z = PyTuple_GET_SIZE(o) == 3 ? tensor(PyTuple_GET_ITEM(o, 2), name, true) : nullptr;
    return weight(c, name, tensor(PyTuple_GET_ITEM(o, 0), name), tensor(PyTuple_GET_ITEM(o, 1), name), z, K, dtype, N);
}

// w4_gemm(x, q, scales, zeros, gamma, bias, residual, out, eps, act, workspace, stream) -> out, workspace made here or None
PyObject* w4_gemm(PyObject* const* a) {
    const Call c(a[11]);
    const at::Tensor* x = tensor(a[0], "x");
    matrix(*x, "x");
    const int64_t M = x->size(0), K = x->size(1);
    const at::ScalarType t = x->scalar_type();
    const fl_dtype dt = dtype_of(*x);
    int64_t N = 0;
    const fl_w4_weight W = weight(c, "W", tensor(a[1], "q"), tensor(a[2], "scales"), tensor(a[3], "zeros", true), K, t, N);
    const at::Tensor *gamma = tensor(a[4], "gamma", true), *bias = tensor(a[5], "bias", true),
                     *residual = tensor(a[6], "residual", true);
    c.fits(x, "x", t);
    c.fits(gamma, "gamma", t);
    c.fits(bias, "bias", t);
    c.fits(residual, "residual", t);
    shaped(gamma, "gamma", {K});
    shaped(bias, "bias", {N});
    shaped(residual, "residual", {M, N});
    at::Tensor own;
    const at::Tensor* out = given_or_new(c, a[7], "out", {M, N}, t, own);
    const int m = size32(M, "M"), k = size32(K, "K");
    const Workspace ws(c, a[10], fl_w4_gemm_workspace_size(m, k, gamma != nullptr));
    check(fl_w4_gemm(x->data_ptr(), addr(gamma), &W, addr(bias), addr(residual), out->data_ptr(), m, size32(N, "N"), k,
                     real(a[8]), (fl_act)integer(a[9], "act"), ws.p, ws.bytes, dt, c.stream));
    return pair_of(as_result(a[7], own), as_result(Py_None, ws.own));
}

// w4_swiglu_ffn(x, gamma, Wg, Wu, Wd, bias_down, out, eps, workspace, stream) -> out, workspace made here or None
PyObject* w4_swiglu_ffn(PyObject* const* a) {
    const Call c(a[9]);
    const at::Tensor* x = tensor(a[0], "x");
    matrix(*x, "x");
    const int64_t M = x->size(0), D = x->size(1);
    const at::ScalarType t = x->scalar_type();
    const fl_dtype dt = dtype_of(*x);
    int64_t F = 0, n = 0, d = 0;
    const fl_w4_weight Wg = weight_tuple(c, "Wg", a[2], D, t, F), Wu = weight_tuple(c, "Wu", a[3], D, t, n);
    const fl_w4_weight Wd = weight_tuple(c, "Wd", a[4], F, t, d);
    if (n != F || d != D)
        raise(PyExc_ValueError, "Wu has %lld rows, expected %lld; Wd has %lld, expected %lld", (long long)n, (long long)F,
              (long long)d, (long long)D);
    const at::Tensor *gamma = tensor(a[1], "gamma"), *bias = tensor(a[5], "bias_down", true);
    c.fits(x, "x", t);
    c.fits(gamma, "gamma", t);
    c.fits(bias, "bias_down", t);
    shaped(gamma, "gamma", {D});
    shaped(bias, "bias_down", {D});
    at::Tensor own;
    const at::Tensor* out = given_or_new(c, a[6], "out", {M, D}, t, own);
    const int m = size32(M, "M"), k = size32(D, "D"), f = size32(F, "F");
    const Workspace ws(c, a[8], fl_w4_swiglu_ffn_workspace_size(m, k, f));
    check(fl_w4_swiglu_ffn(x->data_ptr(), gamma->data_ptr(), &Wg, &Wu, &Wd, addr(bias), out->data_ptr(), m, k, f, real(a[7]),
                           ws.p, ws.bytes, dt, c.stream));
    return pair_of(as_result(a[6], own), as_result(Py_None, ws.own));
}

// ---------------------------------------------------------------------------
// rotary positions and the cache
// ---------------------------------------------------------------------------
// A [rows, heads, head_dim] view with contiguous channels; of an axis of one, the
// stride it would have if dense.
struct Heads {
    int64_t rows, heads, dim, row, head;
    Heads(const Call& c, const at::Tensor& t, const char* name, at::ScalarType dtype) {
        if (t.dim() != 3)
            raise(PyExc_ValueError, "%s has shape %s, expected [rows, heads, head_dim]", name, shape_of(t.sizes()).c_str());
        c.fits(&t, name, dtype, false);
        rows = t.size(0), heads = t.size(1), dim = t.size(2);
        if (t.stride(2) != 1 && dim > 1) raise(PyExc_ValueError, "%s: the channels of a head must be contiguous", name);
        head = heads == 1 ? dim : t.stride(1);
        row = rows == 1 ? heads * head : t.stride(0);
    }
};

// rope(q, k, positions, inv_freq, sections, interleaved, inverse, out_q, out_k, stream) -> (out_q, out_k)
PyObject* rope(PyObject* const* a) {
    const Call c(a[9]);
    const at::Tensor *q = tensor(a[0], "q"), *k = tensor(a[1], "k", true), *pos = tensor(a[2], "positions"),
                     *freq = tensor(a[3], "inv_freq");
    const at::ScalarType t = q->scalar_type();
    fl_rope_desc d = {};
    d.dtype = dtype_of(*q);
    const Heads hq(c, *q, "q", t);
    if (pos->dim() != 1 && pos->dim() != 2)
        raise(PyExc_ValueError, "positions has shape %s, expected [rows] or [axes, rows]", shape_of(pos->sizes()).c_str());
    const int64_t axes = pos->dim() == 2 ? pos->size(0) : 1;
    c.fits(pos, "positions", at::kInt, false);
    if (pos->size(-1) != hq.rows) raise(PyExc_ValueError, "positions has %lld rows, expected %lld", (long long)pos->size(-1), (long long)hq.rows);
    if (hq.rows > 1 && pos->stride(-1) != 1) raise(PyExc_ValueError, "positions must be contiguous along the rows");
    c.fits(freq, "inv_freq", at::kFloat);
    if (freq->dim() != 1) raise(PyExc_ValueError, "inv_freq has shape %s, expected [R / 2]", shape_of(freq->sizes()).c_str());
    const int64_t pairs = freq->size(0);
    if (axes < 1 || axes > 4) raise(PyExc_ValueError, "1..4 axes, got %lld", (long long)axes);
    unsigned char axis_of[FL_ROPE_MAX_DIM / 2];
    if (pairs < 1 || pairs > FL_ROPE_MAX_DIM / 2)
        raise(PyExc_ValueError, "inv_freq has %lld frequencies, 1..%d can be used", (long long)pairs, FL_ROPE_MAX_DIM / 2);
    if (a[4] == Py_None) {
        if (axes != 1) raise(PyExc_ValueError, "positions has %lld axes: sections must say which pairs follow which", (long long)axes);
    } else {
        PyObject* s = PySequence_Fast(a[4], "sections must be a sequence");
        if (s == nullptr) throw Raised{};
        int64_t at = 0, bad = PySequence_Fast_GET_SIZE(s) != axes;
        for (int64_t i = 0; i < axes && !bad; ++i) {
            const long n = PyLong_AsLong(PySequence_Fast_GET_ITEM(s, i));
            if (n < 0 || at + n > pairs) {
                PyErr_Clear();
                bad = 1;
            } else {
                for (long j = 0; j < n; ++j) axis_of[at++] = (unsigned char)i;
            }
        }
        Py_DECREF(s);
        if (bad || at != pairs)
            raise(PyExc_ValueError, "sections must give the %lld pairs to the %lld axes", (long long)pairs, (long long)axes);
        if (axes > 1) d.axis_of = axis_of;
    }
    d.rows = size32(hq.rows, "rows"), d.heads_q = size32(hq.heads, "heads"), d.head_dim = size32(hq.dim, "head_dim");
    d.rotary_dim = (int)(2 * pairs), d.n_axes = (int)axes;
    d.interleaved = PyObject_IsTrue(a[5]), d.inverse = PyObject_IsTrue(a[6]);
    if (d.interleaved < 0 || d.inverse < 0) throw Raised{};
    d.positions = pos->data_ptr<int>(), d.inv_freq = freq->data_ptr<float>();
    d.positions_stride = pos->dim() == 2 ? pos->stride(0) : hq.rows;
    auto output = [&](PyObject* o, const char* name, const at::Tensor& like, at::Tensor& own, long long& row, long long& head) {
        if (o == Py_None) {
            own = c.empty(like.sizes(), t);
            row = like.size(1) * like.size(2), head = like.size(2);
            return own.data_ptr();
        }
        const at::Tensor* out = tensor(o, name);
        const Heads h(c, *out, name, t);
        shaped(out, name, like.sizes());
        row = h.row, head = h.head;
        return out->data_ptr();
    };
    at::Tensor own_q, own_k;
    d.q = q->data_ptr(), d.q_row = hq.row, d.q_head = hq.head;
    d.q_out = output(a[7], "out_q", *q, own_q, d.q_out_row, d.q_out_head);
    if (k != nullptr) {
        const Heads hk(c, *k, "k", t);
        shaped(k, "k", {hq.rows, hk.heads, hq.dim});
        d.heads_k = size32(hk.heads, "heads");
        d.k = k->data_ptr(), d.k_row = hk.row, d.k_head = hk.head;
        d.k_out = output(a[8], "out_k", *k, own_k, d.k_out_row, d.k_out_head);
    } else if (a[8] != Py_None) {
        raise(PyExc_ValueError, "out_k without k");
    }
    check(fl_rope(&d, c.stream));
    return pair_of(as_result(a[7], own_q), as_result(a[8], own_k));
}

// (k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_rows, start, stream)
PyObject* kv(PyObject* const* a, bool write) {
    const Call c(a[9]);
    const at::Tensor *k = tensor(a[0], write ? "k" : "out_k"), *v = tensor(a[1], write ? "v" : "out_v"),
                     *kc = tensor(a[2], "k_cache"), *vc = tensor(a[3], "v_cache"), *ks = tensor(a[4], "k_scale"),
                     *vs = tensor(a[5], "v_scale"), *table = tensor(a[6], "page_table"), *cu = tensor(a[7], "cu_rows", true),
                     *start = tensor(a[8], "start", true);
    const at::ScalarType kind = kc->scalar_type(), t = k->scalar_type();
    if (kind != at::kChar && kind != at::kFloat8_e4m3fn)
        raise(PyExc_TypeError, "k_cache has dtype %s, expected int8 or float8_e4m3fn", c10::toString(kind));
    if (kc->dim() != 4)
        raise(PyExc_ValueError, "k_cache has shape %s, expected [pages, page_size, heads, head_dim]", shape_of(kc->sizes()).c_str());
    c.fits(kc, "k_cache", kind);
    c.fits(vc, "v_cache", kind);
    c.fits(ks, "k_scale", at::kFloat);
    c.fits(vs, "v_scale", at::kFloat);
    c.fits(table, "page_table", at::kInt, false);
    c.fits(cu, "cu_rows", at::kInt);
    c.fits(start, "start", at::kInt);
    shaped(vc, "v_cache", kc->sizes());
    const auto places = kc->sizes().slice(0, 3);
    shaped(ks, "k_scale", places);
    shaped(vs, "v_scale", places);
    fl_kv_desc d = {};
    d.dtype = dtype_of(*k);
    d.format = kind == at::kChar ? FL_KV_INT8 : FL_KV_E4M3;
    const Heads hk(c, *k, write ? "k" : "out_k", t), hv(c, *v, write ? "v" : "out_v", t);
    shaped(k, write ? "k" : "out_k", {hk.rows, kc->size(2), kc->size(3)});
    shaped(v, write ? "v" : "out_v", k->sizes());
    if (table->dim() != 2)
        raise(PyExc_ValueError, "page_table has shape %s, expected [sequences, pages]", shape_of(table->sizes()).c_str());
    const int64_t seqs = table->size(0), per = table->size(1);
    if (table->stride(1) != 1 && per > 1) raise(PyExc_ValueError, "page_table must be contiguous along a sequence's pages");
    shaped(cu, "cu_rows", {seqs + 1});
    shaped(start, "start", {seqs});
    d.rows = size32(hk.rows, "rows"), d.heads = size32(hk.heads, "heads"), d.head_dim = size32(hk.dim, "head_dim");
    d.n_pages = size32(kc->size(0), "pages"), d.page_size = size32(kc->size(1), "page_size");
    d.n_seqs = size32(seqs, "sequences"), d.table_pages = size32(per, "pages of a sequence");
    d.table_stride = seqs > 1 ? table->stride(0) : per;
    d.page_table = table->data_ptr<int>();
    d.cu_rows = static_cast<const int*>(addr(cu)), d.start = static_cast<const int*>(addr(start));
    d.k = k->data_ptr(), d.v = v->data_ptr();
    d.k_row = hk.row, d.k_head = hk.head, d.v_row = hv.row, d.v_head = hv.head;
    d.k_cache = kc->data_ptr(), d.v_cache = vc->data_ptr();
    d.k_scale = ks->data_ptr<float>(), d.v_scale = vs->data_ptr<float>();
    check(write ? fl_kv_write(&d, c.stream) : fl_kv_read(&d, c.stream));
    Py_RETURN_NONE;
}
PyObject* kv_write(PyObject* const* a) { return kv(a, true); }
PyObject* kv_read(PyObject* const* a) { return kv(a, false); }

// ---------------------------------------------------------------------------
// attention and the cache's pages
// ---------------------------------------------------------------------------
// attention(q, k, v, cu_q, cu_k, causal, scale, out, stream) -> out
PyObject* attention(PyObject* const* a) {
    const Call c(a[8]);
    const at::Tensor *q = tensor(a[0], "q"), *k = tensor(a[1], "k"), *v = tensor(a[2], "v"), *cu_q = tensor(a[3], "cu_q", true),
                     *cu_k = tensor(a[4], "cu_k", true);
    const at::ScalarType t = q->scalar_type();
    fl_attention_desc d = {};
    d.dtype = dtype_of(*q);
    const Heads hq(c, *q, "q", t), hk(c, *k, "k", t), hv(c, *v, "v", t);
    shaped(k, "k", {hk.rows, hk.heads, hq.dim});
    shaped(v, "v", k->sizes());
    c.fits(cu_q, "cu_q", at::kInt);
    c.fits(cu_k, "cu_k", at::kInt);
    if (cu_k != nullptr && cu_q == nullptr) raise(PyExc_ValueError, "cu_k without cu_q");
    if (cu_q != nullptr && cu_k == nullptr) {
        if (hk.rows != hq.rows) raise(PyExc_ValueError, "cu_k must be given: k has %lld rows, q %lld", (long long)hk.rows, (long long)hq.rows);
        cu_k = cu_q;
    }
    d.n_seqs = 1;
    if (cu_q != nullptr) {
        if (cu_q->dim() != 1 || cu_q->size(0) < 2)
            raise(PyExc_ValueError, "cu_q has shape %s, expected [sequences + 1]", shape_of(cu_q->sizes()).c_str());
        shaped(cu_k, "cu_k", cu_q->sizes());
        d.n_seqs = size32(cu_q->size(0) - 1, "sequences");
        d.cu_q = cu_q->data_ptr<int>(), d.cu_k = cu_k->data_ptr<int>();
    }
    d.causal = PyObject_IsTrue(a[5]);
    if (d.causal < 0) throw Raised{};
    d.scale = a[6] == Py_None ? 1.f / std::sqrt((float)hq.dim) : real(a[6]);
    at::Tensor own;
    if (a[7] == Py_None) {
        own = c.empty(q->sizes(), t);
        d.out = own.data_ptr(), d.out_row = hq.heads * hq.dim, d.out_head = hq.dim;
    } else {
        const at::Tensor* out = tensor(a[7], "out");
        const Heads h(c, *out, "out", t);
        shaped(out, "out", q->sizes());
        d.out = out->data_ptr(), d.out_row = h.row, d.out_head = h.head;
    }
    d.rows_q = size32(hq.rows, "rows"), d.rows_k = size32(hk.rows, "rows"), d.heads_q = size32(hq.heads, "heads");
    d.heads_k = size32(hk.heads, "heads"), d.head_dim = size32(hq.dim, "head_dim");
    d.q = q->data_ptr(), d.k = k->data_ptr(), d.v = v->data_ptr();
    d.q_row = hq.row, d.q_head = hq.head, d.k_row = hk.row, d.k_head = hk.head, d.v_row = hv.row, d.v_head = hv.head;
    check(fl_attention(&d, c.stream));
    return as_result(a[7], own);
}

// The codes, scales and page table of a cache.
struct Cache {
    const at::Tensor *kc, *vc, *ks, *vs, *table;
    fl_kv_format format;
    int64_t seqs, per;
    Cache(const Call& c, PyObject* const* a)
        : kc(tensor(a[0], "k_cache")), vc(tensor(a[1], "v_cache")), ks(tensor(a[2], "k_scale")), vs(tensor(a[3], "v_scale")),
          table(tensor(a[4], "page_table")) {
        const at::ScalarType kind = kc->scalar_type();
        if (kind != at::kChar && kind != at::kFloat8_e4m3fn)
            raise(PyExc_TypeError, "k_cache has dtype %s, expected int8 or float8_e4m3fn", c10::toString(kind));
        if (kc->dim() != 4)
            raise(PyExc_ValueError, "k_cache has shape %s, expected [pages, page_size, heads, head_dim]", shape_of(kc->sizes()).c_str());
        format = kind == at::kChar ? FL_KV_INT8 : FL_KV_E4M3;
        c.fits(kc, "k_cache", kind);
        c.fits(vc, "v_cache", kind);
        c.fits(ks, "k_scale", at::kFloat);
        c.fits(vs, "v_scale", at::kFloat);
        shaped(vc, "v_cache", kc->sizes());
        const auto places = kc->sizes().slice(0, 3);
        shaped(ks, "k_scale", places);
        shaped(vs, "v_scale", places);
        pages(c, table, seqs, per);
    }
    static void pages(const Call& c, const at::Tensor* table, int64_t& seqs, int64_t& per) {
        c.fits(table, "page_table", at::kInt, false);
        if (table->dim() != 2)
            raise(PyExc_ValueError, "page_table has shape %s, expected [sequences, pages]", shape_of(table->sizes()).c_str());
        seqs = table->size(0), per = table->size(1);
        if (table->stride(1) != 1 && per > 1) raise(PyExc_ValueError, "page_table must be contiguous along a sequence's pages");
    }
    fl_kv_pages desc() const {
        fl_kv_pages d = {};
        d.heads = size32(kc->size(2), "heads"), d.head_dim = size32(kc->size(3), "head_dim");
        d.page_size = size32(kc->size(1), "page_size"), d.n_pages = size32(kc->size(0), "pages");
        d.n_seqs = size32(seqs, "sequences"), d.table_pages = size32(per, "pages of a sequence");
        d.table_stride = seqs > 1 ? table->stride(0) : per;
        d.page_table = table->data_ptr<int>();
        d.k_cache = kc->data_ptr(), d.v_cache = vc->data_ptr();
        d.k_scale = ks->data_ptr<float>(), d.v_scale = vs->data_ptr<float>();
        return d;
    }
};
// An int32 tensor of one axis, of n elements.
int* ints(const Call& c, PyObject* o, const char* name, int64_t n) {
    const at::Tensor* t = tensor(o, name);
    c.fits(t, name, at::kInt);
    shaped(t, name, {n});
    return t->data_ptr<int>();
}

// kv_attend(q, k_cache, v_cache, k_scale, v_scale, page_table, start, cu_rows, tree, scale, out, workspace, stream)
// -> out, workspace made here or None
PyObject* kv_attend(PyObject* const* a) {
    const Call c(a[12]);
    const at::Tensor *q = tensor(a[0], "q"), *cu = tensor(a[7], "cu_rows", true), *tree = tensor(a[8], "tree", true);
    const Cache cache(c, a + 1);
    const fl_kv_pages k = cache.desc();
    const at::ScalarType t = q->scalar_type();
    fl_kv_attend_desc d = {};
    d.dtype = dtype_of(*q);
    const Heads hq(c, *q, "q", t);
    if (hq.dim != k.head_dim) raise(PyExc_ValueError, "q has heads of %lld channels, the cache of %d", (long long)hq.dim, k.head_dim);
    d.format = cache.format;
    d.rows = size32(hq.rows, "rows"), d.heads_q = size32(hq.heads, "heads"), d.heads_k = k.heads, d.head_dim = k.head_dim;
    d.page_size = k.page_size, d.n_pages = k.n_pages, d.n_seqs = k.n_seqs, d.table_pages = k.table_pages;
    d.table_stride = k.table_stride, d.page_table = k.page_table;
    d.start = ints(c, a[6], "start", cache.seqs);
    if (cu != nullptr) d.cu_rows = ints(c, a[7], "cu_rows", cache.seqs + 1);
    if (tree != nullptr) {
        c.fits(tree, "tree", at::kBool, false);
        if (tree->dim() != 2 || tree->size(0) != hq.rows)
            raise(PyExc_ValueError, "tree has shape %s, expected [%lld, drafts]", shape_of(tree->sizes()).c_str(), (long long)hq.rows);
        if (tree->stride(1) != 1 && tree->size(1) > 1) raise(PyExc_ValueError, "tree must be contiguous along a row");
        d.tree = static_cast<const unsigned char*>(tree->data_ptr());
        d.tree_cols = size32(tree->size(1), "drafts");
        d.tree_stride = hq.rows > 1 ? tree->stride(0) : tree->size(1);
        if (tree->size(1) == 0 && hq.rows > 0)  // (a tensor without elements has no address: no row sees a draft)
            d.tree = reinterpret_cast<const unsigned char*>(d.start);
    }
    d.scale = a[9] == Py_None ? 1.f / std::sqrt((float)hq.dim) : real(a[9]);
    at::Tensor own;
    if (a[10] == Py_None) {
        own = c.empty(q->sizes(), t);
        d.out = own.data_ptr(), d.out_row = hq.heads * hq.dim, d.out_head = hq.dim;
    } else {
        const at::Tensor* out = tensor(a[10], "out");
        const Heads h(c, *out, "out", t);
        shaped(out, "out", q->sizes());
        d.out = out->data_ptr(), d.out_row = h.row, d.out_head = h.head;
    }
    d.q = q->data_ptr(), d.q_row = hq.row, d.q_head = hq.head;
    d.k_cache = k.k_cache, d.v_cache = k.v_cache, d.k_scale = k.k_scale, d.v_scale = k.v_scale;
    const Workspace ws(c, a[11], fl_kv_attend_workspace_size(&d));
    check(fl_kv_attend(&d, ws.p, ws.bytes, c.stream));
    return pair_of(as_result(a[10], own), as_result(Py_None, ws.own));
}

// kv_compact(k_cache, v_cache, k_scale, v_scale, page_table, start, accepted, stream)
PyObject* kv_compact(PyObject* const* a) {
    const Call c(a[7]);
    const Cache cache(c, a);
    const at::Tensor* acc = tensor(a[6], "accepted");
    c.fits(acc, "accepted", at::kInt);
    if (acc->dim() != 2 || acc->size(0) != cache.seqs)
        raise(PyExc_ValueError, "accepted has shape %s, expected [%lld, most]", shape_of(acc->sizes()).c_str(), (long long)cache.seqs);
    const fl_kv_pages d = cache.desc();
    check(fl_kv_compact(&d, ints(c, a[5], "start", cache.seqs), acc->data_ptr<int>(), size32(acc->size(1), "accepted"), c.stream));
    Py_RETURN_NONE;
}

// kv_fork(k_cache, v_cache, k_scale, v_scale, page_table, refs, parents, children, lengths, workspace, stream)
// -> workspace made here or None
PyObject* kv_fork(PyObject* const* a) {
    const Call c(a[10]);
    const Cache cache(c, a);
    const fl_kv_pages d = cache.desc();
    const int64_t n = tensor(a[7], "children")->numel();
    int* refs = ints(c, a[5], "refs", d.n_pages);
    const int *parents = ints(c, a[6], "parents", n), *children = ints(c, a[7], "children", n), *lengths = ints(c, a[8], "lengths", n);
    const Workspace ws(c, a[9], n == 0 ? 0 : fl_kv_pages_workspace_size(d.n_pages));
    check(fl_kv_fork(&d, refs, parents, children, lengths, size32(n, "children"), ws.p, ws.bytes, c.stream));
    return as_result(Py_None, ws.own);
}

// kv_resize(page_table, refs, lengths, page_size, workspace, stream) -> workspace made here or None
PyObject* kv_resize(PyObject* const* a) {
    const Call c(a[5]);
    const at::Tensor *table = tensor(a[0], "page_table"), *refs = tensor(a[1], "refs");
    int64_t seqs, per;
    Cache::pages(c, table, seqs, per);
    fl_kv_pages d = {};
    c.fits(refs, "refs", at::kInt);
    if (refs->dim() != 1) raise(PyExc_ValueError, "refs has shape %s, expected [pages]", shape_of(refs->sizes()).c_str());
    d.n_pages = size32(refs->size(0), "pages"), d.page_size = integer(a[3], "page_size");
    d.n_seqs = size32(seqs, "sequences"), d.table_pages = size32(per, "pages of a sequence");
    d.table_stride = seqs > 1 ? table->stride(0) : per;
    d.page_table = table->data_ptr<int>();
    const Workspace ws(c, a[4], fl_kv_pages_workspace_size(d.n_pages));
    check(fl_kv_resize(&d, refs->data_ptr<int>(), ints(c, a[2], "lengths", seqs), ws.p, ws.bytes, c.stream));
    return as_result(Py_None, ws.own);
}

// FusedLinError, told once by the package
PyObject* set_error(PyObject* const* a) {
    Py_INCREF(a[0]);
    Py_XSETREF(g_error, a[0]);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised&) {
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define FL_METHOD(NAME, N) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<NAME, N>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FL_METHOD(set_error, 1),      FL_METHOD(w4_quantize, 5), FL_METHOD(w4_gemm, 12),
                         FL_METHOD(w4_swiglu_ffn, 10), FL_METHOD(rope, 10),       FL_METHOD(kv_write, 10),
                         FL_METHOD(kv_read, 10),       FL_METHOD(attention, 9),   FL_METHOD(kv_attend, 13),
                         FL_METHOD(kv_compact, 8),     FL_METHOD(kv_fork, 11),    FL_METHOD(kv_resize, 6),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding() { return PyModule_Create(&module); }
