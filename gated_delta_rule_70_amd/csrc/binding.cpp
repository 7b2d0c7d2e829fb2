// The short way into the 8-bit and the layer operators from Python: a call whose tensors are all
// given, laid out as the entry point takes them (of the 8-bit operators: contiguous), of matching types
// and shapes and on the current GPU goes straight from here to the C entry point, whose status is returned.  Any other call returns None, and so does one whose
// arguments are refused, and the Python binding takes it: it allocates, handles strides and raises
// the errors.  A call that failed past the checks of its arguments is not handed over: part of it may
// have run, and a second try would add a residual twice.  The checks cost 0.3 us here and 3 us in Python, where the
// kernels of a few tokens take 4 us.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "gdr_i8.h"
#include "gdr_layer.h"

namespace {

using AddNorm = int (*)(const gdr_norm_dims*, const void*, const void*, const void*, int8_t*, float*, void*, void*);
using GatedNorm = int (*)(const gdr_norm_dims*, const void*, const void*, const void*, int8_t*, float*, void*);
using Matmul = int (*)(const gdr_matmul_i8_dims*, const int8_t*, const float*, const int8_t*, const float*, const float*,
                       void* const*, void*);
using Conv = decltype(&gdr_causal_conv);
using QkNorm = decltype(&gdr_qk_norm_rope);
using Scan = decltype(&gdr_selective_scan);
using ScanStep = decltype(&gdr_selective_scan_step);
Conv g_conv = nullptr;
QkNorm g_qk = nullptr;
Scan g_scan = nullptr;
ScanStep g_scan_step = nullptr;
AddNorm g_add = nullptr;
GatedNorm g_gated = nullptr;
Matmul g_matmul = nullptr;
PyObject* g_device = nullptr;  // callables: the current GPU's number, and its current stream's handle
PyObject* g_stream = nullptr;

// A plain dense tensor on a GPU, or nullptr.
const at::Tensor* dense(PyObject* o) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != c10::kStrided || !t.device().is_cuda() || t.is_conj() || t.is_neg() || !t.is_contiguous())
        return nullptr;
    return &t;
}

int code(const at::Tensor& t) {
    return t.scalar_type() == at::kBFloat16 ? GDR_BF16 : t.scalar_type() == at::kFloat ? GDR_F32 : -1;
}

bool same_lead(const at::Tensor& t, const at::Tensor& x, int64_t drop_t, int64_t drop_x) {
    return t.dim() - drop_t == x.dim() - drop_x &&
           t.sizes().slice(0, t.dim() - drop_t) == x.sizes().slice(0, x.dim() - drop_x);
}

// The current stream of GPU dev; false unless dev is the current GPU.
bool stream_of(int dev, void** stream) {
    PyObject* r = PyObject_CallNoArgs(g_device);
    if (!r) return false;
    const long at = PyLong_AsLong(r);
    Py_DECREF(r);
    if (at != dev) return false;
    PyObject* n = PyLong_FromLong(dev);
    if (!n) return false;
    r = PyObject_CallOneArg(g_stream, n);
    Py_DECREF(n);
    if (!r) return false;
    *stream = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return !PyErr_Occurred();
}

PyObject* result(int status) {
    if (status >= GDR_ERR_NULL && status <= GDR_ERR_WORKSPACE) Py_RETURN_NONE;  // nothing was enqueued
    return PyLong_FromLong(status);
}

// Runs f and turns whatever goes wrong into None.
template <typename F>
PyObject* guarded(F f) {
    try {
        PyObject* r = f();
        if (r) return r;
    } catch (...) {
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

// (x, weight, residual, eps, q, scale, out_residual)
PyObject* add_rmsnorm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 7 || !g_add) return nullptr;
        const at::Tensor *x = dense(v[0]), *w = dense(v[1]), *q = dense(v[4]), *s = dense(v[5]);
        const at::Tensor *r = v[2] == Py_None ? nullptr : dense(v[2]), *o = v[6] == Py_None ? nullptr : dense(v[6]);
        if (!x || !w || !q || !s || (v[2] != Py_None) != (r != nullptr) || (r != nullptr) != (o != nullptr)) return nullptr;
        const double eps = PyFloat_AsDouble(v[3]);
        if (PyErr_Occurred() || x->dim() < 1) return nullptr;
        const int64_t D = x->size(-1), rows = s->numel();
        const auto dev = x->device();
        const bool ok = code(*x) >= 0 && (w->scalar_type() == x->scalar_type() || w->scalar_type() == at::kFloat) &&
                        w->dim() == 1 && w->size(0) == D && q->scalar_type() == at::kChar && q->sizes() == x->sizes() &&
                        s->scalar_type() == at::kFloat && same_lead(*s, *x, 0, 1) && w->device() == dev &&
                        q->device() == dev && s->device() == dev && D <= GDR_NORM_MAX_COLS && rows <= GDR_I8_MAX_ROWS &&
                        (!r || (r->sizes() == x->sizes() && r->scalar_type() == x->scalar_type() && r->device() == dev &&
                                o->sizes() == x->sizes() && o->scalar_type() == x->scalar_type() && o->device() == dev));
        void* stream;
        if (!ok || !stream_of(dev.index(), &stream)) return nullptr;
        const gdr_norm_dims d = {(int32_t)rows, 1, (int32_t)D, code(*x), 0, code(*w), (float)eps, D, D, D};
        int st;
        Py_BEGIN_ALLOW_THREADS;
        st = g_add(&d, x->data_ptr(), r ? r->data_ptr() : nullptr, w->data_ptr(), static_cast<int8_t*>(q->data_ptr()),
                   static_cast<float*>(s->data_ptr()), o ? o->data_ptr() : nullptr, stream);
        Py_END_ALLOW_THREADS;
        return result(st);
    });
}

// (o, gate, weight, eps, q, scale)
PyObject* gated_rmsnorm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 6 || !g_gated) return nullptr;
        const at::Tensor *o = dense(v[0]), *g = dense(v[1]), *w = dense(v[2]), *q = dense(v[4]), *s = dense(v[5]);
        if (!o || !g || !w || !q || !s) return nullptr;
        const double eps = PyFloat_AsDouble(v[3]);
        if (PyErr_Occurred() || o->dim() < 2) return nullptr;
        const int64_t H = o->size(-2), V = o->size(-1), rows = s->numel();
        const auto dev = o->device();
        const bool ok = code(*o) >= 0 && code(*g) >= 0 && code(*w) >= 0 && g->sizes() == o->sizes() && w->dim() == 1 &&
                        w->size(0) == V && q->scalar_type() == at::kChar && q->dim() == o->dim() - 1 &&
                        q->size(-1) == H * V && same_lead(*q, *o, 1, 2) && s->scalar_type() == at::kFloat &&
                        same_lead(*s, *o, 0, 2) && g->device() == dev && w->device() == dev && q->device() == dev &&
                        s->device() == dev && H <= GDR_NORM_MAX_COLS && V <= GDR_NORM_MAX_COLS && rows <= GDR_I8_MAX_ROWS;
        void* stream;
        if (!ok || !stream_of(dev.index(), &stream)) return nullptr;
        const gdr_norm_dims d = {(int32_t)rows, (int32_t)H, (int32_t)V, code(*o), code(*g), code(*w), (float)eps,
                                 H * V, H * V, 0};
        int st;
        Py_BEGIN_ALLOW_THREADS;
        st = g_gated(&d, o->data_ptr(), g->data_ptr(), w->data_ptr(), static_cast<int8_t*>(q->data_ptr()),
                     static_cast<float*>(s->data_ptr()), stream);
        Py_END_ALLOW_THREADS;
        return result(st);
    });
}

// (a, a_scale, w, w_scale, bias, out): out a tensor, or a tuple or list of them
PyObject* matmul(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 6 || !g_matmul) return nullptr;
        const at::Tensor *a = dense(v[0]), *as = dense(v[1]), *w = dense(v[2]), *ws = dense(v[3]);
        const at::Tensor* b = v[4] == Py_None ? nullptr : dense(v[4]);
        if (!a || !as || !w || !ws || (v[4] != Py_None) != (b != nullptr) || a->dim() < 1 || w->dim() != 2) return nullptr;
        const bool many = PyTuple_CheckExact(v[5]) || PyList_CheckExact(v[5]);
        const Py_ssize_t count = many ? PySequence_Fast_GET_SIZE(v[5]) : 1;
        if (count < 1 || count > GDR_MATMUL_I8_MAX_OUT) return nullptr;
        const int64_t K = w->size(1), N = w->size(0), M = as->numel();
        const auto dev = a->device();
        if (!(a->scalar_type() == at::kChar && w->scalar_type() == at::kChar && a->size(-1) == K && K <= GDR_MATMUL_I8_MAX_K &&
              as->scalar_type() == at::kFloat && same_lead(*as, *a, 0, 1) && ws->scalar_type() == at::kFloat &&
              ws->dim() == 1 && ws->size(0) == N && M <= GDR_I8_MAX_ROWS && as->device() == dev && w->device() == dev &&
              ws->device() == dev &&
              (!b || (b->scalar_type() == at::kFloat && b->dim() == 1 && b->size(0) == N && b->device() == dev))))
            return nullptr;
        gdr_matmul_i8_dims d = {};
        void* outs[GDR_MATMUL_I8_MAX_OUT];
        int64_t sum = 0;
        for (Py_ssize_t i = 0; i < count; ++i) {
            const at::Tensor* o = dense(many ? PySequence_Fast_GET_ITEM(v[5], i) : v[5]);
            if (!o || code(*o) < 0 || (i > 0 && code(*o) != d.out_dtype) || o->device() != dev || o->dim() != a->dim() ||
                !same_lead(*o, *a, 1, 1) || o->size(-1) > N)
                return nullptr;
            d.out_dtype = code(*o);
            d.out_cols[i] = (int32_t)o->size(-1);
            d.out_stride[i] = o->size(-1);
            outs[i] = o->data_ptr();
            sum += o->size(-1);
        }
        void* stream;
        if (sum != N || N > (1 << 30) || !stream_of(dev.index(), &stream)) return nullptr;
        d.M = (int32_t)M;
        d.K = (int32_t)K;
        d.n_out = (int32_t)count;
        d.a_stride = K;
        d.w_stride = K;
        int st;
        Py_BEGIN_ALLOW_THREADS;
        st = g_matmul(&d, static_cast<const int8_t*>(a->data_ptr()), static_cast<const float*>(as->data_ptr()),
                      static_cast<const int8_t*>(w->data_ptr()), static_cast<const float*>(ws->data_ptr()),
                      b ? static_cast<const float*>(b->data_ptr()) : nullptr, outs, stream);
        Py_END_ALLOW_THREADS;
        return result(st);
    });
}

// ---- layer operators -------------------------------------------------------------------------

// A plain strided tensor on a GPU, or nullptr.
const at::Tensor* strided(PyObject* o) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != c10::kStrided || !t.device().is_cuda() || t.is_conj() || t.is_neg()) return nullptr;
    return &t;
}

// Elements from one row of t to the next, the last `tail` dimensions making a row: false unless a
// row's values lie next to each other and the rows evenly apart.
bool rows_of(const at::Tensor& t, int64_t tail, int64_t* stride) {
    const auto size = t.sizes(), apart = t.strides();
    int64_t row = 1;
    for (int64_t i = t.dim() - 1; i >= t.dim() - tail; --i) {
        if (size[i] != 1 && apart[i] != row) return false;
        row *= size[i];
    }
    int64_t want = -1;
    *stride = row;
    if (t.numel() == 0) return true;
    for (int64_t i = t.dim() - tail - 1; i >= 0; --i) {
        if (size[i] == 1) continue;
        if (want < 0)
            *stride = apart[i];
        else if (apart[i] != want)
            return false;
        want = apart[i] * size[i];
    }
    return true;
}

// An argument that may be None: false for anything else that is not a tensor as wanted.
bool optional(PyObject* o, const at::Tensor** t, bool any_stride = false) {
    *t = o == Py_None ? nullptr : any_stride ? strided(o) : dense(o);
    return o == Py_None || *t != nullptr;
}

bool is(const at::Tensor* t, at::ScalarType type, c10::Device dev, at::IntArrayRef shape) {
    return t->scalar_type() == type && t->device() == dev && t->sizes() == shape;
}
bool none_or(const at::Tensor* t, at::ScalarType type, c10::Device dev, at::IntArrayRef shape) {
    return !t || is(t, type, dev, shape);
}

// The sequences and tokens of x [B, T, D] ([T, D] or [1, T, D] packed, [B, D] single tokens).
bool batch_of(const at::Tensor& x, const at::Tensor* cu, bool step, int64_t* B, int64_t* T) {
    if (step) {
        if (x.dim() != 2 || cu) return false;
        *B = x.size(0), *T = 1;
    } else if (!cu) {
        if (x.dim() != 3) return false;
        *B = x.size(0), *T = x.size(1);
    } else {
        if (!(x.dim() == 2 || (x.dim() == 3 && x.size(0) == 1)) || cu->scalar_type() != at::kInt || cu->dim() != 1 ||
            cu->size(0) < 2 || cu->size(0) > GDR_VARLEN_MAX_SEQS + 1 || cu->device() != x.device())
            return false;
        *B = cu->size(0) - 1, *T = x.size(-2);
    }
    const int64_t D = x.size(-1);
    return D >= 1 && D <= GDR_LAYER_MAX_CHANNELS && *B <= GDR_LAYER_MAX_ROWS && *T <= GDR_LAYER_MAX_ROWS;
}

void* data(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// (x, weight, bias, state, cu_seqlens, activation, out, out_state, want_state, step)
PyObject* causal_conv(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 10 || !g_conv) return nullptr;
        const at::Tensor *x = strided(v[0]), *w = dense(v[1]), *b, *s, *cu, *e;
        if (!x || !w || !optional(v[2], &b) || !optional(v[3], &s) || !optional(v[4], &cu) || !optional(v[7], &e)) return nullptr;
        const bool silu = v[5] != Py_None, step = v[9] == Py_True;
        if (silu && !(PyUnicode_Check(v[5]) && PyUnicode_CompareWithASCIIString(v[5], "silu") == 0)) return nullptr;
        if (!e && v[8] != Py_False) return nullptr;
        const bool many = PyTuple_CheckExact(v[6]) || PyList_CheckExact(v[6]);
        const Py_ssize_t count = many ? PySequence_Fast_GET_SIZE(v[6]) : 1;
        int64_t B, T;
        if (count < 1 || count > GDR_CONV_MAX_OUT || code(*x) < 0 || w->dim() != 2 || !batch_of(*x, cu, step, &B, &T)) return nullptr;
        const int64_t D = x->size(-1), W = w->size(1);
        const auto dev = x->device();
        const auto type = x->scalar_type();
        if (w->size(0) != D || W < 2 || W > 4 || w->device() != dev ||
            (w->scalar_type() != type && w->scalar_type() != at::kFloat) || !none_or(b, w->scalar_type(), dev, {D}) ||
            !none_or(s, type, dev, {B, W - 1, D}) || !none_or(e, type, dev, {B, W - 1, D}))
            return nullptr;
        gdr_conv_dims d = {};
        void* outs[GDR_CONV_MAX_OUT];
        int64_t sum = 0;
        if (!rows_of(*x, 1, &d.x_stride)) return nullptr;
        for (Py_ssize_t i = 0; i < count; ++i) {
            const at::Tensor* o = strided(many ? PySequence_Fast_GET_ITEM(v[6], i) : v[6]);
            if (!o || o->scalar_type() != type || o->device() != dev || o->dim() != x->dim() || !same_lead(*o, *x, 1, 1) ||
                o->size(-1) > D || !rows_of(*o, 1, &d.out_stride[i]))
                return nullptr;
            d.out_cols[i] = (int32_t)o->size(-1);
            outs[i] = o->data_ptr();
            sum += o->size(-1);
        }
        void* stream;
        if (sum != D || !stream_of(dev.index(), &stream)) return nullptr;
        d.B = (int32_t)B, d.T = (int32_t)T, d.D = (int32_t)D, d.W = (int32_t)W;
        d.dtype = code(*x), d.weight_dtype = code(*w), d.flags = silu ? GDR_CONV_SILU : 0, d.n_out = (int32_t)count;
        int st;
        Py_BEGIN_ALLOW_THREADS;
        st = g_conv(&d, static_cast<const int32_t*>(data(cu)), data(x), data(w), data(b), data(s), outs, data(e), stream);
        Py_END_ALLOW_THREADS;
        return result(st);
    });
}

// (q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, out_q, out_k)
PyObject* qk_norm_rope(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 11 || !g_qk) return nullptr;
        const at::Tensor *q = strided(v[0]), *k = strided(v[1]), *oq = strided(v[9]), *ok = strided(v[10]), *qw, *kw, *c, *s, *p;
        if (!q || !k || !oq || !ok || !optional(v[2], &qw) || !optional(v[3], &kw) || !optional(v[4], &c) || !optional(v[5], &s) ||
            !optional(v[6], &p) || (c != nullptr) != (s != nullptr) || (p && !c))
            return nullptr;
        const double eps = PyFloat_AsDouble(v[7]);
        const int interleaved = PyObject_IsTrue(v[8]);
        if (PyErr_Occurred() || q->dim() < 2 || k->dim() != q->dim() || !same_lead(*k, *q, 2, 2)) return nullptr;
        const int64_t H = q->size(-2), HK = k->size(-2), dim = q->size(-1);
        const auto dev = q->device();
        const auto type = q->scalar_type(), wt = qw ? qw->scalar_type() : kw ? kw->scalar_type() : type;
        gdr_qk_dims d = {};
        int64_t rows = 1;
        for (int64_t i = 0; i < q->dim() - 2; ++i) rows *= q->size(i);
        if (code(*q) < 0 || k->scalar_type() != type || k->device() != dev || k->size(-1) != dim || dim < 1 || dim > GDR_QK_MAX_DIM ||
            H < 1 || HK < 1 || H > 65536 || HK > 65536 || rows > GDR_LAYER_MAX_ROWS || (wt != type && wt != at::kFloat) ||
            !none_or(qw, wt, dev, {dim}) || !none_or(kw, wt, dev, {dim}) || !is(oq, type, dev, q->sizes()) ||
            !is(ok, type, dev, k->sizes()) || !rows_of(*q, 2, &d.q_stride) || !rows_of(*k, 2, &d.k_stride) ||
            !rows_of(*oq, 2, &d.out_q_stride) || !rows_of(*ok, 2, &d.out_k_stride))
            return nullptr;
        d.table_rows = 1, d.position_bits = 32, d.period = 1;
        if (q->dim() > 2 && q->size(-3) > 0) d.period = (int32_t)q->size(-3);
        if (c) {
            if (c->dim() != 2 || c->size(0) < 1 || c->size(0) > INT32_MAX || c->size(1) < 1 || 2 * c->size(1) > dim ||
                !is(c, at::kFloat, dev, c->sizes()) || !is(s, at::kFloat, dev, c->sizes()))
                return nullptr;
            d.table_rows = (int32_t)c->size(0), d.rotated = (int32_t)(2 * c->size(1));
        }
        if (p) {
            if ((p->scalar_type() != at::kInt && p->scalar_type() != at::kLong) || p->device() != dev || p->dim() != q->dim() - 2 ||
                !same_lead(*p, *q, 0, 2))
                return nullptr;
            d.position_bits = p->scalar_type() == at::kInt ? 32 : 64;
        }
        void* stream;
        if (!stream_of(dev.index(), &stream)) return nullptr;
        d.rows = (int32_t)rows, d.q_heads = (int32_t)H, d.k_heads = (int32_t)HK, d.dim = (int32_t)dim;
        d.dtype = code(*q), d.weight_dtype = wt == at::kFloat ? GDR_F32 : GDR_BF16;
        d.flags = interleaved ? GDR_QK_INTERLEAVED : 0, d.eps = (float)eps;
        int st;
        Py_BEGIN_ALLOW_THREADS;
        st = g_qk(&d, data(q), data(k), data(qw), data(kw), static_cast<const float*>(data(c)), static_cast<const float*>(data(s)),
                  data(p), data(oq), data(ok), stream);
        Py_END_ALLOW_THREADS;
        return result(st);
    });
}

// (x, dt, A, B, C, D, z, dt_bias, dt_softplus, h0, cu_seqlens, out, ht, want_state, step, workspace)
PyObject* selective_scan(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 16 || !g_scan || !g_scan_step) return nullptr;
        const at::Tensor *x = strided(v[0]), *dt = strided(v[1]), *A = dense(v[2]), *b = strided(v[3]), *c = strided(v[4]);
        const at::Tensor *o = strided(v[11]), *skip, *z, *bias, *h0, *cu, *ht, *ws;
        if (!x || !dt || !A || !b || !c || !o || !optional(v[5], &skip) || !optional(v[6], &z, true) || !optional(v[7], &bias) ||
            !optional(v[9], &h0) || !optional(v[10], &cu) || !optional(v[12], &ht) ||
            !optional(v[15], &ws))
            return nullptr;
        const int softplus = PyObject_IsTrue(v[8]);
        const bool step = v[14] == Py_True;
        if (PyErr_Occurred() || (!ht && v[13] != Py_False)) return nullptr;
        int64_t S, T;
        if (code(*x) < 0 || !batch_of(*x, cu, step, &S, &T) || A->dim() != 2) return nullptr;
        const int64_t D = x->size(-1), N = A->size(1), lead = x->dim() - 1;
        const bool grouped = b->dim() == lead + 2;
        const int64_t G = grouped ? b->size(-2) : 1;
        const auto dev = x->device();
        const auto type = x->scalar_type();
        gdr_scan_dims d = {};
        if (N < 1 || N > GDR_SCAN_MAX_STATES || G < 1 || D % G || !is(A, at::kFloat, dev, {D, N}) || dt->sizes() != x->sizes() ||
            (dt->scalar_type() != type && dt->scalar_type() != at::kFloat) || dt->device() != dev ||
            (!grouped && b->dim() != lead + 1) || b->size(-1) != N || !same_lead(*b, *x, grouped ? 2 : 1, 1) ||
            !is(b, type, dev, b->sizes()) || !is(c, type, dev, b->sizes()) || !none_or(z, type, dev, x->sizes()) ||
            !none_or(skip, at::kFloat, dev, {D}) || !none_or(bias, at::kFloat, dev, {D}) || !none_or(h0, at::kFloat, dev, {S, D, N}) ||
            !none_or(ht, at::kFloat, dev, {S, D, N}) || !is(o, type, dev, x->sizes()) || !rows_of(*x, 1, &d.x_stride) ||
            !rows_of(*dt, 1, &d.dt_stride) || (z && !rows_of(*z, 1, &d.z_stride)) || !rows_of(*b, grouped ? 2 : 1, &d.b_stride) ||
            !rows_of(*c, grouped ? 2 : 1, &d.c_stride) || !rows_of(*o, 1, &d.out_stride))
            return nullptr;
        void* stream;
        if (!stream_of(dev.index(), &stream)) return nullptr;
        d.B = (int32_t)S, d.T = (int32_t)T, d.D = (int32_t)D, d.N = (int32_t)N, d.G = (int32_t)G;
        d.dtype = code(*x), d.dt_dtype = code(*dt), d.flags = softplus ? GDR_SCAN_DT_SOFTPLUS : 0;
        if (ws && (ws->scalar_type() != at::kByte || ws->device() != dev)) return nullptr;
        auto f = [](const at::Tensor* t) { return static_cast<float*>(data(t)); };
        int st;
        Py_BEGIN_ALLOW_THREADS;
        st = step ? g_scan_step(&d, data(x), data(dt), f(A), data(b), data(c), f(skip), data(z), f(bias), f(h0), data(o), f(ht), stream)
                  : g_scan(&d, static_cast<const int32_t*>(data(cu)), data(x), data(dt), f(A), data(b), data(c), f(skip), data(z),
                           f(bias), f(h0), data(o), f(ht), data(ws), ws ? ws->numel() : 0, stream);
        Py_END_ALLOW_THREADS;
        return result(st);
    });
}

// (addresses of gdr_causal_conv, gdr_qk_norm_rope, gdr_selective_scan, gdr_selective_scan_step)
PyObject* bind_layer(PyObject*, PyObject* const* v, Py_ssize_t n) {
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "bind_layer takes four addresses");
        return nullptr;
    }
    void* p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(v[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_conv = reinterpret_cast<Conv>(p[0]);
    g_qk = reinterpret_cast<QkNorm>(p[1]);
    g_scan = reinterpret_cast<Scan>(p[2]);
    g_scan_step = reinterpret_cast<ScanStep>(p[3]);
    Py_RETURN_NONE;
}

// (address of gdr_add_rmsnorm_i8, of gdr_gated_rmsnorm_i8, of gdr_matmul_i8, current_device, current_stream)
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind takes three addresses and two callables");
        return nullptr;
    }
    void* p[3];
    for (int i = 0; i < 3; ++i) {
        p[i] = PyLong_AsVoidPtr(v[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_add = reinterpret_cast<AddNorm>(p[0]);
    g_gated = reinterpret_cast<GatedNorm>(p[1]);
    g_matmul = reinterpret_cast<Matmul>(p[2]);
    Py_INCREF(v[3]);
    Py_INCREF(v[4]);
    Py_XSETREF(g_device, v[3]);
    Py_XSETREF(g_stream, v[4]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"add_rmsnorm", FAST(add_rmsnorm), nullptr},
                         {"gated_rmsnorm", FAST(gated_rmsnorm), nullptr},
                         {"matmul", FAST(matmul), nullptr},
                         {"bind", FAST(bind), nullptr},
                         {"causal_conv", FAST(causal_conv), nullptr},
                         {"qk_norm_rope", FAST(qk_norm_rope), nullptr},
                         {"selective_scan", FAST(selective_scan), nullptr},
                         {"bind_layer", FAST(bind_layer), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    PyObject* m = PyModule_Create(&module);
    // of what bind and the calls take and return: quantized.py refuses another one
    if (m && PyModule_AddIntConstant(m, "VERSION", 2) != 0) Py_CLEAR(m);
    return m;
}
