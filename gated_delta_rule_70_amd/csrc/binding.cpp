// The short way into the 8-bit operators from Python: a call whose tensors are all given,
// contiguous, of matching types and shapes and on the current GPU goes straight from here to the
// C entry point, whose status is returned.  Any other call returns None, and so does one whose
// arguments are refused, and the Python binding takes it: it allocates, handles strides and raises
// the errors.  A call that failed past the checks of its arguments is not handed over: part of it may
// have run, and a second try would add a residual twice.  The checks cost 0.3 us here and 3 us in Python, where the
// kernels of a few tokens take 4 us.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "gdr_i8.h"

namespace {

using AddNorm = int (*)(const gdr_norm_dims*, const void*, const void*, const void*, int8_t*, float*, void*, void*);
using GatedNorm = int (*)(const gdr_norm_dims*, const void*, const void*, const void*, int8_t*, float*, void*);
using Matmul = int (*)(const gdr_matmul_i8_dims*, const int8_t*, const float*, const int8_t*, const float*, const float*,
                       void* const*, void*);
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
    if (status >= GDR_ERR_NULL && status <= GDR_ERR_ALIAS) Py_RETURN_NONE;  // nothing was enqueued
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
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    PyObject* m = PyModule_Create(&module);
    // of what bind and the calls take and return: quantized.py refuses another one
    if (m && PyModule_AddIntConstant(m, "VERSION", 1) != 0) Py_CLEAR(m);
    return m;
}
