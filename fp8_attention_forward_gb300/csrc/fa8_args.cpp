// fa8_args.cpp -- Python module that turns torch tensors into fa8_tensor views and calls an entry point of
// libfa8.so.  Argument marshalling only, as the ctypes binding does it, for the calls of a decode step:
// their kernels run for a few microseconds, less than the views took to build in Python (an attention
// call on the host: 32 us with views packed there, 19 with the tensors' attributes read through Python's C
// API, 11 as here, from the tensors themselves).  So are the outputs that a call makes.
//
// Every function takes the entry point's address, then its arguments in the C order (tensor or None,
// number), the stream handle last, and returns the status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <exception>

#include "fa8.h"

namespace {

int dtype_code(at::ScalarType t) {
    switch (t) {
        case at::kFloat8_e4m3fn: return FA8_DTYPE_E4M3;
        case at::kFloat8_e5m2: return FA8_DTYPE_E5M2;
        case at::kBFloat16: return FA8_DTYPE_BF16;
        case at::kHalf: return FA8_DTYPE_F16;
        case at::kFloat: return FA8_DTYPE_F32;
        case at::kInt: return FA8_DTYPE_I32;
        case at::kDouble: return FA8_DTYPE_F64;
        default: return 0;
    }
}

// Fills *v from tensor `t` and points *out at it; None gives a null pointer.  Every tensor has to be on
// the first one's device, *device (-2: not known yet).
int view(PyObject *t, fa8_tensor *v, fa8_tensor **out, long *device) {
    *out = nullptr;
    if (t == Py_None) return 0;
    if (!THPVariable_Check(t)) {
        PyErr_SetString(PyExc_TypeError, "expected a tensor");
        return -1;
    }
    const at::Tensor &x = THPVariable_Unpack(t);
    if (x.layout() != at::kStrided) {
        PyErr_SetString(PyExc_TypeError, "expected a strided tensor");
        return -1;
    }
    v->dtype = dtype_code(x.scalar_type());
    if (!v->dtype) {
        PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(x.scalar_type()));
        return -1;
    }
    const long dev = x.get_device();
    if (*device == -2) *device = dev;
    if (dev != *device) {
        PyErr_SetString(PyExc_ValueError, "all tensors must be on one device");
        return -1;
    }
    const auto n = x.dim();
    if (n > 4) {
        PyErr_SetString(PyExc_ValueError, "at most 4 dims");
        return -1;
    }
    v->data = const_cast<void *>(x.const_data_ptr());
    v->ndim = (int32_t)n;
    const auto shape = x.sizes(), stride = x.strides();
    for (int64_t i = 0; i < 4; ++i) {
        v->shape[i] = i < n ? shape[i] : 0;
        v->stride[i] = i < n ? stride[i] : 0;
    }
    *out = v;
    return 0;
}

constexpr int kMaxViews = 16;
struct Views {
    fa8_tensor v[kMaxViews];
    fa8_tensor *p[kMaxViews];
};

// Reads the arguments `a` by `form`: 't' tensor, 'i' int, 'f' float; then the stream.  a[0] is the entry
// point's address.
int take(PyObject *const *a, Py_ssize_t n, const char *form, Views *w, int *ints, float *f, void **fn, void **stream) try {
    int nt = 0, ni = 0;
    long device = -2;
    const Py_ssize_t len = (Py_ssize_t)strlen(form);
    if (n != len + 2) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, len + 2);
        return -1;
    }
    *fn = PyLong_AsVoidPtr(a[0]);
    for (Py_ssize_t k = 0; k < len; ++k) {
        PyObject *x = a[k + 1];
        if (form[k] == 't') {
            if (view(x, &w->v[nt], &w->p[nt], &device)) return -1;
            ++nt;
        } else if (form[k] == 'i') {
            const long long v = PyLong_AsLongLong(x);
            if (v < INT32_MIN || v > INT32_MAX) PyErr_SetString(PyExc_OverflowError, "argument does not fit 32 bits");
            if (PyErr_Occurred()) return -1;
            ints[ni++] = (int)v;
        } else {
            *f = (float)PyFloat_AsDouble(x);
        }
    }
    *stream = PyLong_AsVoidPtr(a[n - 1]);
    return PyErr_Occurred() ? -1 : 0;
} catch (const std::exception &e) {  // a tensor without storage or strides
    PyErr_SetString(PyExc_TypeError, e.what());
    return -1;
}

#define ENTRY(name, form, proto, ...)                                                            \
    PyObject *name(PyObject *, PyObject *const *a, Py_ssize_t n) {                               \
        Views w;                                                                                 \
        int i[8], st;                                                                            \
        float f = 0.f;                                                                           \
        void *fn, *s;                                                                            \
        (void)f;                                                                                 \
        if (take(a, n, form, &w, i, &f, &fn, &s)) return nullptr;                                \
        fa8_tensor **t = w.p;                                                                    \
        Py_BEGIN_ALLOW_THREADS st = (int)((fa8_status(*) proto)fn)(__VA_ARGS__);                 \
        Py_END_ALLOW_THREADS return PyLong_FromLong(st);                                         \
    }

typedef const fa8_tensor *T;
ENTRY(rope_append, "tttttiifttttttttti", (T, T, T, T, T, int, int, float, T, T, T, fa8_tensor *, fa8_tensor *, fa8_tensor *, T, T, T, int, void *),
      t[0], t[1], t[2], t[3], t[4], i[0], i[1], f, t[5], t[6], t[7], t[8], t[9], t[10], t[11], t[12], t[13], i[2], s)
ENTRY(page_bounds, "tttttii", (T, fa8_tensor *, T, T, T, int, int, void *), t[0], t[1], t[2], t[3], t[4], i[0], i[1], s)
ENTRY(select_pages, "ttttttiiii", (T, T, fa8_tensor *, T, T, T, int, int, int, int, void *), t[0], t[1], t[2], t[3], t[4], t[5], i[0],
      i[1], i[2], i[3], s)
ENTRY(fwd_pages, "ttttttttttttiitf", (T, T, T, T, T, T, T, fa8_tensor *, fa8_tensor *, T, T, T, int, int, T, float, void *), t[0], t[1], t[2],
      t[3], t[4], t[5], t[6], t[7], t[8], t[9], t[10], t[11], i[0], i[1], t[12], f, s)

// empty(q, dtype code, dims to drop, dims to append ..): a new tensor beside q of its shape with the last
// dims replaced.  empty_lse(q): fp32, (requests, heads, tokens) or, packed, (heads, tokens).
PyObject *wrap(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &q) {
    return THPVariable_Wrap(at::empty(shape, at::TensorOptions().dtype(type).device(q.device())));
}
PyObject *empty(PyObject *, PyObject *const *a, Py_ssize_t n) try {
    if (n < 3 || !THPVariable_Check(a[0])) return PyErr_Format(PyExc_TypeError, "empty(tensor, dtype code, dims to drop, dims ..)");
    const at::Tensor &q = THPVariable_Unpack(a[0]);
    const long code = PyLong_AsLong(a[1]), drop = PyLong_AsLong(a[2]);
    at::ScalarType type = at::kFloat;
    for (at::ScalarType t : {at::kFloat8_e4m3fn, at::kBFloat16, at::kHalf, at::kInt})
        if (dtype_code(t) == code) type = t;
    c10::SmallVector<int64_t, 8> shape(q.sizes().begin(), q.sizes().begin() + std::max<long>(0, q.dim() - drop));
    for (Py_ssize_t k = 3; k < n; ++k) shape.push_back(PyLong_AsLongLong(a[k]));
    if (PyErr_Occurred()) return nullptr;
    return wrap(shape, type, q);
} catch (const std::exception &e) {  // no memory, negative dims
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
}
PyObject *empty_lse(PyObject *, PyObject *x) try {
    if (!THPVariable_Check(x)) return PyErr_Format(PyExc_TypeError, "expected a tensor");
    const at::Tensor &q = THPVariable_Unpack(x);
    if (q.dim() == 4) return wrap({q.size(0), q.size(2), q.size(1)}, at::kFloat, q);
    return wrap({q.size(1), q.size(0)}, at::kFloat, q);
} catch (const std::exception &e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
}

PyMethodDef methods[] = {
    {"empty", (PyCFunction)(void (*)(void))empty, METH_FASTCALL, nullptr},
    {"empty_lse", (PyCFunction)empty_lse, METH_O, nullptr},
    {"fa8_rope_append", (PyCFunction)(void (*)(void))rope_append, METH_FASTCALL, nullptr},
    {"fa8_page_bounds", (PyCFunction)(void (*)(void))page_bounds, METH_FASTCALL, nullptr},
    {"fa8_select_pages", (PyCFunction)(void (*)(void))select_pages, METH_FASTCALL, nullptr},
    {"fa8_fwd_pages", (PyCFunction)(void (*)(void))fwd_pages, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "fa8_args", "argument views for libfa8.so", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fa8_args(void) { return PyModule_Create(&module); }
