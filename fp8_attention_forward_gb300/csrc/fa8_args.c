/* fa8_args.c -- CPython module that turns torch tensors into fa8_tensor views and calls an entry point
 * of libfa8.so.  Argument marshalling only, as the ctypes binding does it, for the calls of a decode
 * step: their kernels run for a few microseconds, less than the views took to build in Python.
 * Uses tensors through their Python attributes only (data_ptr, dtype, shape, stride, get_device).
 *
 * Every function takes the entry point's address, then its arguments in the C order (tensor or None,
 * number), the stream handle last, and returns the status.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "fa8.h"

static PyObject *s_data_ptr, *s_dtype, *s_shape, *s_stride, *s_get_device;
static PyObject *g_dtypes[16];
static int g_codes[16], g_ndtypes;

/* Fills *v from tensor `t` and points *out at it; None gives a null pointer.  Every tensor has to be on
 * the first one's device, *device (-2: not known yet). */
static int view(PyObject *t, fa8_tensor *v, fa8_tensor **out, long *device) {
    PyObject *x, *y;
    Py_ssize_t n, i;
    *out = NULL;
    if (t == Py_None) return 0;
    if (!(x = PyObject_GetAttr(t, s_dtype))) return -1;
    Py_DECREF(x); /* dtypes live as long as torch */
    for (i = 0; i < g_ndtypes && g_dtypes[i] != x; ++i) {}
    if (i == g_ndtypes) {
        PyErr_Format(PyExc_TypeError, "unsupported dtype %R", x);
        return -1;
    }
    v->dtype = g_codes[i];
    if (!(x = PyObject_CallMethodNoArgs(t, s_get_device))) return -1;
    const long dev = PyLong_AsLong(x);
    Py_DECREF(x);
    if (*device == -2) *device = dev;
    if (dev != *device) {
        PyErr_SetString(PyExc_ValueError, "all tensors must be on one device");
        return -1;
    }
    if (!(x = PyObject_CallMethodNoArgs(t, s_data_ptr))) return -1;
    v->data = PyLong_AsVoidPtr(x);
    Py_DECREF(x);
    if (!(x = PyObject_GetAttr(t, s_shape))) return -1;
    if (!(y = PyObject_CallMethodNoArgs(t, s_stride))) {
        Py_DECREF(x);
        return -1;
    }
    if (!PyTuple_Check(x) || !PyTuple_Check(y) || PyTuple_GET_SIZE(x) != PyTuple_GET_SIZE(y)) {
        PyErr_SetString(PyExc_TypeError, "expected a tensor");
    } else if ((n = PyTuple_GET_SIZE(x)) > 4) {
        PyErr_SetString(PyExc_ValueError, "at most 4 dims");
    } else {
        v->ndim = (int32_t)n;
        for (i = 0; i < 4; ++i) {
            v->shape[i] = i < n ? PyLong_AsLongLong(PyTuple_GET_ITEM(x, i)) : 0;
            v->stride[i] = i < n ? PyLong_AsLongLong(PyTuple_GET_ITEM(y, i)) : 0;
        }
        *out = v;
    }
    Py_DECREF(x);
    Py_DECREF(y);
    return PyErr_Occurred() ? -1 : 0;
}

#define MAX_VIEWS 16
typedef struct {
    fa8_tensor v[MAX_VIEWS];
    fa8_tensor *p[MAX_VIEWS];
} views;

/* Reads the arguments `a` by `form`: 't' tensor, 'i' int, 'f' float; then the stream.  a[0] is the entry
 * point's address. */
static int take(PyObject *const *a, Py_ssize_t n, const char *form, views *w, int *ints, float *f, void **fn, void **stream) {
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
}

#define ENTRY(name, form, proto, ...)                                                            \
    static PyObject *name(PyObject *self, PyObject *const *a, Py_ssize_t n) {                    \
        views w;                                                                                 \
        int i[8], st;                                                                            \
        float f = 0.f;                                                                           \
        void *fn, *s;                                                                            \
        (void)self;                                                                              \
        (void)f;                                                                                 \
        if (take(a, n, form, &w, i, &f, &fn, &s)) return NULL;                                   \
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

/* set_dtypes([(torch dtype, fa8_dtype), ...]) */
static PyObject *set_dtypes(PyObject *self, PyObject *list) {
    (void)self;
    const Py_ssize_t n = PySequence_Size(list);
    if (n < 0) return NULL;
    if (n > 16) return PyErr_Format(PyExc_ValueError, "at most 16 dtypes");
    g_ndtypes = 0;
    for (Py_ssize_t k = 0; k < n; ++k) {
        PyObject *pair = PySequence_GetItem(list, k), *d;
        int code;
        if (!pair) return NULL;
        if (!PyArg_ParseTuple(pair, "Oi", &d, &code)) {
            Py_DECREF(pair);
            return NULL;
        }
        Py_INCREF(d);
        g_dtypes[g_ndtypes] = d;
        g_codes[g_ndtypes++] = code;
        Py_DECREF(pair);
    }
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"set_dtypes", set_dtypes, METH_O, "the torch dtypes and their fa8_dtype codes"},
    {"fa8_rope_append", (PyCFunction)(void (*)(void))rope_append, METH_FASTCALL, NULL},
    {"fa8_page_bounds", (PyCFunction)(void (*)(void))page_bounds, METH_FASTCALL, NULL},
    {"fa8_select_pages", (PyCFunction)(void (*)(void))select_pages, METH_FASTCALL, NULL},
    {"fa8_fwd_pages", (PyCFunction)(void (*)(void))fwd_pages, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "fa8_args", "argument views for libfa8.so", -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_fa8_args(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_get_device = PyUnicode_InternFromString("get_device");
    if (!s_data_ptr || !s_dtype || !s_shape || !s_stride || !s_get_device) return NULL;
    return PyModule_Create(&module);
}
