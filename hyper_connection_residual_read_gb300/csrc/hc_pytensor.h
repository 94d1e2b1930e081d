/* What the Python call modules of the operators share: tensors read in C.
 *
 * A tensor is any object with the attributes dtype and shape (a tuple of ints) and the
 * methods data_ptr(), is_contiguous() and stride(). Each module that includes this has its own
 * copy of the bound types.
 */
#ifndef HC_PYTENSOR_H
#define HC_PYTENSOR_H

#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <stdint.h>

/* hc_kv4_cache of hc_window.h */
struct cache {
    void* codes;
    void* scales;
    int blocks, kv_heads, block_size, head_dim;
};

enum { BF16, FP16, FP32, I32, I64, U8, BOUND_TYPES };
#define OTHER BOUND_TYPES
#define ERR_ARG (-1)
static PyObject* types[BOUND_TYPES];
static PyObject *s_dtype, *s_shape, *s_data_ptr, *s_is_contiguous, *s_stride;

#define MAX_DIM 5
struct tensor {
    void* p;
    int type, dims, contiguous;
    int64_t dim[MAX_DIM], stride[MAX_DIM];
};

static int integers(PyObject* t, int64_t* to) {
    const Py_ssize_t n = PyTuple_Check(t) ? PyTuple_GET_SIZE(t) : -1;
    if (n < 0) {
        PyErr_SetString(PyExc_TypeError, "a tensor's shape and strides are tuples");
        return -1;
    }
    for (Py_ssize_t i = 0; i < n && i < MAX_DIM; ++i) {
        to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
        if (to[i] == -1 && PyErr_Occurred()) return -1;
    }
    return (int)n;
}

/* Reads a tensor; with strides if asked (else whether it is contiguous). -1 with an exception
 * set if it is none. */
static int read_tensor(PyObject* o, int strides, struct tensor* t) {
    PyObject* v = PyObject_GetAttr(o, s_dtype);
    if (v == NULL) return -1;
    t->type = OTHER;
    t->contiguous = 0;
    for (int i = 0; i < MAX_DIM; ++i) t->dim[i] = t->stride[i] = 0;
    for (int i = 0; i < BOUND_TYPES; ++i)
        if (v == types[i]) t->type = i;
    Py_DECREF(v);
    if ((v = PyObject_GetAttr(o, s_shape)) == NULL) return -1;
    t->dims = integers(v, t->dim);
    Py_DECREF(v);
    if (t->dims < 0) return -1;
    if (strides) {
        if ((v = PyObject_CallMethodNoArgs(o, s_stride)) == NULL) return -1;
        const int n = integers(v, t->stride);
        Py_DECREF(v);
        if (n < 0) return -1;
    } else {
        if ((v = PyObject_CallMethodNoArgs(o, s_is_contiguous)) == NULL) return -1;
        t->contiguous = PyObject_IsTrue(v);
        Py_DECREF(v);
    }
    if ((v = PyObject_CallMethodNoArgs(o, s_data_ptr)) == NULL) return -1;
    t->p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return t->p == NULL && PyErr_Occurred() ? -1 : 0;
}

static int fits(int64_t x) { return x >= 0 && x <= INT_MAX; }
static int flat1(const struct tensor* t, int type, int64_t n) {
    return t->type == type && t->dims == 1 && t->contiguous && t->dim[0] == n;
}
static int flat2(const struct tensor* t, int type, int64_t m, int64_t n) {
    return t->type == type && t->dims == 2 && t->contiguous && t->dim[0] == m && t->dim[1] == n;
}
static int flat3(const struct tensor* t, int type, const struct tensor* like) {
    return t->type == type && t->dims == 3 && t->contiguous && t->dim[0] == like->dim[0] &&
           t->dim[1] == like->dim[1] && t->dim[2] == like->dim[2];
}

static int to_int(PyObject* o, int* out) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return -1;
    if (v < INT_MIN || v > INT_MAX) {
        PyErr_SetString(PyExc_OverflowError, "argument out of the range of a C int");
        return -1;
    }
    *out = (int)v;
    return 0;
}
static int to_ptr(PyObject* o, void** out) {
    if (o == Py_None) {
        *out = NULL;
        return 0;
    }
    *out = PyLong_AsVoidPtr(o);
    return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

/* The cache of a codes and a scales tensor: 1 if they agree, 0 if not, -1 with an exception. */
static int read_cache(PyObject* codes, PyObject* scales, struct cache* c) {
    struct tensor k, s;
    if (read_tensor(codes, 0, &k) != 0 || read_tensor(scales, 0, &s) != 0) return -1;
    if (k.type != U8 || k.dims != 5 || !k.contiguous || k.dim[1] != 2 || s.type != BF16 || s.dims != 5 ||
        !s.contiguous || s.dim[4] != 2)
        return 0;
    for (int i = 0; i < 4; ++i)
        if (s.dim[i] != k.dim[i] || !fits(k.dim[i])) return 0;
    if (!fits(2 * k.dim[4])) return 0;
    c->codes = k.p, c->scales = s.p;
    c->blocks = (int)k.dim[0], c->kv_heads = (int)k.dim[2], c->block_size = (int)k.dim[3];
    c->head_dim = (int)(2 * k.dim[4]);
    return 1;
}

static int arguments(const char* name, Py_ssize_t n, Py_ssize_t want, const void* fn) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", name, want);
        return -1;
    }
    if (fn == NULL) {
        PyErr_Format(PyExc_RuntimeError, "%s: not bound to a library", name);
        return -1;
    }
    return 0;
}

/* The dtypes bf16, fp16, fp32, int32, int64, uint8. */
static void bind_types(PyObject* const* given) {
    for (int i = 0; i < BOUND_TYPES; ++i) {
        Py_INCREF(given[i]);
        Py_XSETREF(types[i], given[i]);
    }
}

static int intern_names(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_stride = PyUnicode_InternFromString("stride");
    return s_dtype && s_shape && s_data_ptr && s_is_contiguous && s_stride ? 0 : -1;
}

#endif
