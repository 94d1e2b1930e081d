/* Python call path of the verify-window operators (include/hc_window.h): the shapes, types
 * and strides of the tensors are read and compared in C, and the library's entry point is
 * called with them. Marshalling only, as hc_pycall.c: the module links nothing and calls
 * the entry points whose addresses the binding hands over (bind). It returns the entry
 * point's status code, or HC_ERR_ARG (-1) for tensors whose shapes or types disagree.
 */
#include "hc_pytensor.h"

typedef int (*plan_fn)(int, int, int, int, int, void*, void*, void*, void*, void*, void*, void*, void*,
                       void*, void*, void*, void*);
typedef int (*append_fn)(const struct cache*, int, int, void*, int64_t, int64_t, void*, int64_t, int64_t,
                         void*, void*);
typedef int (*load_fn)(const struct cache*, int, void*, int, void*, void*, void*);
typedef int (*attention_fn)(const struct cache*, int, int, int, int, int, float, int, void*, int64_t,
                            int64_t, void*, void*, void*, void*, void*, void*, void*);
typedef int (*logprobs_fn)(int, int, int, int, void*, int64_t, void*, void*, void*, void*, void*, void*,
                           void*, void*);

static plan_fn p_plan;
static append_fn p_append;
static load_fn p_load;
static attention_fn p_attention;
static logprobs_fn p_logprobs;

/* plan(cached_lens, new_lens, free_blocks, free_count, block_size, block_table, slots, request_of,
 * positions, cu_lens, kv_lens, free_left, stream) */
static PyObject* py_plan(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (arguments("plan", n, 13, (const void*)p_plan) != 0) return NULL;
    static const int at[11] = {0, 1, 2, 3, 5, 6, 7, 8, 9, 10, 11};
    struct tensor t[11];
    for (int i = 0; i < 11; ++i)
        if (read_tensor(args[at[i]], 0, &t[i]) != 0) return NULL;
    int block;
    void* stream;
    if (to_int(args[4], &block) != 0 || to_ptr(args[12], &stream) != 0) return NULL;
    const int64_t r = t[0].dim[0], free = t[2].dim[0], cap = t[5].dim[0], width = t[4].dim[1];
    if (t[0].dims != 1 || t[2].dims != 1 || t[4].dims != 2 || t[5].dims != 1 || !fits(r) || !fits(free) ||
        !fits(cap) || !fits(width) || !flat1(&t[0], I32, r) || !flat1(&t[1], I32, r) ||
        !flat1(&t[2], I32, free) || !flat1(&t[3], I32, 1) || !flat2(&t[4], I32, r, width) ||
        !flat1(&t[5], I64, cap) || !flat1(&t[6], I32, cap) || !flat1(&t[7], I32, cap) ||
        !flat1(&t[8], I32, r + 1) || !flat1(&t[9], I32, r) || !flat1(&t[10], I32, 1))
        return PyLong_FromLong(ERR_ARG);
    return PyLong_FromLong(p_plan((int)r, (int)width, block, (int)cap, (int)free, t[0].p, t[1].p, t[2].p,
                                  t[3].p, t[4].p, t[5].p, t[6].p, t[7].p, t[8].p, t[9].p, t[10].p, stream));
}

/* append(k, v, slots, codes, scales, stream) */
static PyObject* py_append(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (arguments("append", n, 6, (const void*)p_append) != 0) return NULL;
    struct cache c;
    struct tensor k, v, s;
    void* stream;
    const int ok = read_cache(args[3], args[4], &c);
    if (ok < 0 || read_tensor(args[0], 1, &k) != 0 || read_tensor(args[1], 1, &v) != 0 ||
        read_tensor(args[2], 0, &s) != 0 || to_ptr(args[5], &stream) != 0)
        return NULL;
    if (!ok || k.type > FP32 || v.type != k.type || k.dims != 3 || v.dims != 3 || k.dim[0] != v.dim[0] ||
        k.dim[1] != v.dim[1] || k.dim[2] != v.dim[2] || k.dim[1] != c.kv_heads || k.dim[2] != c.head_dim ||
        k.stride[2] != 1 || v.stride[2] != 1 || !fits(k.dim[0]) || !flat1(&s, I64, k.dim[0]))
        return PyLong_FromLong(ERR_ARG);
    return PyLong_FromLong(p_append(&c, (int)k.dim[0], k.type, k.p, k.stride[0], k.stride[1], v.p,
                                    v.stride[0], v.stride[1], s.p, stream));
}

/* load(slots, codes, scales, k_out, v_out, stream) */
static PyObject* py_load(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (arguments("load", n, 6, (const void*)p_load) != 0) return NULL;
    struct cache c;
    struct tensor s, k, v;
    void* stream;
    const int ok = read_cache(args[1], args[2], &c);
    if (ok < 0 || read_tensor(args[0], 0, &s) != 0 || read_tensor(args[3], 0, &k) != 0 ||
        read_tensor(args[4], 0, &v) != 0 || to_ptr(args[5], &stream) != 0)
        return NULL;
    if (!ok || k.type > FP32 || k.dims != 3 || k.dim[1] != c.kv_heads || k.dim[2] != c.head_dim ||
        !fits(k.dim[0]) || !flat3(&k, k.type, &k) || !flat3(&v, k.type, &k) || !flat1(&s, I64, k.dim[0]))
        return PyLong_FromLong(ERR_ARG);
    return PyLong_FromLong(p_load(&c, (int)k.dim[0], s.p, k.type, k.p, v.p, stream));
}

/* attention(q, codes, scales, block_table, cu_lens, kv_lens, max_new, out, lse, mask, scale,
 * stream) */
static PyObject* py_attention(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (arguments("attention", n, 12, (const void*)p_attention) != 0) return NULL;
    struct cache c;
    struct tensor q, table, cu, kv, out, lse, mask;
    int max_new;
    void* stream;
    const int ok = read_cache(args[1], args[2], &c);
    if (ok < 0 || read_tensor(args[0], 1, &q) != 0 || read_tensor(args[3], 0, &table) != 0 ||
        read_tensor(args[4], 0, &cu) != 0 || read_tensor(args[5], 0, &kv) != 0 ||
        to_int(args[6], &max_new) != 0 || read_tensor(args[7], 0, &out) != 0)
        return NULL;
    lse.p = mask.p = NULL;
    if (args[8] != Py_None && read_tensor(args[8], 0, &lse) != 0) return NULL;
    if (args[9] != Py_None && read_tensor(args[9], 0, &mask) != 0) return NULL;
    const double scale = PyFloat_AsDouble(args[10]);
    if ((scale == -1.0 && PyErr_Occurred()) || to_ptr(args[11], &stream) != 0) return NULL;
    const int64_t r = kv.dim[0];
    if (!ok || q.dims != 3 || q.type > FP32 || q.dim[2] != c.head_dim || q.stride[2] != 1 ||
        !fits(q.dim[0]) || !fits(q.dim[1]) || !flat3(&out, q.type, &q) ||
        (args[8] != Py_None && !flat2(&lse, FP32, q.dim[0], q.dim[1])) ||
        (args[9] != Py_None && !flat1(&mask, I64, q.dim[0])) || kv.dims != 1 || !fits(r) || table.dims != 2 ||
        !fits(table.dim[1]) || !flat2(&table, I32, r, table.dim[1]) || !flat1(&cu, I32, r + 1) ||
        !flat1(&kv, I32, r))
        return PyLong_FromLong(ERR_ARG);
    return PyLong_FromLong(p_attention(&c, (int)r, (int)q.dim[0], (int)q.dim[1], max_new, (int)table.dim[1],
                                       (float)scale, q.type, q.p, q.stride[0], q.stride[1], cu.p, kv.p,
                                       table.p, mask.p, out.p, lse.p, stream));
}

/* logprobs(logits, tokens, logprob, entropy, lse, rank, top_ids, top_logprobs, stream) */
static PyObject* py_logprobs(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (arguments("logprobs", n, 9, (const void*)p_logprobs) != 0) return NULL;
    struct tensor x, t[7];
    void* stream;
    if (read_tensor(args[0], 1, &x) != 0) return NULL;
    for (int i = 0; i < 7; ++i)
        if (read_tensor(args[1 + i], 0, &t[i]) != 0) return NULL;
    if (to_ptr(args[8], &stream) != 0) return NULL;
    if (x.dims != 2 || x.type > FP32 || !fits(x.dim[0]) || !fits(x.dim[1]) ||
        (x.dim[1] != 1 && x.stride[1] != 1) || t[5].dims != 2 || !fits(t[5].dim[1]))
        return PyLong_FromLong(ERR_ARG);
    const int64_t r = x.dim[0], top = t[5].dim[1];
    if (!flat1(&t[0], I32, r) || !flat1(&t[1], FP32, r) || !flat1(&t[2], FP32, r) || !flat1(&t[3], FP32, r) ||
        !flat1(&t[4], I32, r) || !flat2(&t[5], I32, r, top) || !flat2(&t[6], FP32, r, top))
        return PyLong_FromLong(ERR_ARG);
    return PyLong_FromLong(p_logprobs((int)r, (int)x.dim[1], (int)top, x.type, x.p, x.stride[0], t[0].p,
                                      t[1].p, t[2].p, t[3].p, t[4].p, t[5].p, t[6].p, stream));
}

/* bind(addresses of the five entry points in the order above, then the dtypes bf16, fp16,
 * fp32, int32, int64, uint8) */
static PyObject* py_bind(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (n != 5 + BOUND_TYPES) {
        PyErr_SetString(PyExc_TypeError, "bind takes 5 addresses and 6 dtypes");
        return NULL;
    }
    void* a[5];
    for (int i = 0; i < 5; ++i) {
        a[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return NULL;
    }
    p_plan = (plan_fn)a[0];
    p_append = (append_fn)a[1];
    p_load = (load_fn)a[2];
    p_attention = (attention_fn)a[3];
    p_logprobs = (logprobs_fn)a[4];
    bind_types(args + 5);
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))py_bind, METH_FASTCALL, "bind the entry points and dtypes"},
    {"plan", (PyCFunction)(void (*)(void))py_plan, METH_FASTCALL, "hc_window_plan"},
    {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, "hc_kv4_append"},
    {"load", (PyCFunction)(void (*)(void))py_load, METH_FASTCALL, "hc_kv4_load"},
    {"attention", (PyCFunction)(void (*)(void))py_attention, METH_FASTCALL, "hc_kv4_attention"},
    {"logprobs", (PyCFunction)(void (*)(void))py_logprobs, METH_FASTCALL, "hc_token_logprobs"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hcpywindow", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__hcpywindow(void) {
    return intern_names() == 0 ? PyModule_Create(&module) : NULL;
}
