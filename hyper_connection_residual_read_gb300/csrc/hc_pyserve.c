/* Python call path of the operators of include/hc_serve.h, as hc_pywindow.c is that of the window
 * operators: the shapes, types and strides of the tensors are read and compared in C, and the
 * library's entry point is called with them. It returns the entry point's status code, or
 * HC_ERR_ARG (-1) for tensors whose shapes or types disagree.
 */
#include "hc_pytensor.h"

/* hc_rotary of hc_serve.h */
struct rotary {
    const void *cos_sin, *axis_of, *q_norm, *k_norm;
    float eps;
    int length, dim, axes, interleaved;
};

typedef int (*rotary_fn)(const struct cache*, const struct rotary*, int, int, int, void*, int64_t, int64_t, void*,
                         int64_t, int64_t, void*, int64_t, int64_t, void*, void*, void*, void*);
typedef int (*shared_fn)(const struct cache*, int, int, int, int, int, int, int, int, float, int, void*, int64_t,
                         int64_t, void*, void*, void*, void*, void*, void*, void*, void*, void*, void*, void*);
typedef int (*sample_fn)(int, int, int, void*, int64_t, void*, void*, void*, void*, void*, void*, void*, void*);

static rotary_fn p_rotary;
static shared_fn p_shared;
static sample_fn p_sample;

/* A tensor or None (p NULL); 1 if there is one. */
static int read_optional(PyObject* o, struct tensor* t) {
    t->p = NULL;
    if (o == Py_None) return 0;
    return read_tensor(o, 0, t) != 0 ? -1 : 1;
}
static int to_float(PyObject* o, float* out) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) return -1;
    *out = (float)v;
    return 0;
}
static int rows3(const struct tensor* t, int type, int64_t tokens, int64_t heads, int64_t dim) {
    return t->type == type && t->dims == 3 && t->dim[0] == tokens && t->dim[1] == heads && t->dim[2] == dim &&
           t->stride[2] == 1;
}

/* rotary(q, k, v, cos_sin, positions, slots, codes, scales, q_out, q_norm, k_norm, eps, axis_of,
 * interleaved, stream); q and q_out, and cos_sin and positions, None together */
static PyObject* py_rotary(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (arguments("rotary", n, 15, (const void*)p_rotary) != 0) return NULL;
    struct cache c;
    struct tensor q, k, v, table, pos, slots, out, qn, kn, axis;
    struct rotary r;
    void* stream;
    int has_q, has_table, has_pos, has_out, has_qn, has_kn, has_axis;
    const int ok = read_cache(args[6], args[7], &c);
    q.p = NULL;
    if (ok < 0 || ((has_q = args[0] != Py_None) && read_tensor(args[0], 1, &q) != 0) ||
        read_tensor(args[1], 1, &k) != 0 || read_tensor(args[2], 1, &v) != 0 ||
        (has_table = read_optional(args[3], &table)) < 0 || (has_pos = read_optional(args[4], &pos)) < 0 ||
        read_tensor(args[5], 0, &slots) != 0 || (has_out = read_optional(args[8], &out)) < 0 ||
        (has_qn = read_optional(args[9], &qn)) < 0 || (has_kn = read_optional(args[10], &kn)) < 0 ||
        to_float(args[11], &r.eps) != 0 || (has_axis = read_optional(args[12], &axis)) < 0)
        return NULL;
    r.interleaved = PyObject_IsTrue(args[13]);
    if (r.interleaved < 0 || to_ptr(args[14], &stream) != 0) return NULL;
    const int64_t t = k.dim[0], heads = has_q ? q.dim[1] : 0;
    if (!ok || k.dims != 3 || k.type > FP32 || !fits(t) || !fits(heads) || !rows3(&k, k.type, t, c.kv_heads, c.head_dim) ||
        !rows3(&v, k.type, t, c.kv_heads, c.head_dim) || !flat1(&slots, I64, t) || has_q != has_out ||
        has_table != has_pos || (has_axis && !has_table))
        return PyLong_FromLong(ERR_ARG);
    if (has_q && (q.dims != 3 || !rows3(&q, k.type, t, heads, c.head_dim) || !flat3(&out, k.type, &q)))
        return PyLong_FromLong(ERR_ARG);
    r.length = r.dim = r.axes = 0;
    if (has_table) {
        if (table.dims != 3 || table.type != FP32 || !table.contiguous || table.dim[1] != 2 || !fits(table.dim[0]) ||
            !fits(2 * table.dim[2]) || pos.type != I32 || !pos.contiguous || pos.dims < 1 || pos.dims > 2 ||
            pos.dim[pos.dims - 1] != t || (pos.dims == 2 && !fits(pos.dim[0])) ||
            (has_axis && !flat1(&axis, I32, table.dim[2])))
            return PyLong_FromLong(ERR_ARG);
        r.length = (int)table.dim[0], r.dim = (int)(2 * table.dim[2]), r.axes = pos.dims == 2 ? (int)pos.dim[0] : 1;
    }
    if ((has_qn && !flat1(&qn, k.type, c.head_dim)) || (has_kn && !flat1(&kn, k.type, c.head_dim)))
        return PyLong_FromLong(ERR_ARG);
    r.cos_sin = table.p, r.axis_of = axis.p, r.q_norm = qn.p, r.k_norm = kn.p;
    return PyLong_FromLong(p_rotary(&c, &r, (int)t, (int)heads, k.type, q.p, has_q ? q.stride[0] : 0,
                                    has_q ? q.stride[1] : 0, k.p, k.stride[0], k.stride[1], v.p, v.stride[0],
                                    v.stride[1], pos.p, slots.p, out.p, stream));
}

/* shared(q, codes, scales, prefix_table, prefix_lens, cu_groups, max_shared, block_table, cu_lens,
 * kv_lens, max_new, workspace, out, lse, mask, scale, stream) */
static PyObject* py_shared(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (arguments("shared", n, 17, (const void*)p_shared) != 0) return NULL;
    struct cache c;
    struct tensor q, ptable, plens, groups, table, cu, kv, work, out, lse, mask;
    int max_shared, max_new, has_lse, has_mask;
    float scale;
    void* stream;
    const int ok = read_cache(args[1], args[2], &c);
    if (ok < 0 || read_tensor(args[0], 1, &q) != 0 || read_tensor(args[3], 0, &ptable) != 0 ||
        read_tensor(args[4], 0, &plens) != 0 || read_tensor(args[5], 0, &groups) != 0 ||
        to_int(args[6], &max_shared) != 0 || read_tensor(args[7], 0, &table) != 0 ||
        read_tensor(args[8], 0, &cu) != 0 || read_tensor(args[9], 0, &kv) != 0 || to_int(args[10], &max_new) != 0 ||
        read_tensor(args[11], 0, &work) != 0 || read_tensor(args[12], 0, &out) != 0 ||
        (has_lse = read_optional(args[13], &lse)) < 0 || (has_mask = read_optional(args[14], &mask)) < 0 ||
        to_float(args[15], &scale) != 0 || to_ptr(args[16], &stream) != 0)
        return NULL;
    const int64_t r = kv.dim[0], g = plens.dim[0];
    if (!ok || q.dims != 3 || q.type > FP32 || q.dim[2] != c.head_dim || q.stride[2] != 1 || !fits(q.dim[0]) ||
        !fits(q.dim[1]) || !flat3(&out, q.type, &q) || (has_lse && !flat2(&lse, FP32, q.dim[0], q.dim[1])) ||
        (has_mask && !flat1(&mask, I64, q.dim[0])) || kv.dims != 1 || plens.dims != 1 || !fits(r) || !fits(g) ||
        table.dims != 2 || !fits(table.dim[1]) || !flat2(&table, I32, r, table.dim[1]) || ptable.dims != 2 ||
        !fits(ptable.dim[1]) || !flat2(&ptable, I32, g, ptable.dim[1]) || !flat1(&plens, I32, g) ||
        !flat1(&groups, I32, g + 1) || !flat1(&cu, I32, r + 1) || !flat1(&kv, I32, r) || work.dims != 1 ||
        !flat1(&work, FP32, work.dim[0]) ||
        work.dim[0] / (c.head_dim + 2) < (q.dim[1] > 0 ? q.dim[0] * q.dim[1] : 0))
        return PyLong_FromLong(ERR_ARG);
    return PyLong_FromLong(p_shared(&c, (int)r, (int)g, (int)q.dim[0], (int)q.dim[1], max_new, max_shared,
                                    (int)table.dim[1], (int)ptable.dim[1], scale, q.type, q.p, q.stride[0],
                                    q.stride[1], cu.p, kv.p, table.p, groups.p, plens.p, ptable.p, mask.p, work.p,
                                    out.p, lse.p, stream));
}

/* sample(logits, uniform, tokens, logprobs, temperature, top_k, top_p, min_p, stream) */
static PyObject* py_sample(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (arguments("sample", n, 9, (const void*)p_sample) != 0) return NULL;
    struct tensor x, u, ids, lp, s[4];
    int has[4];
    void* stream;
    if (read_tensor(args[0], 1, &x) != 0 || read_tensor(args[1], 0, &u) != 0 || read_tensor(args[2], 0, &ids) != 0 ||
        read_tensor(args[3], 0, &lp) != 0)
        return NULL;
    for (int i = 0; i < 4; ++i)
        if ((has[i] = read_optional(args[4 + i], &s[i])) < 0) return NULL;
    if (to_ptr(args[8], &stream) != 0) return NULL;
    const int64_t t = x.dim[0];
    if (x.dims != 2 || x.type > FP32 || !fits(t) || !fits(x.dim[1]) || (x.dim[1] != 1 && x.stride[1] != 1) ||
        !flat1(&u, FP32, t) || !flat1(&ids, I32, t) || !flat1(&lp, FP32, t))
        return PyLong_FromLong(ERR_ARG);
    for (int i = 0; i < 4; ++i)
        if (has[i] && !flat1(&s[i], i == 1 ? I32 : FP32, t)) return PyLong_FromLong(ERR_ARG);
    return PyLong_FromLong(p_sample((int)t, (int)x.dim[1], x.type, x.p, x.stride[0], u.p, s[0].p, s[1].p, s[2].p,
                                    s[3].p, ids.p, lp.p, stream));
}

/* bind(addresses of the three entry points in the order above, then the dtypes bf16, fp16, fp32,
 * int32, int64, uint8) */
static PyObject* py_bind(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    (void)self;
    if (n != 3 + BOUND_TYPES) {
        PyErr_SetString(PyExc_TypeError, "bind takes 3 addresses and 6 dtypes");
        return NULL;
    }
    void* a[3];
    for (int i = 0; i < 3; ++i) {
        a[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return NULL;
    }
    p_rotary = (rotary_fn)a[0];
    p_shared = (shared_fn)a[1];
    p_sample = (sample_fn)a[2];
    bind_types(args + 3);
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))py_bind, METH_FASTCALL, "bind the entry points and dtypes"},
    {"rotary", (PyCFunction)(void (*)(void))py_rotary, METH_FASTCALL, "hc_kv4_append_rotary"},
    {"shared", (PyCFunction)(void (*)(void))py_shared, METH_FASTCALL, "hc_kv4_attention_shared"},
    {"sample", (PyCFunction)(void (*)(void))py_sample, METH_FASTCALL, "hc_sample_tokens"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hcpyserve", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__hcpyserve(void) { return intern_names() == 0 ? PyModule_Create(&module) : NULL; }
