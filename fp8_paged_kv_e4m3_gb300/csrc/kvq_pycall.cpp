/*
 * kvq_pycall.cpp -- a CPython module that marshals the calls of the 4-bit cache
 * and the rotary appends.  It checks the tensors (type, device, shape,
 * layout) and calls the C ABI, as kvq.py does through ctypes, but reads the
 * tensors in C++: on small calls, which are as long as their host time, ctypes
 * marshalling costs more than the kernels (a decode call 21.6 us).
 *
 * Every function returns the C ABI's status, or None when an argument is not
 * what a plain call passes; kvq.py then takes its own path, whose checks name
 * the argument.  Of torch only tensors are read (torch.Tensor and Parameter
 * themselves, no subclass).
 */
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>
#include <stdint.h>

#include "kvq.h"

namespace {

/* the library's entry points and torch's objects, set by setup() */
struct {
    __typeof__(&paged_decode_attn_e2m1) decode;
    __typeof__(&paged_decode_attn_e2m1_partial) decode_partial;
    __typeof__(&paged_prefill_attn_e2m1) prefill;
    __typeof__(&kv_append_e2m1) append;
    __typeof__(&kv_gather_e2m1) gather;
    __typeof__(&kv_append_rope_e4m3) rope_e4m3;
    __typeof__(&kv_append_rope_e2m1) rope_e2m1;
    __typeof__(&kv_append_rope_fp16) rope_fp16;
} fn;
PyObject *get_stream, *get_device;
constexpr at::ScalarType t_half = at::kHalf, t_float = at::kFloat, t_int = at::kInt, t_byte = at::kByte;

#define MAX_DIMS 4

/* a pointer of whatever type the C ABI asks for */
struct address {
    void *a = nullptr;
    template <typename T>
    operator T *() const { return static_cast<T *>(a); }
    explicit operator bool() const { return a != nullptr; }
};

struct view {
    address p;
    int64_t dim[MAX_DIMS] = {};
    int64_t stride = 0;  /* between tokens, where asked for */
};

int long_of(PyObject *o, int64_t *x)
{
    if (!o) return 0;
    *x = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return !(*x == -1 && PyErr_Occurred());
}

/* Reads tensor `o`; `heads`: 3 dims of which the last two are contiguous, any stride between tokens.
 * 0 when it is not of this type, number of dims and layout, or not on device `dev` (*dev = -1: any, kept). */
int tensor(PyObject *o, at::ScalarType dtype, int dims, int heads, int64_t *dev, view *v)
try {
    if (!THPVariable_CheckExact(o)) return 0;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.defined() || t.scalar_type() != dtype || t.layout() != at::kStrided || !t.is_cuda() || t.dim() != dims) return 0;
    const int64_t x = t.get_device();
    if (*dev < 0) *dev = x;
    if (x != *dev) return 0;
    const at::IntArrayRef shape = t.sizes(), st = t.strides();
    for (int i = 0; i < dims; ++i) v->dim[i] = shape[i];
    if (heads) {
        if ((v->dim[2] > 1 && st[2] != 1) || (v->dim[1] > 1 && st[1] != v->dim[2])) return 0;
        v->stride = v->dim[1] * v->dim[2];
        if (v->dim[0] > 1) {
            if (st[0] < v->stride) return 0;
            v->stride = st[0];
        }
    } else if (!t.is_contiguous()) {
        return 0;
    }
    v->p.a = t.data_ptr();
    return 1;
} catch (...) {   // a tensor without storage of its own: none of these calls'
    return 0;
}

/* an optional int32 tensor of any length (the error flag): its pointer, NULL for None */
int flag(PyObject *o, int64_t *dev, address *p)
{
    view v;
    p->a = nullptr;
    if (o == Py_None) return 1;
    if (!tensor(o, t_int, 1, 0, dev, &v) || v.dim[0] < 1) return 0;
    *p = v.p;
    return 1;
}

int real(PyObject *o, float *x)
{
    const double d = PyFloat_AsDouble(o);
    *x = (float)d;
    return !(d == -1.0 && PyErr_Occurred());
}

int whole(PyObject *o, int32_t *x)
{
    const long d = PyLong_AsLong(o);
    *x = (int32_t)d;
    return !(d == -1 && PyErr_Occurred()) && d == (long)*x;
}

/* torch's current stream on `dev`, when that is the current device */
int current_stream(int64_t dev, void **stream)
{
    int64_t x;
    if (!long_of(PyObject_CallNoArgs(get_device), &x) || x != dev) return 0;
    PyObject *d = PyLong_FromLongLong(dev);
    if (!d) return 0;
    PyObject *r = PyObject_CallOneArg(get_stream, d);
    Py_DECREF(d);
    if (!r) return 0;
    *stream = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return !PyErr_Occurred();
}

PyObject *not_plain(void)
{
    PyErr_Clear();
    Py_RETURN_NONE;
}

/* a K and a V pool of E2M1 pages, or (page4) of [4][head_dim] elements of `dtype` */
int pools(PyObject *k, PyObject *v, at::ScalarType dtype, int page4, int64_t head_dim, int64_t *dev, view *kc, view *vc)
{
    const int dims = page4 ? 4 : 3;
    if (!tensor(k, dtype, dims, 0, dev, kc) || !tensor(v, dtype, dims, 0, dev, vc)) return 0;
    for (int i = 0; i < dims; ++i)
        if (kc->dim[i] != vc->dim[i]) return 0;
    if (page4) return kc->dim[2] == KVQ_PAGE_SIZE && kc->dim[3] == head_dim;
    return kc->dim[2] == 9 * head_dim / 4;
}

/* (q, k_cache, v_cache, block_tables, context_lens, k_scale, v_scale, workspace, out or None, topk_idx, topk_lens,
 *  num_splits, sm_scale, err_flag, split_pages, flags); out None: the partials alone */
PyObject *py_decode(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    view q, kc, vc, bt, cl, ws, out, idx, tl;
    int64_t dev = -1;
    float ks, vs, sm;
    int32_t splits, pages, flags;
    address err;
    void *stream;
    (void)self;
    if (n != 16 || !tensor(a[0], t_half, 4, 0, &dev, &q) || !pools(a[1], a[2], t_byte, 0, q.dim[3], &dev, &kc, &vc) ||
        !tensor(a[3], t_int, 2, 0, &dev, &bt) || !tensor(a[4], t_int, 1, 0, &dev, &cl) || !real(a[5], &ks) ||
        !real(a[6], &vs) || !tensor(a[7], t_float, 1, 0, &dev, &ws) || !whole(a[11], &splits) || !real(a[12], &sm) ||
        !flag(a[13], &dev, &err) || !whole(a[14], &pages) || !whole(a[15], &flags))
        return not_plain();
    if (bt.dim[0] != q.dim[0] || cl.dim[0] != q.dim[0]) return not_plain();
    if (a[8] != Py_None) {
        if (!tensor(a[8], t_half, 4, 0, &dev, &out)) return not_plain();
        for (int i = 0; i < 4; ++i)
            if (out.dim[i] != q.dim[i]) return not_plain();
    }
    if ((a[9] == Py_None) != (a[10] == Py_None)) return not_plain();
    if (a[9] != Py_None &&
        (!tensor(a[9], t_int, 3, 0, &dev, &idx) || !tensor(a[10], t_int, 1, 0, &dev, &tl) || idx.dim[0] != q.dim[0] ||
         idx.dim[1] != kc.dim[1] || tl.dim[0] != q.dim[0]))
        return not_plain();
    for (int i = 0; i < 4; ++i)
        if (q.dim[i] > INT32_MAX) return not_plain();
    if (kc.dim[1] > INT32_MAX || bt.dim[1] > INT32_MAX || idx.dim[2] > INT32_MAX || !current_stream(dev, &stream))
        return not_plain();
    const kvq_attn_params p = {(int32_t)q.dim[0], (int32_t)q.dim[1], (int32_t)q.dim[2], (int32_t)kc.dim[1],
                               (int32_t)q.dim[3], splits, (int32_t)bt.dim[1], idx.p ? (int32_t)idx.dim[2] : 0, sm, pages,
                               flags};
    const int st = a[8] != Py_None
                       ? fn.decode(q.p, kc.p, vc.p, kc.dim[0], bt.p, cl.p, ks, vs, idx.p, tl.p, ws.p,
                                   (size_t)ws.dim[0] * 4, out.p, &p, err, stream)
                       : fn.decode_partial(q.p, kc.p, vc.p, kc.dim[0], bt.p, cl.p, ks, vs, idx.p, tl.p, ws.p,
                                           (size_t)ws.dim[0] * 4, &p, err, stream);
    return PyLong_FromLong(st);
}

/* (q, k_cache, v_cache, block_tables, context_lens, q_start, k_scale, v_scale, workspace, out, max_q_len, sm_scale, err_flag) */
PyObject *py_prefill(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    view q, kc, vc, bt, cl, qs, ws, out;
    int64_t dev = -1;
    float ks, vs, sm;
    int32_t longest;
    address err;
    void *stream;
    (void)self;
    if (n != 13 || !tensor(a[0], t_half, 3, 0, &dev, &q) || !pools(a[1], a[2], t_byte, 0, q.dim[2], &dev, &kc, &vc) ||
        !tensor(a[3], t_int, 2, 0, &dev, &bt) || !tensor(a[4], t_int, 1, 0, &dev, &cl) ||
        !tensor(a[5], t_int, 1, 0, &dev, &qs) || !real(a[6], &ks) || !real(a[7], &vs) ||
        !tensor(a[8], t_byte, 1, 0, &dev, &ws) || !tensor(a[9], t_half, 3, 0, &dev, &out) || !whole(a[10], &longest) ||
        !real(a[11], &sm) || !flag(a[12], &dev, &err))
        return not_plain();
    if (bt.dim[0] != cl.dim[0] || qs.dim[0] != cl.dim[0] + 1) return not_plain();
    for (int i = 0; i < 3; ++i)
        if (out.dim[i] != q.dim[i] || q.dim[i] > INT32_MAX) return not_plain();
    if (cl.dim[0] > INT32_MAX || kc.dim[1] > INT32_MAX || bt.dim[1] > INT32_MAX || !current_stream(dev, &stream))
        return not_plain();
    const kvq_prefill_params p = {(int32_t)cl.dim[0], (int32_t)q.dim[1], (int32_t)kc.dim[1], (int32_t)q.dim[2],
                                  (int32_t)bt.dim[1], longest, (int32_t)q.dim[0], sm, 0};
    return PyLong_FromLong(fn.prefill(q.p, kc.p, vc.p, kc.dim[0], bt.p, cl.p, qs.p, ks, vs, ws.p, (size_t)ws.dim[0], out.p,
                                      &p, err, stream));
}

/* (k_new, v_new, slot_mapping, k_cache, v_cache, k_scale, v_scale, err_flag) */
PyObject *py_append(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    view k, v, sl, kc, vc;
    int64_t dev = -1;
    float ks, vs;
    address err;
    void *stream;
    (void)self;
    if (n != 8 || !tensor(a[0], t_half, 3, 0, &dev, &k) || !tensor(a[1], t_half, 3, 0, &dev, &v) ||
        !tensor(a[2], t_int, 1, 0, &dev, &sl) || !pools(a[3], a[4], t_byte, 0, k.dim[2], &dev, &kc, &vc) ||
        !real(a[5], &ks) || !real(a[6], &vs) || !flag(a[7], &dev, &err))
        return not_plain();
    for (int i = 0; i < 3; ++i)
        if (k.dim[i] != v.dim[i] || k.dim[i] > INT32_MAX) return not_plain();
    if (sl.dim[0] != k.dim[0] || kc.dim[1] != k.dim[1] || !current_stream(dev, &stream)) return not_plain();
    return PyLong_FromLong(fn.append(k.p, v.p, sl.p, (int32_t)k.dim[0], (int32_t)k.dim[1], (int32_t)k.dim[2], kc.p, vc.p,
                                     kc.dim[0], ks, vs, err, stream));
}

/* (k_cache, v_cache, slots, k_scale, v_scale, k_out, v_out, err_flag) */
PyObject *py_gather(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    view sl, kc, vc, k, v;
    int64_t dev = -1;
    float ks, vs;
    address err;
    void *stream;
    (void)self;
    if (n != 8 || !tensor(a[5], t_half, 3, 0, &dev, &k) || !tensor(a[6], t_half, 3, 0, &dev, &v) ||
        !pools(a[0], a[1], t_byte, 0, k.dim[2], &dev, &kc, &vc) || !tensor(a[2], t_int, 1, 0, &dev, &sl) ||
        !real(a[3], &ks) || !real(a[4], &vs) || !flag(a[7], &dev, &err))
        return not_plain();
    for (int i = 0; i < 3; ++i)
        if (k.dim[i] != v.dim[i] || k.dim[i] > INT32_MAX) return not_plain();
    if (sl.dim[0] != k.dim[0] || kc.dim[1] != k.dim[1] || !current_stream(dev, &stream)) return not_plain();
    return PyLong_FromLong(fn.gather(kc.p, vc.p, kc.dim[0], sl.p, (int32_t)k.dim[0], (int32_t)k.dim[1], (int32_t)k.dim[2],
                                     ks, vs, k.p, v.p, err, stream));
}

/* (kind, q or None, k_new, v_new, positions, table, slot_mapping, q_out or None, k_cache, v_cache, k_scale, v_scale,
 *  flags, err_flag); kind 0 = E4M3, 1 = fp16, 2 = E2M1 */
PyObject *py_rope(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    view q, k, v, pos, tb, sl, qo, kc, vc;
    int64_t dev = -1;
    int32_t kind, flags;
    float ks, vs;
    address err;
    void *stream;
    (void)self;
    if (n != 14 || !whole(a[0], &kind) || !tensor(a[2], t_half, 3, 1, &dev, &k) || !tensor(a[3], t_half, 3, 1, &dev, &v) ||
        !tensor(a[4], t_int, 1, 0, &dev, &pos) || !tensor(a[5], t_float, 2, 0, &dev, &tb) ||
        !tensor(a[6], t_int, 1, 0, &dev, &sl) ||
        !pools(a[8], a[9], kind == 1 ? t_half : t_byte, kind != 2, k.dim[2], &dev, &kc, &vc) || !real(a[10], &ks) ||
        !real(a[11], &vs) || !whole(a[12], &flags) || !flag(a[13], &dev, &err))
        return not_plain();
    for (int i = 0; i < 3; ++i)
        if (k.dim[i] != v.dim[i] || k.dim[i] > INT32_MAX) return not_plain();
    if (pos.dim[0] != k.dim[0] || sl.dim[0] != k.dim[0] || kc.dim[1] != k.dim[1] || tb.dim[0] > INT32_MAX ||
        tb.dim[1] > INT32_MAX || (a[1] == Py_None) != (a[7] == Py_None))
        return not_plain();
    if (a[1] != Py_None) {
        if (!tensor(a[1], t_half, 3, 1, &dev, &q) || !tensor(a[7], t_half, 3, 0, &dev, &qo)) return not_plain();
        for (int i = 0; i < 3; ++i)
            if (q.dim[i] != qo.dim[i]) return not_plain();
        if (q.dim[0] != k.dim[0] || q.dim[2] != k.dim[2] || q.dim[1] < 1 || q.dim[1] > INT32_MAX) return not_plain();
    }
    if (!current_stream(dev, &stream)) return not_plain();
    const kvq_rope_params p = {(int32_t)k.dim[0], (int32_t)q.dim[1], (int32_t)k.dim[1], (int32_t)k.dim[2],
                               (int32_t)tb.dim[1], (int32_t)tb.dim[0], flags, q.stride, k.stride, v.stride};
    const int st =
        kind == 1 ? fn.rope_fp16(q.p, k.p, v.p, pos.p, tb.p, sl.p, qo.p, kc.p, vc.p, kc.dim[0], &p, err, stream)
                  : (kind == 0 ? fn.rope_e4m3 : fn.rope_e2m1)(q.p, k.p, v.p, pos.p, tb.p, sl.p, qo.p, kc.p, vc.p, kc.dim[0],
                                                              ks, vs, &p, err, stream);
    return PyLong_FromLong(st);
}

/* (addresses of the eight entry points in the order of `fn`, current raw stream of a device, current device) */
PyObject *py_setup(PyObject *self, PyObject *args)
{
    PyObject *at;
    (void)self;
    if (!PyArg_ParseTuple(args, "O!OO", &PyTuple_Type, &at, &get_stream, &get_device)) return NULL;
    if (PyTuple_GET_SIZE(at) != 8) {
        PyErr_SetString(PyExc_ValueError, "eight addresses expected");
        return NULL;
    }
    void *p[8];
    for (int i = 0; i < 8; ++i) p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(at, i));
    if (PyErr_Occurred()) return NULL;
    fn.decode = (__typeof__(fn.decode))p[0];
    fn.decode_partial = (__typeof__(fn.decode_partial))p[1];
    fn.prefill = (__typeof__(fn.prefill))p[2];
    fn.append = (__typeof__(fn.append))p[3];
    fn.gather = (__typeof__(fn.gather))p[4];
    fn.rope_e4m3 = (__typeof__(fn.rope_e4m3))p[5];
    fn.rope_e2m1 = (__typeof__(fn.rope_e2m1))p[6];
    fn.rope_fp16 = (__typeof__(fn.rope_fp16))p[7];
    Py_INCREF(get_stream);   /* kept for the life of the process */
    Py_INCREF(get_device);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"setup", py_setup, METH_VARARGS, NULL},
                                {"decode", (PyCFunction)(void (*)(void))py_decode, METH_FASTCALL, NULL},
                                {"prefill", (PyCFunction)(void (*)(void))py_prefill, METH_FASTCALL, NULL},
                                {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, NULL},
                                {"gather", (PyCFunction)(void (*)(void))py_gather, METH_FASTCALL, NULL},
                                {"rope", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};

struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "kvq_pycall", NULL, -1, methods, NULL, NULL, NULL, NULL};

}  // namespace

PyMODINIT_FUNC PyInit_kvq_pycall(void) { return PyModule_Create(&module); }
