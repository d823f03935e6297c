/* The usual call of a mixture-of-experts operator in one step, for CPython: plain torch tensors on the
 * current GPU, the current stream, every argument as binding.py's functions want it. A function here
 * looks at its arguments, makes the outputs that are not given, calls the library and returns what
 * binding.py's function of that name returns; where anything is not as usual it returns None and has
 * done nothing, and binding.py goes the long way, whose checks say what is wrong (so too where this part
 * was not built). What is accepted here is a part of what is accepted there. A tensor is read through its Python attributes, so nothing
 * depends on torch's binary interface.
 *
 * Why: for few tokens these operators' kernels take 3 to 9 us and the launch 3.3. A call here takes 4.6
 * us (route, outputs given), 4.7 (combine), 5.1 (dispatch) and 5.3 (product); through binding.py's
 * checks and ctypes 6.8, 6.9, 7.4 and 9.1. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>
#include <stdint.h>

#include "blockwise_fp8.h"

/* ---- what bind() is given */
static PyObject *tensor_type, *error_type, *get_stream, *get_device;
enum { F32, BF16, I32, I64, U8, FP8, TYPES };
static PyObject* types[TYPES];
static __typeof__(&moe_route) call_route;
static __typeof__(&moe_route_backward) call_route_backward;
static __typeof__(&moe_plan_workspace) call_plan_workspace;
static __typeof__(&moe_plan) call_plan;
static __typeof__(&moe_dispatch) call_dispatch;
static __typeof__(&moe_combine) call_combine;
static __typeof__(&moe_combine_backward) call_combine_backward;
static __typeof__(&gemm_1x128_128x128_routed) call_product;

static PyObject *n_dtype, *n_shape, *n_stride, *n_get_device, *n_data_ptr, *n_new_empty, *n_dtype_only;

/* ---- tensors */
typedef struct {
    PyObject* t;    /* borrowed; owned by the call where it made the tensor */
    int type, dims; /* index into types; 1 to 3 */
    int64_t n[3], s[3];
    long device;
    void* p;
    int made;
} View;

static int ints(PyObject* tuple, int64_t* out, int* count) {
    if (tuple == NULL || !PyTuple_Check(tuple)) return 0;
    const Py_ssize_t n = PyTuple_GET_SIZE(tuple);
    if (n < 1 || n > 3) return 0;
    for (Py_ssize_t i = 0; i < n; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
        if (out[i] == -1 && PyErr_Occurred()) return 0;
    }
    *count = (int)n;
    return 1;
}

static int place(PyObject* t, View* v) {
    PyObject* o = PyObject_CallMethodNoArgs(t, n_get_device);
    v->device = o != NULL ? PyLong_AsLong(o) : -1;
    Py_XDECREF(o);
    if (v->device < 0) return 0;
    o = PyObject_CallMethodNoArgs(t, n_data_ptr);
    v->p = o != NULL ? PyLong_AsVoidPtr(o) : NULL;
    Py_XDECREF(o);
    return !PyErr_Occurred();
}

/* A plain tensor of 1 to 3 dimensions on a GPU. */
static int look(PyObject* t, View* v) {
    if ((PyObject*)Py_TYPE(t) != tensor_type) return 0;
    PyObject* o = PyObject_GetAttr(t, n_dtype);
    v->type = TYPES;
    for (int i = 0; i < TYPES; ++i)
        if (o == types[i]) v->type = i;
    Py_XDECREF(o);
    if (v->type == TYPES) return 0;
    o = PyObject_GetAttr(t, n_shape);
    int ok = ints(o, v->n, &v->dims), dims = 0;
    Py_XDECREF(o);
    if (!ok) return 0;
    o = PyObject_CallMethodNoArgs(t, n_stride);
    ok = ints(o, v->s, &dims) && dims == v->dims;
    Py_XDECREF(o);
    v->t = t;
    v->made = 0;
    return ok && place(t, v);
}

/* rows contiguous, at a stride the library takes */
static int rows_at_stride(const View* v) { return v->dims == 2 && v->n[0] > 0 && v->n[1] > 0 && v->s[1] == 1 && v->s[0] >= v->n[1]; }
static int64_t stride(const View* v) { return v->n[0] > 1 ? v->s[0] : v->n[1]; } /* of the rows */
static int dense2(const View* v, int type, int64_t a, int64_t b) {
    return v->type == type && v->dims == 2 && v->n[0] == a && v->n[1] == b && (b == 1 || v->s[1] == 1) && (a == 1 || v->s[0] == b);
}
static int dense1(const View* v, int type, int64_t a) { return v->type == type && v->dims == 1 && v->n[0] == a && (a == 1 || v->s[0] == 1); }
static int matrix(PyObject* t, View* v, int type, int64_t a, int64_t b) {
    return look(t, v) && v->type == type && rows_at_stride(v) && v->n[0] == a && v->n[1] == b;
}

/* A new dense tensor on like's device: b < 0 for one dimension. */
static int make(const View* like, View* v, int type, int64_t a, int64_t b) {
    PyObject* shape = b < 0 ? PyLong_FromLongLong(a) : Py_BuildValue("(LL)", (long long)a, (long long)b);
    if (shape == NULL) return 0;
    PyObject* args[3] = {like->t, shape, types[type]};
    v->t = PyObject_VectorcallMethod(n_new_empty, args, 2, type == like->type ? NULL : n_dtype_only);
    Py_DECREF(shape);
    v->made = v->t != NULL;
    v->type = type;
    v->dims = b < 0 ? 1 : 2;
    v->n[0] = a;
    v->n[1] = v->s[0] = b;
    return v->made && place(v->t, v);
}

static int number(PyObject* o, int64_t* out) {
    if (!PyLong_CheckExact(o)) return 0;
    *out = PyLong_AsLongLong(o);
    return !(*out == -1 && PyErr_Occurred());
}
static int flag(PyObject* o, int* out) {
    if (!PyBool_Check(o)) return 0;
    *out = o == Py_True;
    return 1;
}
static int score_of(PyObject* o, int* out) {
    if (!PyUnicode_CheckExact(o)) return 0;
    const int softmax = PyUnicode_CompareWithASCIIString(o, "softmax") == 0;
    *out = softmax ? BSFP8_SOFTMAX : BSFP8_SIGMOID;
    return softmax || PyUnicode_CompareWithASCIIString(o, "sigmoid") == 0;
}
static int scale_of(PyObject* o, float* out) {
    if (!PyFloat_CheckExact(o) && !PyLong_CheckExact(o)) return 0;
    *out = (float)PyFloat_AsDouble(o);
    return isfinite(*out) && !PyErr_Occurred();
}

/* The current stream where the current device is the tensors'. */
static int stream_of(long device, void** stream) {
    PyObject* o = PyObject_CallNoArgs(get_device);
    const long current = o != NULL ? PyLong_AsLong(o) : -1;
    if (current == device) {
        PyObject* s = PyObject_CallOneArg(get_stream, o);
        *stream = s != NULL ? PyLong_AsVoidPtr(s) : NULL;
        Py_XDECREF(s);
    }
    Py_XDECREF(o);
    return current == device && !PyErr_Occurred();
}

/* ---- ends of a call */
static void drop(View* v, int n) {
    for (int i = 0; i < n; ++i)
        if (v[i].made) Py_CLEAR(v[i].t);
}
static PyObject* unusual(View* v, int n) {
    drop(v, n);
    PyErr_Clear();
    Py_RETURN_NONE;
}
static PyObject* failed(View* v, int n, const char* name, int status) {
    drop(v, n);
    PyObject* e = PyObject_CallFunction(error_type, "si", name, status);
    if (e != NULL) {
        PyErr_SetObject(error_type, e);
        Py_DECREF(e);
    }
    return NULL;
}
static PyObject* out(View* v) { /* a reference for the caller */
    if (!v->made) Py_INCREF(v->t);
    v->made = 0;
    return v->t;
}
#define LAUNCH(status, expression)          \
    do {                                    \
        Py_BEGIN_ALLOW_THREADS;             \
        status = (expression);              \
        Py_END_ALLOW_THREADS;               \
    } while (0)

static int choices(PyObject* t, View* v) { /* [T, k] int32 */
    return look(t, v) && v->dims == 2 && v->n[0] > 0 && v->n[1] >= 1 && v->n[1] <= 64 && dense2(v, I32, v->n[0], v->n[1]) &&
           v->n[0] < ((int64_t)1 << 31) / v->n[1];
}
static int logits_of(PyObject* t, View* v) {
    return look(t, v) && (v->type == F32 || v->type == BF16) && rows_at_stride(v) && v->n[1] <= 1024;
}
static int logits_type(const View* v) { return v->type == F32 ? BSFP8_F32 : BSFP8_BF16; }

/* logits, k, score, bias, groups, top_groups, renormalize, scale, weights, ids */
static PyObject* route(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[4] = {{0}};
    View *z = v, *b = v + 1, *w = v + 2, *ids = v + 3;
    int64_t k, groups, top;
    int score, renormalize, status;
    float scale;
    void* stream;
    if (n != 10 || !logits_of(a[0], z) || !number(a[1], &k) || !score_of(a[2], &score) || !number(a[4], &groups) ||
        !number(a[5], &top) || !flag(a[6], &renormalize) || !scale_of(a[7], &scale))
        return unusual(v, 4);
    const int64_t T = z->n[0], E = z->n[1];
    if (k < 1 || k > E || k > 64 || groups < 1 || E % groups != 0 || top < 1 || top > groups || k > top * (E / groups) ||
        T >= ((int64_t)1 << 31) / k)
        return unusual(v, 4);
    if (a[3] != Py_None && (!look(a[3], b) || !dense1(b, F32, E) || b->device != z->device)) return unusual(v, 4);
    if (a[8] != Py_None ? !look(a[8], w) || !dense2(w, F32, T, k) : !make(z, w, F32, T, k)) return unusual(v, 4);
    if (a[9] != Py_None ? !look(a[9], ids) || !dense2(ids, I32, T, k) : !make(z, ids, I32, T, k)) return unusual(v, 4);
    if (w->device != z->device || ids->device != z->device || !stream_of(z->device, &stream)) return unusual(v, 4);
    LAUNCH(status, call_route(z->p, logits_type(z), T, E, stride(z), b->p, score, k, groups, top, renormalize, scale, w->p, ids->p, stream));
    if (status != 0) return failed(v, 4, "moe_route", status);
    return Py_BuildValue("(NN)", out(w), out(ids));
}

/* logits, ids, dweights, score, renormalize, scale, dlogits */
static PyObject* route_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[4] = {{0}};
    View *z = v, *ids = v + 1, *dw = v + 2, *dz = v + 3;
    int score, renormalize, status;
    float scale;
    void* stream;
    if (n != 7 || !logits_of(a[0], z) || !choices(a[1], ids) || !look(a[2], dw) || !score_of(a[3], &score) ||
        !flag(a[4], &renormalize) || !scale_of(a[5], &scale))
        return unusual(v, 4);
    const int64_t T = z->n[0], E = z->n[1], k = ids->n[1];
    if (ids->n[0] != T || k > E || !dense2(dw, F32, T, k)) return unusual(v, 4);
    if (a[6] != Py_None ? !matrix(a[6], dz, z->type, T, E) : !make(z, dz, z->type, T, E)) return unusual(v, 4);
    if (ids->device != z->device || dw->device != z->device || dz->device != z->device || !stream_of(z->device, &stream))
        return unusual(v, 4);
    LAUNCH(status, call_route_backward(z->p, logits_type(z), T, E, stride(z), score, k, renormalize, scale, ids->p, dw->p, dz->p,
                                       stride(dz), stream));
    if (status != 0) return failed(v, 4, "moe_route_backward", status);
    return out(dz);
}

/* ids, E, offsets, slots, rows, workspace */
static PyObject* plan(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[5] = {{0}};
    View *ids = v, *off = v + 1, *slots = v + 2, *rows = v + 3, *ws = v + 4;
    int64_t E;
    int status;
    void* stream;
    if (n != 6 || !choices(a[0], ids) || !number(a[1], &E) || E < 1 || E > 1024) return unusual(v, 5);
    const int64_t T = ids->n[0], k = ids->n[1], need = call_plan_workspace(T, k, E);
    if (need < 0) return unusual(v, 5);
    if (a[2] != Py_None ? !look(a[2], off) || !dense1(off, I64, E + 1) : !make(ids, off, I64, E + 1, -1)) return unusual(v, 5);
    if (a[3] != Py_None ? !look(a[3], slots) || !dense2(slots, I32, T, k) : !make(ids, slots, I32, T, k)) return unusual(v, 5);
    if (a[4] != Py_None ? !look(a[4], rows) || !dense1(rows, I32, T * k) : !make(ids, rows, I32, T * k, -1)) return unusual(v, 5);
    if (a[5] != Py_None ? !look(a[5], ws) || !dense1(ws, U8, ws->n[0]) || ws->n[0] < need
                        : need > 0 && !make(ids, ws, U8, need, -1))
        return unusual(v, 5);
    if (off->device != ids->device || slots->device != ids->device || rows->device != ids->device ||
        (ws->t != NULL && ws->device != ids->device) || !stream_of(ids->device, &stream))
        return unusual(v, 5);
    LAUNCH(status, call_plan(ids->p, T, k, E, off->p, slots->p, rows->p, ws->p, ws->t != NULL ? ws->n[0] : 0, stream));
    if (status != 0) return failed(v, 5, "moe_plan", status);
    PyObject* r = Py_BuildValue("(NNN)", out(off), out(slots), out(rows));
    drop(v, 5);
    return r;
}

/* x, slots, q, a_s, copy, want_copy */
static PyObject* dispatch(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[5] = {{0}};
    View *x = v, *slots = v + 1, *q = v + 2, *s = v + 3, *copy = v + 4;
    int want, status;
    void* stream;
    if (n != 6 || !look(a[0], x) || x->type != BF16 || !rows_at_stride(x) || !choices(a[1], slots) || !flag(a[5], &want))
        return unusual(v, 5);
    const int64_t T = x->n[0], H = x->n[1], k = slots->n[1], R = T * k;
    if (slots->n[0] != T) return unusual(v, 5);
    if (a[2] != Py_None ? !look(a[2], q) || (q->type != U8 && q->type != FP8) || !rows_at_stride(q) || q->n[0] != R || q->n[1] != H
                        : !make(x, q, U8, R, H))
        return unusual(v, 5);
    if (a[3] != Py_None ? !look(a[3], s) || !dense2(s, F32, (H + 127) / 128, R) : !make(x, s, F32, (H + 127) / 128, R))
        return unusual(v, 5);
    if (a[4] != Py_None ? !matrix(a[4], copy, BF16, R, H) : want && !make(x, copy, BF16, R, H)) return unusual(v, 5);
    if (slots->device != x->device || q->device != x->device || s->device != x->device ||
        (copy->t != NULL && copy->device != x->device) || !stream_of(x->device, &stream))
        return unusual(v, 5);
    LAUNCH(status, call_dispatch(x->p, T, H, stride(x), slots->p, k, q->p, stride(q), s->p, copy->p, copy->t != NULL ? stride(copy) : 0, stream));
    if (status != 0) return failed(v, 5, "moe_dispatch", status);
    if (copy->t == NULL) return Py_BuildValue("(NNO)", out(q), out(s), Py_None);
    return Py_BuildValue("(NNN)", out(q), out(s), out(copy));
}

/* rows, slots, weights, y */
static PyObject* combine(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[4] = {{0}};
    View *rows = v, *slots = v + 1, *w = v + 2, *y = v + 3;
    int status;
    void* stream;
    if (n != 4 || !look(a[0], rows) || rows->type != BF16 || !rows_at_stride(rows) || !choices(a[1], slots)) return unusual(v, 4);
    const int64_t T = slots->n[0], k = slots->n[1], H = rows->n[1];
    if (a[2] != Py_None && (!look(a[2], w) || !dense2(w, F32, T, k) || w->device != rows->device)) return unusual(v, 4);
    if (a[3] != Py_None ? !matrix(a[3], y, BF16, T, H) : !make(rows, y, BF16, T, H)) return unusual(v, 4);
    if (slots->device != rows->device || y->device != rows->device || !stream_of(rows->device, &stream)) return unusual(v, 4);
    LAUNCH(status, call_combine(rows->p, rows->n[0], stride(rows), slots->p, w->p, T, k, H, y->p, stride(y), stream));
    if (status != 0) return failed(v, 4, "moe_combine", status);
    return out(y);
}

/* dy, rows, slots, weights, drows, dweights */
static PyObject* combine_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[6] = {{0}};
    View *dy = v, *rows = v + 1, *slots = v + 2, *w = v + 3, *dr = v + 4, *dw = v + 5;
    int status;
    void* stream;
    if (n != 6 || !choices(a[2], slots) || !look(a[0], dy) || dy->type != BF16 || !rows_at_stride(dy)) return unusual(v, 6);
    const int64_t T = slots->n[0], k = slots->n[1], H = dy->n[1], R = T * k;
    if (dy->n[0] != T || !matrix(a[1], rows, BF16, R, H) || !look(a[3], w) || !dense2(w, F32, T, k)) return unusual(v, 6);
    if (a[4] != Py_None ? !matrix(a[4], dr, BF16, R, H) : !make(dy, dr, BF16, R, H)) return unusual(v, 6);
    if (a[5] != Py_None ? !look(a[5], dw) || !dense2(dw, F32, T, k) : !make(dy, dw, F32, T, k)) return unusual(v, 6);
    for (int i = 1; i < 6; ++i)
        if (v[i].device != dy->device) return unusual(v, 6);
    if (!stream_of(dy->device, &stream)) return unusual(v, 6);
    LAUNCH(status, call_combine_backward(dy->p, stride(dy), rows->p, stride(rows), slots->p, w->p, T, k, H, dr->p, stride(dr), dw->p, stream));
    if (status != 0) return failed(v, 6, "moe_combine_backward", status);
    return Py_BuildValue("(NN)", out(dr), out(dw));
}

/* a, a_s, b, b_s, offsets, E, b_stride, bs_stride, bs_stride_nb, bs_stride_kb, ldb, rows, k, swiglu, c, N */
static PyObject* product(PyObject* self, PyObject* const* o, Py_ssize_t n) {
    View v[7] = {{0}};
    View *a = v, *a_s = v + 1, *b = v + 2, *b_s = v + 3, *off = v + 4, *rows = v + 5, *c = v + 6;
    int64_t E, bst, bss, nb, kb, ldb, k, N;
    int swiglu, status;
    void* stream;
    if (n != 16 || !look(o[0], a) || !look(o[1], a_s) || !look(o[2], b) || !look(o[3], b_s) || !look(o[4], off) || !number(o[5], &E) ||
        !number(o[6], &bst) || !number(o[7], &bss) || !number(o[8], &nb) || !number(o[9], &kb) || !number(o[12], &k) || !flag(o[13], &swiglu))
        return unusual(v, 7);
    if ((a->type != U8 && a->type != FP8) || !rows_at_stride(a) || (b->type != U8 && b->type != FP8) || !rows_at_stride(b)) return unusual(v, 7);
    const int64_t A = a->n[0], K = a->n[1], halves = swiglu ? 2 : 1;
    if (E < 1 || E > 1024 || k < 1 || k > 64 || K % 128 != 0 || bst < 0 || bss < 0 || nb < 0 || kb < 0) return unusual(v, 7);
    if (o[10] == Py_None) ldb = b->n[0] > 1 ? b->s[0] : K;
    else if (!number(o[10], &ldb) || ldb < 0) return unusual(v, 7);
    if (o[15] == Py_None) N = b->n[0] / E / halves;
    else if (!number(o[15], &N)) return unusual(v, 7);
    if (N < 1 || N >= (int64_t)1 << 31 || (swiglu && N % 128 != 0)) return unusual(v, 7);
    if (o[11] != Py_None && (!look(o[11], rows) || !dense1(rows, I32, rows->n[0]) || rows->n[0] < 1 || rows->device != a->device))
        return unusual(v, 7);
    const int64_t M = rows->t != NULL ? rows->n[0] : A;
    if (!dense2(a_s, F32, K / 128, A) || off->type != I64 || off->dims != 1 || off->n[0] < E + 1 || off->s[0] != 1) return unusual(v, 7);
    /* what the strides reach lies in b's own rows and in b_s */
    int64_t floats = 1;
    for (int i = b_s->dims - 1; i >= 0; --i) {
        if (b_s->n[i] != 1 && b_s->s[i] != floats) return unusual(v, 7);
        floats *= b_s->n[i];
    }
    const __int128 codes = (__int128)(E - 1) * bst + (__int128)(halves * N - 1) * ldb + K;
    const __int128 scales = (__int128)(E - 1) * bss + (__int128)((halves * N + 127) / 128 - 1) * nb + (__int128)(K / 128 - 1) * kb + 1;
    if (b_s->type != F32 || scales > floats || codes > (__int128)(b->n[0] - 1) * b->s[0] + b->n[1]) return unusual(v, 7);
    if (o[14] != Py_None ? !matrix(o[14], c, BF16, M, N) : !make(a, c, BF16, M, N)) return unusual(v, 7);
    if (a_s->device != a->device || b->device != a->device || b_s->device != a->device || off->device != a->device ||
        c->device != a->device || !stream_of(a->device, &stream))
        return unusual(v, 7);
    LAUNCH(status, call_product(a->p, stride(a), a_s->p, A, rows->p, k, b->p, ldb, bst, b_s->p, bss, nb, kb, off->p, E, c->p, stride(c), M,
                                N, K, swiglu, stream));
    if (status != 0) return failed(v, 7, "gemm_1x128_128x128_routed", status);
    return out(c);
}

/* tensor type, error type, function of the current device, of its current stream, the types in the order
 * above, the addresses of the library's functions in the order above */
static PyObject* bind(PyObject* self, PyObject* args) {
    PyObject *t, *e, *d, *s, *ty[TYPES];
    unsigned long long f[8];
    if (!PyArg_ParseTuple(args, "OOOO(OOOOOO)(KKKKKKKK)", &t, &e, &d, &s, &ty[0], &ty[1], &ty[2], &ty[3], &ty[4], &ty[5], &f[0], &f[1],
                          &f[2], &f[3], &f[4], &f[5], &f[6], &f[7]))
        return NULL;
    Py_INCREF(t), Py_INCREF(e), Py_INCREF(d), Py_INCREF(s);
    tensor_type = t, error_type = e, get_device = d, get_stream = s;
    for (int i = 0; i < TYPES; ++i) {
        Py_INCREF(ty[i]);
        types[i] = ty[i];
    }
    call_route = (__typeof__(call_route))(uintptr_t)f[0];
    call_route_backward = (__typeof__(call_route_backward))(uintptr_t)f[1];
    call_plan_workspace = (__typeof__(call_plan_workspace))(uintptr_t)f[2];
    call_plan = (__typeof__(call_plan))(uintptr_t)f[3];
    call_dispatch = (__typeof__(call_dispatch))(uintptr_t)f[4];
    call_combine = (__typeof__(call_combine))(uintptr_t)f[5];
    call_combine_backward = (__typeof__(call_combine_backward))(uintptr_t)f[6];
    call_product = (__typeof__(call_product))(uintptr_t)f[7];
    Py_RETURN_NONE;
}

#define FAST(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, NULL},
    FAST("moe_route", route),
    FAST("moe_route_backward", route_backward),
    FAST("moe_plan", plan),
    FAST("moe_dispatch", dispatch),
    FAST("moe_combine", combine),
    FAST("moe_combine_backward", combine_backward),
    FAST("gemm_1x128_128x128_routed", product),
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) {
    PyObject* only = NULL;
    if ((n_dtype = PyUnicode_InternFromString("dtype")) == NULL || (n_shape = PyUnicode_InternFromString("shape")) == NULL ||
        (n_stride = PyUnicode_InternFromString("stride")) == NULL || (n_get_device = PyUnicode_InternFromString("get_device")) == NULL ||
        (n_data_ptr = PyUnicode_InternFromString("data_ptr")) == NULL || (n_new_empty = PyUnicode_InternFromString("new_empty")) == NULL ||
        (only = PyTuple_Pack(1, n_dtype)) == NULL)
        return NULL;
    n_dtype_only = only;
    return PyModule_Create(&module);
}
