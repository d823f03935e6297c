/* The usual call of an operator whose kernels take a few microseconds (those of a mixture-of-experts layer, those
 * between the 8-bit products, the int8 product, the gradient norm) in one step, for CPython: plain torch tensors on the
 * current GPU, the current stream, every argument as binding.py's functions want it. A function here
 * looks at its arguments, makes the outputs that are not given, calls the library and returns what
 * binding.py's function of that name returns; where anything is not as usual it returns None and has
 * done nothing, and binding.py goes the long way, whose checks say what is wrong (so too where this part
 * was not built). What is accepted here is a part of what is accepted there. A tensor is read through its Python attributes, so nothing
 * depends on torch's binary interface.
 *
 * Why: for few tokens these operators' kernels take 3 to 9 us and the launch 3.3. A call here takes 4.6
 * us (route, outputs given), 4.7 (combine), 5.1 (dispatch) and 5.3 (product); through binding.py's
 * checks and ctypes 6.8, 6.9, 7.4 and 9.1. The norm of one token takes 5.4 to 6.2 us a call (9.8 the other
 * way), the gated activation of 64 rows 5.3 (7.5), int8 rows and product of 1000 rows 10.2 together (14.2),
 * clipping a layer's four gradients 12.3 (20.9). */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>
#include <stdint.h>

#include "blockwise_fp8.h"

/* ---- what bind() is given */
static PyObject *tensor_type, *error_type, *get_stream, *get_device;
enum { F32, BF16, I32, I64, U8, FP8, I8, TYPES };
static PyObject* types[TYPES];
static __typeof__(&moe_route) call_route;
static __typeof__(&moe_route_backward) call_route_backward;
static __typeof__(&moe_plan_workspace) call_plan_workspace;
static __typeof__(&moe_plan) call_plan;
static __typeof__(&moe_dispatch) call_dispatch;
static __typeof__(&moe_combine) call_combine;
static __typeof__(&moe_combine_backward) call_combine_backward;
static __typeof__(&gemm_1x128_128x128_routed) call_product;
static __typeof__(&rms_norm_quantize) call_norm;
static __typeof__(&rms_norm_quantize_rhs) call_norm_rhs;
static __typeof__(&rms_norm_backward_workspace) call_norm_workspace;
static __typeof__(&rms_norm_backward) call_norm_backward;
static __typeof__(&swiglu_quantize) call_swiglu;
static __typeof__(&swiglu_quantize_lhs_and_rhs) call_swiglu_dual;
static __typeof__(&swiglu_backward) call_swiglu_backward;
static __typeof__(&swiglu_backward_quantize) call_swiglu_backward_dual;
static __typeof__(&quantize_rows_i8) call_rows_i8;
static __typeof__(&gemm_i8) call_gemm_i8;
static __typeof__(&grad_workspace) call_grad_workspace;
static __typeof__(&grad_norm) call_grad_norm;
static __typeof__(&clip_grads) call_clip;

static PyObject *n_dtype, *n_shape, *n_stride, *n_get_device, *n_data_ptr, *n_new_empty, *n_dtype_only, *n_numel, *n_is_contiguous;

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

/* ---- between the 8-bit products */
static int codes_of(PyObject* o, int* out) {
    if (o == Py_None) {
        *out = BSFP8_CODES_NONE;
        return 1;
    }
    if (!PyUnicode_CheckExact(o)) return 0;
    if (PyUnicode_CompareWithASCIIString(o, "e4m3fn") == 0) *out = BSFP8_CODES_E4M3FN;
    else if (PyUnicode_CompareWithASCIIString(o, "int8") == 0) *out = BSFP8_CODES_INT8;
    else if (PyUnicode_CompareWithASCIIString(o, "e4m3fnuz") == 0) *out = BSFP8_CODES_E4M3FNUZ;
    else return 0;
    return 1;
}
static int fp8_codes_of(PyObject* o, int* out) {
    return codes_of(o, out) && (*out == BSFP8_CODES_E4M3FN || *out == BSFP8_CODES_E4M3FNUZ);
}
static int code_type(int type, int codes) {
    return codes == BSFP8_CODES_INT8 ? type == I8 : type == U8 || (codes == BSFP8_CODES_E4M3FN && type == FP8);
}
static int codes_matrix(PyObject* t, const View* like, View* v, int codes, int64_t a, int64_t b) {
    if (t == Py_None) return make(like, v, codes == BSFP8_CODES_INT8 ? I8 : U8, a, b);
    return look(t, v) && code_type(v->type, codes) && rows_at_stride(v) && v->n[0] == a && v->n[1] == b;
}
static int scales(PyObject* t, const View* like, View* v, int64_t a, int64_t b) { /* fp32 [a, b], b < 0: [a] */
    if (t == Py_None) return make(like, v, F32, a, b);
    return look(t, v) && (b < 0 ? dense1(v, F32, a) : dense2(v, F32, a, b));
}
static int bf16_rows(PyObject* t, View* v) { return look(t, v) && v->type == BF16 && rows_at_stride(v); }
static int bf16_or_f32(const View* v) { return v->type == BF16 || v->type == F32; }
static int dtype_of(const View* v) { return v->type == F32 ? BSFP8_F32 : BSFP8_BF16; }
static int weight_of(PyObject* t, View* v, int64_t H) { return look(t, v) && bf16_or_f32(v) && dense1(v, v->type, H); }
static int one_device(const View* v, int n) { /* of the tensors that are there */
    for (int i = 1; i < n; ++i)
        if (v[i].t != NULL && v[i].device != v[0].device) return 0;
    return 1;
}
static PyObject* out_or_none(View* v) {
    if (v->t == NULL) Py_RETURN_NONE;
    return out(v);
}
static int64_t stride_or_0(const View* v) { return v->t != NULL ? stride(v) : 0; }

/* q, s, y of rows [T, H] */
static int row_outputs(const View* like, int64_t T, int64_t H, int codes, PyObject* oq, PyObject* os, PyObject* oy, int want_y, View* q, View* s,
                       View* y) {
    if (T > ((int64_t)1 << 24) - 16) return 0;
    if (codes == BSFP8_CODES_NONE) {
        if (oq != Py_None || os != Py_None) return 0;
        want_y = 1;
    } else {
        const int i8 = codes == BSFP8_CODES_INT8;
        if (!codes_matrix(oq, like, q, codes, T, H) || !scales(os, like, s, i8 ? T : (H + 127) / 128, i8 ? -1 : T)) return 0;
    }
    return oy != Py_None ? matrix(oy, y, BF16, T, H) : !want_y || make(like, y, BF16, T, H);
}

/* x, weight, residual, eps, fmt, q, s, h, y, rstd, want_y, want_rstd */
static PyObject* norm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[8] = {{0}};
    View *x = v, *w = v + 1, *r = v + 2, *h = v + 3, *q = v + 4, *s = v + 5, *y = v + 6, *rstd = v + 7;
    int codes, want_y, want_rstd, status;
    void* stream;
    if (n != 12 || !bf16_rows(a[0], x) || !PyFloat_CheckExact(a[3]) || !codes_of(a[4], &codes) || !flag(a[10], &want_y) || !flag(a[11], &want_rstd))
        return unusual(v, 8);
    const float eps = (float)PyFloat_AS_DOUBLE(a[3]);
    const int64_t T = x->n[0], H = x->n[1];
    if (!(eps > 0) || !isfinite(eps) || !weight_of(a[1], w, H)) return unusual(v, 8);
    if (a[2] != Py_None) {
        if (!look(a[2], r) || !bf16_or_f32(r) || !rows_at_stride(r) || r->n[0] != T || r->n[1] != H) return unusual(v, 8);
        if (a[7] != Py_None ? !matrix(a[7], h, r->type, T, H) : !make(r, h, r->type, T, H)) return unusual(v, 8);
    } else if (a[7] != Py_None) {
        return unusual(v, 8);
    }
    if (!row_outputs(x, T, H, codes, a[5], a[6], a[8], want_y, q, s, y)) return unusual(v, 8);
    if (a[9] != Py_None ? !look(a[9], rstd) || !dense1(rstd, F32, T) : want_rstd && !make(x, rstd, F32, T, -1)) return unusual(v, 8);
    if (!one_device(v, 8) || !stream_of(x->device, &stream)) return unusual(v, 8);
    LAUNCH(status, call_norm(x->p, T, H, stride(x), r->p, r->t != NULL ? dtype_of(r) : BSFP8_BF16, stride_or_0(r), w->p, dtype_of(w), eps, h->p,
                             stride_or_0(h), rstd->p, codes, q->p, stride_or_0(q), s->p, y->p, stride_or_0(y), stream));
    if (status != 0) return failed(v, 8, "rms_norm_quantize", status);
    return Py_BuildValue("(NNNNN)", out_or_none(q), out_or_none(s), out_or_none(h), out_or_none(y), out_or_none(rstd));
}

/* h, weight, rstd, qT, s, fmt */
static PyObject* norm_rhs(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[5] = {{0}};
    View *h = v, *w = v + 1, *rstd = v + 2, *q = v + 3, *s = v + 4;
    int codes, status;
    void* stream;
    if (n != 6 || !look(a[0], h) || !bf16_or_f32(h) || !rows_at_stride(h) || !fp8_codes_of(a[5], &codes)) return unusual(v, 5);
    const int64_t T = h->n[0], H = h->n[1];
    if (!weight_of(a[1], w, H) || !look(a[2], rstd) || !dense1(rstd, F32, T) || !codes_matrix(a[3], h, q, codes, H, T) ||
        !scales(a[4], h, s, (T + 127) / 128, H) || !one_device(v, 5) || !stream_of(h->device, &stream))
        return unusual(v, 5);
    LAUNCH(status, call_norm_rhs(h->p, dtype_of(h), T, H, stride(h), w->p, dtype_of(w), rstd->p, codes, q->p, stride(q), s->p, stream));
    if (status != 0) return failed(v, 5, "rms_norm_quantize_rhs", status);
    return Py_BuildValue("(NN)", out(q), out(s));
}

/* dy, h, weight, rstd, dh, dx, dweight, workspace */
static PyObject* norm_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[8] = {{0}};
    View *dy = v, *h = v + 1, *w = v + 2, *rstd = v + 3, *dh = v + 4, *dx = v + 5, *dw = v + 6, *ws = v + 7;
    int status;
    void* stream;
    if (n != 8 || !bf16_rows(a[0], dy) || !look(a[1], h) || !bf16_or_f32(h) || !rows_at_stride(h)) return unusual(v, 8);
    const int64_t T = dy->n[0], H = dy->n[1], need = call_norm_workspace(T, H);
    if (need < 0 || h->n[0] != T || h->n[1] != H || !weight_of(a[2], w, H) || !look(a[3], rstd) || !dense1(rstd, F32, T)) return unusual(v, 8);
    if (a[4] != Py_None && !matrix(a[4], dh, h->type, T, H)) return unusual(v, 8);
    if (a[5] != Py_None ? !matrix(a[5], dx, h->type, T, H) : !make(h, dx, h->type, T, H)) return unusual(v, 8);
    if (a[6] != Py_None ? !look(a[6], dw) || !dense1(dw, w->type, H) : !make(w, dw, w->type, H, -1)) return unusual(v, 8);
    if (a[7] != Py_None ? !look(a[7], ws) || !dense1(ws, U8, ws->n[0]) || ws->n[0] < need || ((uintptr_t)ws->p & 15) != 0
                        : !make(dy, ws, U8, need, -1))
        return unusual(v, 8);
    if (!one_device(v, 8) || !stream_of(dy->device, &stream)) return unusual(v, 8);
    LAUNCH(status, call_norm_backward(dy->p, stride(dy), h->p, dtype_of(h), stride(h), w->p, dtype_of(w), rstd->p, dh->p, stride_or_0(dh), T, H, dx->p,
                                      stride(dx), dw->p, ws->p, ws->n[0], stream));
    if (status != 0) return failed(v, 8, "rms_norm_backward", status);
    PyObject* r = Py_BuildValue("(NN)", out(dx), out(dw));
    drop(v, 8);
    return r;
}

/* gu, fmt, q, s, y, want_y */
static PyObject* swiglu(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[4] = {{0}};
    View *gu = v, *q = v + 1, *s = v + 2, *y = v + 3;
    int codes, want_y, status;
    void* stream;
    if (n != 6 || !bf16_rows(a[0], gu) || gu->n[1] % 2 != 0 || !codes_of(a[1], &codes) || !flag(a[5], &want_y)) return unusual(v, 4);
    const int64_t T = gu->n[0], F = gu->n[1] / 2;
    if (!row_outputs(gu, T, F, codes, a[2], a[3], a[4], want_y, q, s, y) || !one_device(v, 4) || !stream_of(gu->device, &stream))
        return unusual(v, 4);
    LAUNCH(status, call_swiglu(gu->p, T, F, stride(gu), codes, q->p, stride_or_0(q), s->p, y->p, stride_or_0(y), stream));
    if (status != 0) return failed(v, 4, "swiglu_quantize", status);
    return Py_BuildValue("(NNN)", out_or_none(q), out_or_none(s), out_or_none(y));
}

/* q, a_s, qT, s of [T, C] in v[0..3] */
static int tile_outputs(PyObject* const* a, const View* like, int64_t T, int64_t C, int codes, View* v) {
    return codes_matrix(a[0], like, v, codes, T, C) && scales(a[1], like, v + 1, (C + 127) / 128, T) &&
           codes_matrix(a[2], like, v + 2, codes, C, T) && scales(a[3], like, v + 3, (T + 127) / 128, C);
}

/* gu, q, a_s, qT, s, fmt */
static PyObject* swiglu_dual(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[5] = {{0}};
    View* gu = v;
    int codes, status;
    void* stream;
    if (n != 6 || !bf16_rows(a[0], gu) || gu->n[1] % 2 != 0 || !fp8_codes_of(a[5], &codes)) return unusual(v, 5);
    const int64_t T = gu->n[0], F = gu->n[1] / 2;
    if (!tile_outputs(a + 1, gu, T, F, codes, v + 1) || !one_device(v, 5) || !stream_of(gu->device, &stream)) return unusual(v, 5);
    LAUNCH(status, call_swiglu_dual(gu->p, T, F, stride(gu), codes, v[1].p, stride(v + 1), v[2].p, v[3].p, stride(v + 3), v[4].p, stream));
    if (status != 0) return failed(v, 5, "swiglu_quantize_lhs_and_rhs", status);
    return Py_BuildValue("(NNNN)", out(v + 1), out(v + 2), out(v + 3), out(v + 4));
}

/* dy, gu, dgu */
static PyObject* swiglu_back(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[3] = {{0}};
    View *gu = v, *dy = v + 1, *d = v + 2;
    int status;
    void* stream;
    if (n != 3 || !bf16_rows(a[1], gu) || gu->n[1] % 2 != 0) return unusual(v, 3);
    const int64_t T = gu->n[0], F = gu->n[1] / 2;
    if (!matrix(a[0], dy, BF16, T, F) || (a[2] != Py_None ? !matrix(a[2], d, BF16, T, 2 * F) : !make(gu, d, BF16, T, 2 * F)) ||
        !one_device(v, 3) || !stream_of(gu->device, &stream))
        return unusual(v, 3);
    LAUNCH(status, call_swiglu_backward(dy->p, stride(dy), gu->p, stride(gu), T, F, d->p, stride(d), stream));
    if (status != 0) return failed(v, 3, "swiglu_backward", status);
    return out(d);
}

/* dy, gu, q, a_s, qT, s, fmt */
static PyObject* swiglu_back_dual(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[6] = {{0}};
    View *gu = v, *dy = v + 1;
    int codes, status;
    void* stream;
    if (n != 7 || !bf16_rows(a[1], gu) || gu->n[1] % 2 != 0 || !fp8_codes_of(a[6], &codes)) return unusual(v, 6);
    const int64_t T = gu->n[0], F = gu->n[1] / 2;
    if (!matrix(a[0], dy, BF16, T, F) || !tile_outputs(a + 2, gu, T, 2 * F, codes, v + 2) || !one_device(v, 6) || !stream_of(gu->device, &stream))
        return unusual(v, 6);
    LAUNCH(status, call_swiglu_backward_dual(dy->p, stride(dy), gu->p, stride(gu), T, F, codes, v[2].p, stride(v + 2), v[3].p, v[4].p, stride(v + 4),
                                             v[5].p, stream));
    if (status != 0) return failed(v, 6, "swiglu_backward_quantize", status);
    return Py_BuildValue("(NNNN)", out(v + 2), out(v + 3), out(v + 4), out(v + 5));
}

/* x, q, s */
static PyObject* rows_i8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    View v[4] = {{0}};
    View *x = v, *q = v + 1, *s = v + 2;
    int status;
    void* stream;
    if (n != 3 || !bf16_rows(a[0], x) || !row_outputs(x, x->n[0], x->n[1], BSFP8_CODES_INT8, a[1], a[2], Py_None, 0, q, s, v + 3) ||
        !one_device(v, 3) || !stream_of(x->device, &stream))
        return unusual(v, 4);
    LAUNCH(status, call_rows_i8(x->p, x->n[0], x->n[1], stride(x), q->p, stride(q), s->p, stream));
    if (status != 0) return failed(v, 4, "quantize_rows_i8", status);
    return Py_BuildValue("(NN)", out(q), out(s));
}

static int64_t i8_stride(const View* v) { return v->n[0] > 1 ? v->s[0] : (v->n[1] + 15) / 16 * 16; }

/* a, a_s, b, b_s, c, K */
static PyObject* i8_product(PyObject* self, PyObject* const* o, Py_ssize_t n) {
    View v[5] = {{0}};
    View *a = v, *a_s = v + 1, *b = v + 2, *b_s = v + 3, *c = v + 4;
    int64_t K;
    int status;
    void* stream;
    if (n != 6 || !look(o[0], a) || a->type != I8 || !rows_at_stride(a) || !look(o[2], b) || b->type != I8 || !rows_at_stride(b)) return unusual(v, 5);
    const int64_t M = a->n[0], N = b->n[0];
    if (o[5] == Py_None) K = a->n[1];
    else if (!number(o[5], &K)) return unusual(v, 5);
    if (K < 0 || K > a->n[1] || K > b->n[1] || K > 131071 || !look(o[1], a_s) || !dense1(a_s, F32, M) || !look(o[3], b_s) || !dense1(b_s, F32, N))
        return unusual(v, 5);
    if (o[4] != Py_None ? !matrix(o[4], c, BF16, M, N) : !make(a, c, BF16, M, N)) return unusual(v, 5);
    if (!one_device(v, 5) || !stream_of(a->device, &stream)) return unusual(v, 5);
    LAUNCH(status, call_gemm_i8(a->p, i8_stride(a), a_s->p, b->p, i8_stride(b), b_s->p, c->p, stride(c), M, N, K, stream));
    if (status != 0) return failed(v, 5, "gemm_i8", status);
    return out(c);
}

/* ---- gradients of many tensors */
static int64_t whole(PyObject* t, PyObject* method) { /* a method's number, -1 with an error */
    PyObject* o = PyObject_CallMethodNoArgs(t, method);
    const int64_t r = o != NULL ? PyLong_AsLongLong(o) : -1;
    Py_XDECREF(o);
    return r;
}

typedef struct {
    void** p;
    int64_t* n;
    int* type;
} Many;

/* The tensors of a list, contiguous, on one device (< 0: the first one's, which is set). */
static int look_at_all(PyObject** t, Py_ssize_t count, Many m, long* device) {
    for (Py_ssize_t i = 0; i < count; ++i) {
        if ((PyObject*)Py_TYPE(t[i]) != tensor_type) return 0;
        PyObject* o = PyObject_GetAttr(t[i], n_dtype);
        m.type[i] = o == types[F32] ? BSFP8_F32 : o == types[BF16] ? BSFP8_BF16 : -1;
        Py_XDECREF(o);
        if (m.type[i] < 0) return 0;
        o = PyObject_CallMethodNoArgs(t[i], n_is_contiguous);
        const int dense = o == Py_True;
        Py_XDECREF(o);
        if (!dense) return 0;
        const long at = (long)whole(t[i], n_get_device);
        if (at < 0 || (*device >= 0 && at != *device)) return 0;
        *device = at;
        m.n[i] = whole(t[i], n_numel);
        o = PyObject_CallMethodNoArgs(t[i], n_data_ptr);
        m.p[i] = o != NULL ? PyLong_AsVoidPtr(o) : NULL;
        Py_XDECREF(o);
        if (m.n[i] < 0 || PyErr_Occurred()) return 0;
    }
    return 1;
}

static int same_shapes(PyObject** a, PyObject** b, Py_ssize_t count) {
    int same = 1;
    for (Py_ssize_t i = 0; same && i < count; ++i) {
        PyObject *x = PyObject_GetAttr(a[i], n_shape), *y = PyObject_GetAttr(b[i], n_shape);
        same = x != NULL && y != NULL && PyObject_RichCompareBool(x, y, Py_EQ) == 1;
        Py_XDECREF(x);
        Py_XDECREF(y);
    }
    return same;
}

/* grads, out (a list, or None: in place), norm, workspace; the launch with max_norm and eps where clip is set */
static PyObject* gradients(PyObject* grads, PyObject* outs, PyObject* o_norm, PyObject* o_ws, int clip, float max_norm, float eps) {
    View v[2] = {{0}};
    View *norm = v, *ws = v + 1;
    if (!PyList_CheckExact(grads) || (outs != Py_None && !PyList_CheckExact(outs))) Py_RETURN_NONE;
    const Py_ssize_t count = PyList_GET_SIZE(grads);
    if (count == 0 || count > 0xFFFFFF || (outs != Py_None && PyList_GET_SIZE(outs) != count)) Py_RETURN_NONE;
    /* the tensors are held while Python code may run */
    const size_t each = 2 * (sizeof(PyObject*) + sizeof(void*) + sizeof(int64_t) + sizeof(int));
    char* memory = PyMem_Malloc(each * (size_t)count);
    if (memory == NULL) return PyErr_NoMemory();
    PyObject **g = (PyObject**)memory, **o = g + count;
    void** p = (void**)(o + count);
    int64_t* n = (int64_t*)(p + 2 * count);
    int* type = (int*)(n + 2 * count);
    const Many mg = {p, n, type}, mo = {p + count, n + count, type + count};
    const int apart = outs != Py_None;
    for (Py_ssize_t i = 0; i < count; ++i) {
        g[i] = PyList_GET_ITEM(grads, i);
        Py_INCREF(g[i]);
        if (apart) {
            o[i] = PyList_GET_ITEM(outs, i);
            Py_INCREF(o[i]);
        }
    }
    PyObject* result = NULL;
    int usual = 0, status = 0;
    long device = -1;
    void* stream;
    View first = {0};
    if (look_at_all(g, count, mg, &device) && (!apart || (look_at_all(o, count, mo, &device) && same_shapes(g, o, count)))) {
        const int64_t need = call_grad_workspace(mg.n, count);
        first.t = g[0], first.type = TYPES, first.device = device;
        usual = need > 0 && (o_norm != Py_None ? look(o_norm, norm) && dense1(norm, F32, 1) : make(&first, norm, F32, 1, -1)) &&
                (o_ws != Py_None ? look(o_ws, ws) && dense1(ws, U8, ws->n[0]) && ws->n[0] >= need && ((uintptr_t)ws->p & 7) == 0
                                 : make(&first, ws, U8, need, -1)) &&
                norm->device == device && ws->device == device && stream_of(device, &stream);
    }
    if (usual) {
        if (clip)
            LAUNCH(status, call_clip((const void* const*)mg.p, apart ? mo.p : mg.p, mg.n, mg.type, apart ? mo.type : mg.type, count, max_norm, eps,
                                     norm->p, ws->p, ws->n[0], stream));
        else
            LAUNCH(status, call_grad_norm((const void* const*)mg.p, mg.n, mg.type, count, norm->p, ws->p, ws->n[0], stream));
        result = status != 0 ? failed(v, 2, clip ? "clip_grads" : "grad_norm", status) : out(norm);
        drop(v, 2);
    } else {
        result = unusual(v, 2);
    }
    for (Py_ssize_t i = 0; i < count; ++i) {
        Py_DECREF(g[i]);
        if (apart) Py_DECREF(o[i]);
    }
    PyMem_Free(memory);
    return result;
}

/* grads, norm, workspace */
static PyObject* norm_of_many(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    if (n != 3) Py_RETURN_NONE;
    return gradients(a[0], Py_None, a[1], a[2], 0, 0.0f, 0.0f);
}

/* grads, max_norm, out, norm, eps, workspace */
static PyObject* clip_many(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    if (n != 6 || !PyFloat_CheckExact(a[1]) || !PyFloat_CheckExact(a[4])) Py_RETURN_NONE;
    const double max_norm = PyFloat_AS_DOUBLE(a[1]), eps = PyFloat_AS_DOUBLE(a[4]);
    if (!(max_norm >= 0) || !(eps >= 0) || !isfinite((float)eps)) Py_RETURN_NONE;
    return gradients(a[0], a[2], a[3], a[5], 1, (float)max_norm, (float)eps);
}

/* tensor type, error type, function of the current device, of its current stream, the types in the order
 * above, the addresses of the library's functions in the order above */
static PyObject* bind(PyObject* self, PyObject* args) {
    void** const functions[] = {(void**)&call_route, (void**)&call_route_backward, (void**)&call_plan_workspace, (void**)&call_plan,
                                (void**)&call_dispatch, (void**)&call_combine, (void**)&call_combine_backward, (void**)&call_product,
                                (void**)&call_norm, (void**)&call_norm_rhs, (void**)&call_norm_workspace, (void**)&call_norm_backward,
                                (void**)&call_swiglu, (void**)&call_swiglu_dual, (void**)&call_swiglu_backward, (void**)&call_swiglu_backward_dual,
                                (void**)&call_rows_i8, (void**)&call_gemm_i8, (void**)&call_grad_workspace, (void**)&call_grad_norm,
                                (void**)&call_clip};
    const Py_ssize_t count = (Py_ssize_t)(sizeof(functions) / sizeof(functions[0]));
    PyObject *t, *e, *d, *s, *ty, *f;
    if (!PyArg_ParseTuple(args, "OOOOO!O!", &t, &e, &d, &s, &PyTuple_Type, &ty, &PyTuple_Type, &f)) return NULL;
    if (PyTuple_GET_SIZE(ty) != TYPES || PyTuple_GET_SIZE(f) != count) {
        PyErr_SetString(PyExc_ValueError, "another number of types or functions");
        return NULL;
    }
    for (Py_ssize_t i = 0; i < count; ++i) {
        *functions[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(f, i));
        if (PyErr_Occurred()) return NULL;
    }
    Py_INCREF(t), Py_INCREF(e), Py_INCREF(d), Py_INCREF(s);
    tensor_type = t, error_type = e, get_device = d, get_stream = s;
    for (int i = 0; i < TYPES; ++i) {
        types[i] = PyTuple_GET_ITEM(ty, i);
        Py_INCREF(types[i]);
    }
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
    FAST("rms_norm_quantize", norm),
    FAST("rms_norm_quantize_rhs", norm_rhs),
    FAST("rms_norm_backward", norm_backward),
    FAST("swiglu_quantize", swiglu),
    FAST("swiglu_quantize_lhs_and_rhs", swiglu_dual),
    FAST("swiglu_backward", swiglu_back),
    FAST("swiglu_backward_quantize", swiglu_back_dual),
    FAST("quantize_rows_i8", rows_i8),
    FAST("gemm_i8", i8_product),
    FAST("grad_norm", norm_of_many),
    FAST("clip_grads", clip_many),
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) {
    PyObject* only = NULL;
    if ((n_dtype = PyUnicode_InternFromString("dtype")) == NULL || (n_shape = PyUnicode_InternFromString("shape")) == NULL ||
        (n_stride = PyUnicode_InternFromString("stride")) == NULL || (n_get_device = PyUnicode_InternFromString("get_device")) == NULL ||
        (n_data_ptr = PyUnicode_InternFromString("data_ptr")) == NULL || (n_new_empty = PyUnicode_InternFromString("new_empty")) == NULL ||
        (n_numel = PyUnicode_InternFromString("numel")) == NULL || (n_is_contiguous = PyUnicode_InternFromString("is_contiguous")) == NULL ||
        (only = PyTuple_Pack(1, n_dtype)) == NULL)
        return NULL;
    n_dtype_only = only;
    return PyModule_Create(&module);
}
