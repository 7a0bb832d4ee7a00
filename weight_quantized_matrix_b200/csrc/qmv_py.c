/*
 * qmv_py.c -- CPython extension "_qmv_fast": the per-call entry points of
 * libqmv.so for Python callers, with arguments passed as plain Python ints
 * (device pointers, sizes, enum values, the cudaStream_t).  It only converts
 * arguments and forwards to the C ABI of include/qmv.h; the status code is
 * returned unchanged.  Exists because ctypes argument conversion costs more
 * host time per call than a decode-size qmv takes on the GPU.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>

#include "qmv.h"

static int as_ptr(PyObject* o, void** out) {
    if (o == Py_None) { *out = NULL; return 0; }
    *out = PyLong_AsVoidPtr(o);
    return (*out == NULL && PyErr_Occurred()) ? -1 : 0;
}

/* A Python int that fits a C int; anything larger raises OverflowError
 * instead of being narrowed. */
static int as_int(PyObject* o, int* out) {
    long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return -1;
    if (v < INT_MIN || v > INT_MAX) {
        PyErr_SetString(PyExc_OverflowError, "argument does not fit a C int");
        return -1;
    }
    *out = (int)v;
    return 0;
}

static int as_ll(PyObject* o, long long* out) {
    *out = PyLong_AsLongLong(o);
    return (*out == -1 && PyErr_Occurred()) ? -1 : 0;
}

static int as_float(PyObject* o, float* out) {
    double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) return -1;
    *out = (float)v;
    return 0;
}

/* An array argument of the calls below: None, an int (a device address), or a
 * tensor, of which data_ptr() is taken.  A tensor that is not on device `dev` (-1:
 * not known) or not on a CUDA device at all sets *elsewhere. */
static PyObject *s_data_ptr, *s_get_device, *s_nbytes, *s_is_contiguous;
static int as_array(PyObject* o, int dev, void** out, int* elsewhere) {
    if (o == Py_None || PyLong_Check(o)) return as_ptr(o, out);
    PyObject* r = PyObject_CallMethodNoArgs(o, s_data_ptr);
    if (!r) return -1;
    *out = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    if (*out == NULL && PyErr_Occurred()) return -1;
    r = PyObject_CallMethodNoArgs(o, s_get_device);
    if (!r) return -1;
    const long d = PyLong_AsLong(r);
    Py_DECREF(r);
    if (d == -1 && PyErr_Occurred()) return -1;
    if (d < 0 || (dev >= 0 && d != dev)) *elsewhere = 1;
    return 0;
}

/* Whether a tensor does not hold `bytes` bytes in one piece: 1, 0, or -1 on an
 * error.  Addresses and None: 0, their size is not known. */
static int as_too_small(PyObject* o, long long bytes) {
    if (o == Py_None || PyLong_Check(o)) return 0;
    PyObject* r = PyObject_GetAttr(o, s_nbytes);
    if (!r) return -1;
    const long long has = PyLong_AsLongLong(r);
    Py_DECREF(r);
    if (has == -1 && PyErr_Occurred()) return -1;
    if (has < bytes) return 1;
    r = PyObject_CallMethodNoArgs(o, s_is_contiguous);
    if (!r) return -1;
    const int whole = PyObject_IsTrue(r);
    Py_DECREF(r);
    return whole < 0 ? -1 : !whole;
}

/* affine(x, w, scales, biases, y, M, N, K, bits, group, dtype, batch, x_batched, stream) -> status */
static PyObject* py_affine(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 14) { PyErr_SetString(PyExc_TypeError, "affine() takes 14 arguments"); return NULL; }
    void* p[5];
    int v[8];
    void* st;
    for (int i = 0; i < 5; ++i) if (as_ptr(a[i], &p[i])) return NULL;
    for (int i = 0; i < 8; ++i) if (as_int(a[5 + i], &v[i])) return NULL;
    if (as_ptr(a[13], &st)) return NULL;
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = qmv_affine_batched(p[0], p[1], p[2], p[3], p[4], v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

/* fp(x, w, scales, global_scale, y, M, N, K, mode, dtype, batch, x_batched, stream) -> status */
static PyObject* py_fp(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 13) { PyErr_SetString(PyExc_TypeError, "fp() takes 13 arguments"); return NULL; }
    void* p[5];
    int v[7];
    void* st;
    for (int i = 0; i < 5; ++i) if (as_ptr(a[i], &p[i])) return NULL;
    for (int i = 0; i < 7; ++i) if (as_int(a[5 + i], &v[i])) return NULL;
    if (as_ptr(a[12], &st)) return NULL;
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = qmv_fp_batched(p[0], p[1], p[2], (const float*)p[3], p[4], v[0], v[1], v[2], v[3], v[4], v[5], v[6], st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

/* block_scaled(x, w, scales, global_scale, y, M, N, K, format, dtype, batch, x_batched, stream) -> status */
static PyObject* py_block_scaled(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 13) { PyErr_SetString(PyExc_TypeError, "block_scaled() takes 13 arguments"); return NULL; }
    void* p[5];
    int v[7];
    void* st;
    for (int i = 0; i < 5; ++i) if (as_ptr(a[i], &p[i])) return NULL;
    for (int i = 0; i < 7; ++i) if (as_int(a[5 + i], &v[i])) return NULL;
    if (as_ptr(a[12], &st)) return NULL;
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = qmv_block_scaled_batched(p[0], p[1], p[2], (const float*)p[3], p[4], v[0], v[1], v[2], v[3], v[4], v[5],
                                 v[6], st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

/* rope(x, y, positions, inv_freq, T, H, D, rot, layout, dtype, xt, xh, yt, yh, magnitude, stream, device) -> status */
static PyObject* py_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 17) { PyErr_SetString(PyExc_TypeError, "rope() takes 17 arguments"); return NULL; }
    void* p[4];
    int v[6], dev, elsewhere = 0;
    long long s[4];
    float mag;
    void* st;
    if (as_int(a[16], &dev)) return NULL;
    for (int i = 0; i < 4; ++i) if (as_array(a[i], dev, &p[i], &elsewhere)) return NULL;
    for (int i = 0; i < 6; ++i) if (as_int(a[4 + i], &v[i])) return NULL;
    for (int i = 0; i < 4; ++i) if (as_ll(a[10 + i], &s[i])) return NULL;
    if (as_float(a[14], &mag) || as_ptr(a[15], &st)) return NULL;
    if (elsewhere) return PyLong_FromLong(QMV_EINVAL);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = qmv_rope(p[0], p[1], (const int*)p[2], (const float*)p[3], v[0], v[1], v[2], v[3], v[4], mag, s[0], s[1], s[2],
                 s[3], v[5], st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

/* The 15 leading arguments of the two calls on a paged cache: k, v,
 * page_table, q_starts, kv_lens, n_pages, page_size, n_kv_heads, head_dim,
 * dtype, n_seqs, max_pages, page_stride, token_stride, head_stride. */
static int as_cache(PyObject* const* a, int dev, qmv_paged_kv* kv, int* elsewhere) {
    void* p[5];
    int v[7];
    long long s[3];
    for (int i = 0; i < 5; ++i) if (as_array(a[i], dev, &p[i], elsewhere)) return -1;
    for (int i = 0; i < 7; ++i) if (as_int(a[5 + i], &v[i])) return -1;
    for (int i = 0; i < 3; ++i) if (as_ll(a[12 + i], &s[i])) return -1;
    kv->k = p[0]; kv->v = p[1];
    kv->page_table = (const int*)p[2]; kv->q_starts = (const int*)p[3]; kv->kv_lens = (const int*)p[4];
    kv->n_pages = v[0]; kv->page_size = v[1]; kv->n_kv_heads = v[2]; kv->head_dim = v[3]; kv->dtype = v[4];
    kv->n_seqs = v[5]; kv->max_pages = v[6];
    kv->page_stride = s[0]; kv->token_stride = s[1]; kv->head_stride = s[2];
    return 0;
}

/* kv_append(<cache>, qkv, positions, inv_freq, q_out, T, n_q_heads, rot, layout, qkv_stride, q_out_stride,
 * magnitude, stream, device) -> status */
static PyObject* py_kv_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 28) { PyErr_SetString(PyExc_TypeError, "kv_append() takes 28 arguments"); return NULL; }
    qmv_paged_kv kv;
    void* p[4];
    int v[4], dev, elsewhere = 0;
    long long s[2];
    float mag;
    void* st;
    if (as_int(a[27], &dev) || as_cache(a, dev, &kv, &elsewhere)) return NULL;
    for (int i = 0; i < 4; ++i) if (as_array(a[15 + i], dev, &p[i], &elsewhere)) return NULL;
    for (int i = 0; i < 4; ++i) if (as_int(a[19 + i], &v[i])) return NULL;
    for (int i = 0; i < 2; ++i) if (as_ll(a[23 + i], &s[i])) return NULL;
    if (as_float(a[25], &mag) || as_ptr(a[26], &st)) return NULL;
    if (elsewhere) return PyLong_FromLong(QMV_EINVAL);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = qmv_kv_append(p[0], s[0], &kv, (const int*)p[1], (const float*)p[2], p[3], s[1], v[0], v[1], v[2], v[3], mag,
                      st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

/* paged_attention(<cache>, q, out, lse, slopes, workspace, T, n_q_heads, causal, window, max_q_len, q_ts, q_hs,
 * out_ts, out_hs, scale, softcap, stream, device) -> status */
static PyObject* py_paged_attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 33) { PyErr_SetString(PyExc_TypeError, "paged_attention() takes 33 arguments"); return NULL; }
    qmv_paged_kv kv;
    void* p[5];
    int v[5], dev, elsewhere = 0;
    long long s[4];
    float f[2];
    void* st;
    if (as_int(a[32], &dev) || as_cache(a, dev, &kv, &elsewhere)) return NULL;
    for (int i = 0; i < 5; ++i) if (as_array(a[15 + i], dev, &p[i], &elsewhere)) return NULL;
    for (int i = 0; i < 5; ++i) if (as_int(a[20 + i], &v[i])) return NULL;
    for (int i = 0; i < 4; ++i) if (as_ll(a[25 + i], &s[i])) return NULL;
    for (int i = 0; i < 2; ++i) if (as_float(a[29 + i], &f[i])) return NULL;
    if (as_ptr(a[31], &st)) return NULL;
    const int small = as_too_small(a[19], QMV_PAGED_ATTENTION_WORKSPACE_BYTES);
    if (small < 0) return NULL;
    if (elsewhere || small) return PyLong_FromLong(QMV_EINVAL);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = qmv_paged_attention(p[0], &kv, p[1], (float*)p[2], v[0], v[1], f[0], v[2], v[3], f[1], (const float*)p[3],
                            s[0], s[1], s[2], s[3], v[4], p[4], st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

static PyMethodDef methods[] = {
    {"affine", (PyCFunction)(void (*)(void))py_affine, METH_FASTCALL, "qmv_affine_batched"},
    {"fp", (PyCFunction)(void (*)(void))py_fp, METH_FASTCALL, "qmv_fp_batched"},
    {"block_scaled", (PyCFunction)(void (*)(void))py_block_scaled, METH_FASTCALL, "qmv_block_scaled_batched"},
    {"rope", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, "qmv_rope"},
    {"kv_append", (PyCFunction)(void (*)(void))py_kv_append, METH_FASTCALL, "qmv_kv_append"},
    {"paged_attention", (PyCFunction)(void (*)(void))py_paged_attention, METH_FASTCALL, "qmv_paged_attention"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmv_fast", NULL, -1, methods};

PyMODINIT_FUNC PyInit__qmv_fast(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_nbytes = PyUnicode_InternFromString("nbytes");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    if (!s_data_ptr || !s_get_device || !s_nbytes || !s_is_contiguous) return NULL;
    return PyModule_Create(&module);
}
