/* The short calls' way from Python into libestream: what estream.py's kv_append,
 * kv_attend and sample_tokens check and hand over, without an interpreted step for
 * each. A function returns the status, or None for whatever it does not take as it is
 * (a wrong type or size, another device, a stream of its own, a workspace to be
 * allocated): Python then does the call, or says what is wrong with it. Tensors are
 * asked through their public methods; the current device and stream come from the
 * functions that setup is given. The file's name has the interpreter's tag and the
 * module the header's version, so that another interpreter or library leaves it alone. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "estream.h"

typedef estream_status (*append_fn)(const estream_kv_cache*, int, int, const void*, long long, long long, const void*,
                                    long long, long long, const int32_t*, const int32_t*, const int32_t*, int, int, long long,
                                    const void*, long long, long long, int, void*, long long, long long, const float*, int,
                                    int, void*);
typedef estream_status (*attend_fn)(const estream_kv_cache*, int, int, int, const void*, long long, long long, const int32_t*,
                                    int, long long, const int32_t*, float, int, void*, long long, long long, float*, void*,
                                    size_t, void*);
typedef size_t (*bytes_fn)(const estream_kv_cache*, int, int, int, int);
typedef estream_status (*sample_fn)(const void*, int, long long, int, int, const float*, float, const float*, int,
                                    const int32_t*, float, const float*, float, const float*, int32_t*, float*, void*);

static struct {
    append_fn append;
    attend_fn attend;
    bytes_fn attend_bytes;
    sample_fn sample;
    PyObject *tensor, *bf16, *f16, *f32, *i32, *u8, *device, *stream; /* types; the current device and its stream */
    PyObject *s_shape, *s_stride, *s_dtype, *s_get_device, *s_data_ptr;
} g;

typedef struct {
    PyObject* dtype; /* not owned: the types live as long as torch */
    void* p;
    long long n[4], s[4];
    int dims;
} Tensor;

static int numbers(PyObject* t, long long* to) { /* a tuple's; -1: not up to four of them */
    if (!t || !PyTuple_Check(t) || PyTuple_GET_SIZE(t) > 4) return -1;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(t); ++i) {
        PyObject* x = PyTuple_GET_ITEM(t, i);
        if (!PyLong_Check(x)) return -1;
        to[i] = PyLong_AsLongLong(x);
    }
    return (int)PyTuple_GET_SIZE(t);
}

/* A tensor on device `index`; 0: something else. */
static int tensor(PyObject* o, long index, Tensor* t) {
    int ok = 0;
    PyObject *shape = NULL, *stride = NULL, *dtype = NULL, *dev = NULL, *ptr = NULL;
    if ((PyObject*)Py_TYPE(o) != g.tensor) return 0;
    shape = PyObject_GetAttr(o, g.s_shape);
    stride = PyObject_CallMethodNoArgs(o, g.s_stride);
    dtype = PyObject_GetAttr(o, g.s_dtype);
    dev = PyObject_CallMethodNoArgs(o, g.s_get_device);
    ptr = PyObject_CallMethodNoArgs(o, g.s_data_ptr);
    if (shape && stride && dtype && dev && ptr && PyLong_Check(dev) && PyLong_AsLong(dev) == index) {
        t->dims = numbers(shape, t->n);
        if (t->dims >= 0 && numbers(stride, t->s) == t->dims) {
            t->dtype = dtype;
            t->p = PyLong_AsVoidPtr(ptr);
            ok = 1;
        }
    }
    Py_XDECREF(shape);
    Py_XDECREF(stride);
    Py_XDECREF(dtype);
    Py_XDECREF(dev);
    Py_XDECREF(ptr);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        ok = 0;
    }
    return ok;
}

static int row_of(PyObject* o, long index, long long n, PyObject* dtype, void** p) { /* [n], contiguous */
    Tensor t;
    if (!tensor(o, index, &t) || t.dims != 1 || t.n[0] != n || t.dtype != dtype || (n > 1 && t.s[0] != 1)) return 0;
    *p = t.p;
    return 1;
}
static int heads_of(PyObject* o, long index, long long n, long long heads, int dim, PyObject* dtype, int written, Tensor* t) {
    return tensor(o, index, t) && t->dims == 3 && t->n[0] == n && (heads < 0 || t->n[1] == heads) && t->n[2] == dim &&
           (!dtype || t->dtype == dtype) && t->s[2] == 1 &&
           !(written && ((n > 1 && t->s[0] < dim) || (t->n[1] > 1 && t->s[1] < dim)));
}
static int table_of(PyObject* o, long index, Tensor* t) {
    return tensor(o, index, t) && t->dims == 2 && t->dtype == g.i32 && (t->n[1] <= 1 || t->s[1] == 1) &&
           t->n[0] <= 1 << 24 && t->n[1] <= 1 << 30;
}
/* The current stream of device `index` when that is the current device. */
static int stream_of(long index, PyObject* py_index, void** stream) {
    PyObject* now = PyObject_CallNoArgs(g.device);
    const int here = now && PyLong_AsLong(now) == index;
    PyObject* s = here ? PyObject_CallOneArg(g.stream, py_index) : NULL;
    if (s) *stream = PyLong_AsVoidPtr(s);
    Py_XDECREF(now);
    Py_XDECREF(s);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return 0;
    }
    return s != NULL;
}
static int elem_of(PyObject* dtype, const estream_kv_cache* c) { /* of a call's rows; -1: not next to this cache */
    const int e = dtype == g.bf16 ? ESTREAM_KV_BF16 : dtype == g.f16 ? ESTREAM_KV_F16 : -1;
    return c->elem == ESTREAM_KV_E4M3 || c->elem == e ? e : -1;
}

/* (cache, index, k, v, positions, table, rows, q, inv_freq, interleaved, q_out) */
static PyObject* kv_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 11) Py_RETURN_NONE;
    const estream_kv_cache* c = (const estream_kv_cache*)PyLong_AsVoidPtr(a[0]);
    const long index = PyLong_AsLong(a[1]);
    Tensor k, v, table, q = {0}, out = {0};
    void *positions, *rows = NULL, *inv = NULL, *stream;
    int rot = 0;
    if (!c || !tensor(a[2], index, &k) || k.dims != 3) Py_RETURN_NONE;
    const long long T = k.n[0];
    const int elem = elem_of(k.dtype, c);
    if (elem < 0 || T > 1 << 24 || k.n[1] != c->heads || k.n[2] != c->dim || k.s[2] != 1 ||
        !heads_of(a[3], index, T, c->heads, c->dim, k.dtype, 0, &v) || !row_of(a[4], index, T, g.i32, &positions) ||
        !table_of(a[5], index, &table))
        Py_RETURN_NONE;
    if (a[6] == Py_None ? table.n[0] < T : !row_of(a[6], index, T, g.i32, &rows)) Py_RETURN_NONE;
    if (a[7] != Py_None) {
        if (!heads_of(a[7], index, T, -1, c->dim, k.dtype, 0, &q) || q.n[1] > 1 << 16 ||
            !heads_of(a[10], index, T, q.n[1], c->dim, k.dtype, 1, &out))
            Py_RETURN_NONE;
    } else if (a[10] != Py_None) {
        Py_RETURN_NONE;
    }
    if (a[8] != Py_None) {
        Tensor f;
        if (!tensor(a[8], index, &f) || f.dims != 1 || f.dtype != g.f32 || (f.n[0] > 1 && f.s[0] != 1) || 2 * f.n[0] > c->dim)
            Py_RETURN_NONE;
        rot = 2 * (int)f.n[0];
        inv = f.p;
    }
    const int interleaved = PyObject_IsTrue(a[9]);
    if (interleaved < 0 || !stream_of(index, a[1], &stream)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    estream_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g.append(c, elem, (int)T, k.p, k.s[0], k.s[1], v.p, v.s[0], v.s[1], positions, rows, table.p, (int)table.n[0],
                  (int)table.n[1], table.s[0], q.p, q.s[0], q.s[1], (int)q.n[1], out.p, out.s[0], out.s[1], inv, rot,
                  interleaved, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* (cache, index, q, table, lens, scale, window, out, lse, workspace) */
static PyObject* kv_attend(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 10) Py_RETURN_NONE;
    const estream_kv_cache* c = (const estream_kv_cache*)PyLong_AsVoidPtr(a[0]);
    const long index = PyLong_AsLong(a[1]);
    Tensor q, table, out;
    void *lens, *lse = NULL, *stream, *room = NULL;
    if (!c || !tensor(a[2], index, &q) || q.dims != 3 || q.n[2] != c->dim || q.s[2] != 1 || q.n[0] > 1 << 24 ||
        q.n[1] < 1 || q.n[1] > 1 << 16 || q.n[1] % c->heads)
        Py_RETURN_NONE;
    const int elem = elem_of(q.dtype, c), B = (int)q.n[0], Hq = (int)q.n[1];
    if (elem < 0 || !table_of(a[3], index, &table) || table.n[0] != B || !row_of(a[4], index, B, g.i32, &lens) ||
        !heads_of(a[7], index, B, Hq, c->dim, q.dtype, 1, &out))
        Py_RETURN_NONE;
    if (a[8] != Py_None) {
        Tensor t;
        if (!tensor(a[8], index, &t) || t.dims != 2 || t.n[0] != B || t.n[1] != Hq || t.dtype != g.f32 ||
            (Hq > 1 && t.s[1] != 1) || (B > 1 && t.s[0] != Hq))
            Py_RETURN_NONE;
        lse = t.p;
    }
    /* numbers alone: a tensor would be read, and waited for */
    if ((!PyFloat_Check(a[5]) && !PyLong_Check(a[5])) || !PyLong_Check(a[6])) Py_RETURN_NONE;
    const double scale = PyFloat_AsDouble(a[5]);
    const long window = PyLong_AsLong(a[6]);
    if (PyErr_Occurred() || window < 0 || window > 0x7fffffffl || !stream_of(index, a[1], &stream)) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    const size_t bytes = g.attend_bytes(c, B, Hq, (int)table.n[1], (int)window);
    if (a[9] != Py_None) {
        Tensor t;
        if (!tensor(a[9], index, &t) || t.dims != 1 || t.dtype != g.u8 || (t.n[0] > 1 && t.s[0] != 1) || (size_t)t.n[0] < bytes) Py_RETURN_NONE;
        room = t.p;
    } else if (bytes) {
        Py_RETURN_NONE;
    }
    estream_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g.attend(c, elem, B, Hq, q.p, q.s[0], q.s[1], table.p, (int)table.n[1], table.s[0], lens, (float)scale,
                  (int)window, out.p, out.s[0], out.s[1], lse, room, bytes, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* A choice: a number for all rows, or [B], one for each. */
static int choice(PyObject* o, long index, long long B, PyObject* dtype, double* number, void** rows) {
    *rows = NULL;
    *number = 0.0;
    if ((PyObject*)Py_TYPE(o) == g.tensor) return row_of(o, index, B, dtype, rows);
    if (!PyFloat_Check(o) && !PyLong_Check(o)) return 0;
    *number = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return 0;
    }
    return 1;
}

/* (index, logits, u, temperature, top_k, top_p, min_p, ids, prob) */
static PyObject* sample(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 9) Py_RETURN_NONE;
    const long index = PyLong_AsLong(a[0]);
    Tensor l;
    if (index < 0 || !tensor(a[1], index, &l) || l.dims != 2 || (l.n[1] > 1 && l.s[1] != 1) || l.n[0] > 1 << 20 ||
        l.n[1] < 1 || l.n[1] > ESTREAM_SAMPLE_MAX_V)
        Py_RETURN_NONE;
    const int elem = l.dtype == g.bf16 ? ESTREAM_MX4_BF16 : l.dtype == g.f16 ? ESTREAM_MX4_F16 : l.dtype == g.f32 ? ESTREAM_MX4_F32 : -1;
    const long long B = l.n[0];
    double temperature, top_k, top_p, min_p;
    void *u, *ts, *ks, *ps, *ms, *ids, *prob = NULL, *stream;
    if (elem < 0 || !row_of(a[2], index, B, g.f32, &u) || !choice(a[3], index, B, g.f32, &temperature, &ts) ||
        !choice(a[4], index, B, g.i32, &top_k, &ks) || !choice(a[5], index, B, g.f32, &top_p, &ps) ||
        !choice(a[6], index, B, g.f32, &min_p, &ms) || !row_of(a[7], index, B, g.i32, &ids) ||
        (a[8] != Py_None && !row_of(a[8], index, B, g.f32, &prob)))
        Py_RETURN_NONE;
    if (!ks && (PyFloat_Check(a[4]) || top_k < -0x7fffffff || top_k > 0x7fffffff)) Py_RETURN_NONE;
    if (!stream_of(index, a[0], &stream)) Py_RETURN_NONE;
    estream_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g.sample(l.p, elem, l.s[0], (int)B, (int)l.n[1], u, (float)temperature, ts, (int)top_k, ks, (float)top_p, ps,
                  (float)min_p, ms, ids, prob, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* (addresses of the four functions, torch.Tensor, bfloat16, float16, float32, int32, uint8, current device, raw stream) */
static PyObject* setup(PyObject* self, PyObject* args) {
    (void)self;
    unsigned long long append, attend, bytes, sampler;
    if (!PyArg_ParseTuple(args, "KKKKOOOOOOOO", &append, &attend, &bytes, &sampler, &g.tensor, &g.bf16, &g.f16, &g.f32, &g.i32,
                          &g.u8, &g.device, &g.stream))
        return NULL;
    PyObject* kept[] = {g.tensor, g.bf16, g.f16, g.f32, g.i32, g.u8, g.device, g.stream};
    for (size_t i = 0; i < sizeof kept / sizeof *kept; ++i) Py_INCREF(kept[i]);
    g.append = (append_fn)(uintptr_t)append;
    g.attend = (attend_fn)(uintptr_t)attend;
    g.attend_bytes = (bytes_fn)(uintptr_t)bytes;
    g.sample = (sample_fn)(uintptr_t)sampler;
    g.s_shape = PyUnicode_InternFromString("shape");
    g.s_stride = PyUnicode_InternFromString("stride");
    g.s_dtype = PyUnicode_InternFromString("dtype");
    g.s_get_device = PyUnicode_InternFromString("get_device");
    g.s_data_ptr = PyUnicode_InternFromString("data_ptr");
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, NULL},
    {"kv_attend", (PyCFunction)(void (*)(void))kv_attend, METH_FASTCALL, NULL},
    {"sample", (PyCFunction)(void (*)(void))sample, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "The short calls' way into libestream.", -1, methods,
                                    NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__binding(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddIntConstant(m, "version", ESTREAM_VERSION)) {
        Py_DECREF(m);
        return NULL;
    }
    return m;
}
