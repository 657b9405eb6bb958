/*
 * Argument marshalling of the calls that a serving loop makes for every layer
 * and token: from torch tensors to the C ABI in one step. Interpreting the
 * checks in Python and converting the arguments with ctypes took 4 of the 6 us
 * that a small call cost; here they take under one.
 *
 * Knows torch only by attributes (dtype, shape, stride(), data_ptr(),
 * get_device()). init() receives the entry points' addresses, the dtype
 * objects and torch's current-device and current-stream functions. Each call
 * returns the patch_status; a tensor that does not fit raises ValueError or
 * TypeError before anything is launched.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "patch_hybrid.h"

static PyObject *g_dtype[4];                       /* by patch_dtype */
static PyObject *g_device, *g_stream;
static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_get_device;
static __typeof__(&patch_linear_q8) f_linear;
static __typeof__(&patch_group_linear_q8) f_group;
static __typeof__(&patch_quantize_q8) f_quantize;
static __typeof__(&patch_rmsnorm_q8) f_rmsnorm;
static __typeof__(&patch_silu_mul_q8) f_silu_mul;
static __typeof__(&patch_dequantize_q8) f_dequantize;

typedef struct {
    void *p;
    int64_t rows, cols, ld;
    int type;
} Mat;

static int as_i64(PyObject *o, int64_t *v) {
    *v = o ? PyLong_AsLongLong(o) : -1;
    return *v == -1 && PyErr_Occurred() ? -1 : 0;
}

/* A tensor of `dims` dimensions (1 or 2) with contiguous elements in a row, on device `dev`. */
static int matrix(PyObject *t, const char *name, int dims, long dev, Mat *m) {
    PyObject *o = PyObject_GetAttr(t, s_dtype);
    if (!o) return -1;
    Py_DECREF(o);  /* the dtype objects live as long as torch */
    m->type = -1;
    for (int i = 0; i < 4; ++i)
        if (o == g_dtype[i]) m->type = i;
    PyObject *shape = PyObject_GetAttr(t, s_shape);
    if (!shape) return -1;
    if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != dims) {
        Py_DECREF(shape);
        PyErr_Format(PyExc_TypeError, "%s must be a %d-D tensor", name, dims);
        return -1;
    }
    int64_t step = 1;
    int bad = as_i64(PyTuple_GET_ITEM(shape, dims - 1), &m->cols);
    m->rows = 1;
    if (dims == 2) bad |= as_i64(PyTuple_GET_ITEM(shape, 0), &m->rows);
    Py_DECREF(shape);
    PyObject *stride = bad ? NULL : PyObject_CallMethodNoArgs(t, s_stride);
    if (!stride) return -1;
    if (!PyTuple_Check(stride) || PyTuple_GET_SIZE(stride) != dims) {
        Py_DECREF(stride);
        PyErr_Format(PyExc_TypeError, "%s must be a strided tensor", name);
        return -1;
    }
    bad = as_i64(PyTuple_GET_ITEM(stride, dims - 1), &step);
    m->ld = m->cols;
    if (dims == 2) bad |= as_i64(PyTuple_GET_ITEM(stride, 0), &m->ld);
    Py_DECREF(stride);
    if (bad) return -1;
    if (step != 1 && m->cols > 1) {
        PyErr_Format(PyExc_ValueError, "%s: the elements of a row must be contiguous", name);
        return -1;
    }
    int64_t on;
    o = PyObject_CallMethodNoArgs(t, s_get_device);
    bad = as_i64(o, &on);
    Py_XDECREF(o);
    if (bad) return -1;
    if (on != dev) {
        PyErr_Format(PyExc_ValueError, "%s is on device %lld (-1: the CPU), the current CUDA device is %ld", name,
                     (long long)on, dev);
        return -1;
    }
    o = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!o) return -1;
    m->p = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    return PyErr_Occurred() ? -1 : 0;
}

static int want(const Mat *m, const char *name, int64_t rows, int64_t cols, int type) {
    if (m->type != type) {
        PyErr_Format(PyExc_TypeError, "%s is not of type %R", name, g_dtype[type]);
        return -1;
    }
    if (m->rows != rows || m->cols != cols) {
        PyErr_Format(PyExc_ValueError, "%s has %lld x %lld elements, not %lld x %lld", name, (long long)m->rows,
                     (long long)m->cols, (long long)rows, (long long)cols);
        return -1;
    }
    return 0;
}

static int number_type(const Mat *m, const char *name) {
    if (m->type < 0 || m->type == PATCH_INT8) {
        PyErr_Format(PyExc_TypeError, "%s must be bf16, fp16 or fp32", name);
        return -1;
    }
    return 0;
}

static int current_device(PyObject *first, long *dev) {
    if (!g_device) {
        PyErr_SetString(PyExc_RuntimeError, "init() has not run");
        return -1;
    }
    /* a tensor on the CPU is refused before torch is asked for a CUDA device */
    PyObject *o = PyObject_CallMethodNoArgs(first, s_get_device);
    if (!o) return -1;
    const long on = PyLong_AsLong(o);
    Py_DECREF(o);
    if (PyErr_Occurred()) return -1;
    if (on < 0) {
        PyErr_SetString(PyExc_ValueError, "the tensors must be on the current CUDA device");
        return -1;
    }
    if (!(o = PyObject_CallNoArgs(g_device))) return -1;
    *dev = PyLong_AsLong(o);
    Py_DECREF(o);
    return PyErr_Occurred() ? -1 : 0;
}

/* stream: None (the current one), an int, or an object with .cuda_stream */
static int stream_of(PyObject *stream, long dev, void **out) {
    PyObject *o;
    if (stream == Py_None) {
        PyObject *d = PyLong_FromLong(dev);
        if (!d) return -1;
        o = PyObject_CallOneArg(g_stream, d);
        Py_DECREF(d);
    } else if (PyLong_Check(stream)) {
        o = Py_NewRef(stream);
    } else {
        o = PyObject_GetAttrString(stream, "cuda_stream");
    }
    if (!o) return -1;
    *out = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    return PyErr_Occurred() ? -1 : 0;
}

#define CALL(expr)                \
    int st;                       \
    Py_BEGIN_ALLOW_THREADS        \
    st = (int)(expr);             \
    Py_END_ALLOW_THREADS          \
    return PyLong_FromLong(st)

static int count(Py_ssize_t n, Py_ssize_t need) {
    if (n != need) PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", need, n);
    return n == need ? 0 : -1;
}

/* linear_q8(handle, N, K, X, x_scale, Y, path, stream) */
static PyObject *linear_q8(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Mat x, s, y;
    long dev;
    void *stream;
    (void)self;
    if (count(n, 8)) return NULL;
    void *h = PyLong_AsVoidPtr(a[0]);
    const int64_t N = PyLong_AsLongLong(a[1]), K = PyLong_AsLongLong(a[2]);
    const long path = PyLong_AsLong(a[6]);
    if (PyErr_Occurred() || current_device(a[3], &dev) || matrix(a[3], "X", 2, dev, &x) ||
        matrix(a[4], "x_scale", 1, dev, &s) || matrix(a[5], "Y", 2, dev, &y) || want(&x, "X", x.rows, K, PATCH_INT8) ||
        want(&s, "x_scale", 1, x.rows, PATCH_FP32) || number_type(&y, "Y") || want(&y, "Y", x.rows, N, y.type) ||
        stream_of(a[7], dev, &stream))
        return NULL;
    CALL(f_linear(h, x.p, x.ld, s.p, x.rows, y.p, y.ld, y.type, (int)path, stream));
}

/*
 * group_linear_q8(handle, (N0, K0, N1, K1, ...), Xs, x_scales, outs, path, stream),
 * the operands in tuples; one that several members share is looked at once
 */
enum { kMembers = 8 };
static PyObject *group_linear_q8(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    const void *xp[kMembers], *sp[kMembers];
    void *yp[kMembers], *stream;
    int64_t ldx[kMembers], ldy[kMembers];
    Mat x = {0}, s = {0}, y = {0};
    int type = -1;
    int64_t M = -1;
    long dev;
    (void)self;
    if (count(n, 7)) return NULL;
    void *h = PyLong_AsVoidPtr(a[0]);
    const long path = PyLong_AsLong(a[5]);
    if (PyErr_Occurred()) return NULL;
    for (int i = 1; i < 5; ++i)
        if (!PyTuple_Check(a[i])) {
            PyErr_SetString(PyExc_TypeError, "shapes, Xs, x_scales and outs must be tuples");
            return NULL;
        }
    const Py_ssize_t g = PyTuple_GET_SIZE(a[2]);
    if (g < 1 || g > kMembers || PyTuple_GET_SIZE(a[1]) != 2 * g || PyTuple_GET_SIZE(a[3]) != g ||
        PyTuple_GET_SIZE(a[4]) != g) {
        PyErr_Format(PyExc_ValueError, "one X, x_scale and out for each of 1 to %d members", (int)kMembers);
        return NULL;
    }
    if (current_device(PyTuple_GET_ITEM(a[2], 0), &dev) || stream_of(a[6], dev, &stream)) return NULL;
    for (Py_ssize_t l = 0; l < g; ++l) {
        int64_t N, K;
        PyObject *xo = PyTuple_GET_ITEM(a[2], l), *so = PyTuple_GET_ITEM(a[3], l);
        if (as_i64(PyTuple_GET_ITEM(a[1], 2 * l), &N) || as_i64(PyTuple_GET_ITEM(a[1], 2 * l + 1), &K)) return NULL;
        if ((l == 0 || xo != PyTuple_GET_ITEM(a[2], l - 1)) && matrix(xo, "X", 2, dev, &x)) return NULL;
        if ((l == 0 || so != PyTuple_GET_ITEM(a[3], l - 1)) && matrix(so, "x_scale", 1, dev, &s)) return NULL;
        if (matrix(PyTuple_GET_ITEM(a[4], l), "out", 2, dev, &y) || number_type(&y, "out")) return NULL;
        if (l == 0) {
            M = x.rows;
            type = y.type;
        }
        if (want(&x, "X", M, K, PATCH_INT8) || want(&s, "x_scale", 1, M, PATCH_FP32) || want(&y, "out", M, N, type))
            return NULL;
        xp[l] = x.p;
        ldx[l] = x.ld;
        sp[l] = s.p;
        yp[l] = y.p;
        ldy[l] = y.ld;
    }
    CALL(f_group(h, (const int8_t *const *)xp, ldx, (const float *const *)sp, M, yp, ldy, type, (int)path, stream));
}

/* quantize_q8(x, q, scale, stream) */
static PyObject *quantize_q8(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Mat x, q, s;
    long dev;
    void *stream;
    (void)self;
    if (count(n, 4) || current_device(a[0], &dev) || matrix(a[0], "x", 2, dev, &x) || number_type(&x, "x") ||
        matrix(a[1], "q", 2, dev, &q) || matrix(a[2], "scale", 1, dev, &s) ||
        want(&q, "q", x.rows, x.cols, PATCH_INT8) || want(&s, "scale", 1, x.rows, PATCH_FP32) ||
        stream_of(a[3], dev, &stream))
        return NULL;
    CALL(f_quantize(x.p, x.ld, x.type, x.rows, x.cols, q.p, q.ld, s.p, stream));
}

/* rmsnorm_q8(x, gamma, eps, q, scale, residual, residual_out, stream) */
static PyObject *rmsnorm_q8(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Mat x, g, q, s, r = {0}, ro = {0};
    long dev;
    void *stream;
    (void)self;
    if (count(n, 8)) return NULL;
    const double eps = PyFloat_AsDouble(a[2]);
    if (PyErr_Occurred()) return NULL;
    if ((a[5] == Py_None) != (a[6] == Py_None)) {
        PyErr_SetString(PyExc_ValueError, "residual and residual_out go together");
        return NULL;
    }
    if (current_device(a[0], &dev) || matrix(a[0], "x", 2, dev, &x) || number_type(&x, "x") ||
        matrix(a[1], "gamma", 1, dev, &g) || matrix(a[3], "q", 2, dev, &q) || matrix(a[4], "scale", 1, dev, &s) ||
        want(&g, "gamma", 1, x.cols, x.type) || want(&q, "q", x.rows, x.cols, PATCH_INT8) ||
        want(&s, "scale", 1, x.rows, PATCH_FP32) || stream_of(a[7], dev, &stream))
        return NULL;
    if (a[5] != Py_None &&
        (matrix(a[5], "residual", 2, dev, &r) || matrix(a[6], "residual_out", 2, dev, &ro) ||
         want(&r, "residual", x.rows, x.cols, x.type) || want(&ro, "residual_out", x.rows, x.cols, x.type)))
        return NULL;
    CALL(f_rmsnorm(x.p, x.ld, r.p, r.ld, ro.p, ro.ld, g.p, x.type, (float)eps, x.rows, x.cols, q.p, q.ld, s.p, stream));
}

/* silu_mul_q8(gate, up, q, scale, stream) */
static PyObject *silu_mul_q8(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Mat x, u, q, s;
    long dev;
    void *stream;
    (void)self;
    if (count(n, 5) || current_device(a[0], &dev) || matrix(a[0], "gate", 2, dev, &x) || number_type(&x, "gate") ||
        matrix(a[1], "up", 2, dev, &u) || matrix(a[2], "q", 2, dev, &q) || matrix(a[3], "scale", 1, dev, &s) ||
        want(&u, "up", x.rows, x.cols, x.type) || want(&q, "q", x.rows, x.cols, PATCH_INT8) ||
        want(&s, "scale", 1, x.rows, PATCH_FP32) || stream_of(a[4], dev, &stream))
        return NULL;
    CALL(f_silu_mul(x.p, x.ld, u.p, u.ld, x.type, x.rows, x.cols, q.p, q.ld, s.p, stream));
}

/* dequantize_q8(q, scale, out, stream) */
static PyObject *dequantize_q8(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Mat q, s, x;
    long dev;
    void *stream;
    (void)self;
    if (count(n, 4) || current_device(a[2], &dev) || matrix(a[0], "q", 2, dev, &q) || matrix(a[1], "scale", 1, dev, &s) ||
        matrix(a[2], "out", 2, dev, &x) || number_type(&x, "out") || want(&q, "q", x.rows, x.cols, PATCH_INT8) ||
        want(&s, "scale", 1, x.rows, PATCH_FP32) || stream_of(a[3], dev, &stream))
        return NULL;
    CALL(f_dequantize(q.p, q.ld, s.p, x.rows, x.cols, x.p, x.ld, x.type, stream));
}

/* init((dtypes by patch_dtype), current_device, current_raw_stream, (addresses)) */
static PyObject *init(PyObject *self, PyObject *args) {
    PyObject *dtypes, *device, *stream;
    unsigned long long f[6];
    (void)self;
    if (!PyArg_ParseTuple(args, "O!OO(KKKKKK)", &PyTuple_Type, &dtypes, &device, &stream, &f[0], &f[1], &f[2], &f[3],
                          &f[4], &f[5]))
        return NULL;
    if (PyTuple_GET_SIZE(dtypes) != 4) {
        PyErr_SetString(PyExc_ValueError, "four dtypes");
        return NULL;
    }
    for (int i = 0; i < 4; ++i) Py_XSETREF(g_dtype[i], Py_NewRef(PyTuple_GET_ITEM(dtypes, i)));
    Py_XSETREF(g_device, Py_NewRef(device));
    Py_XSETREF(g_stream, Py_NewRef(stream));
    f_linear = (__typeof__(f_linear))(uintptr_t)f[0];
    f_quantize = (__typeof__(f_quantize))(uintptr_t)f[1];
    f_rmsnorm = (__typeof__(f_rmsnorm))(uintptr_t)f[2];
    f_silu_mul = (__typeof__(f_silu_mul))(uintptr_t)f[3];
    f_dequantize = (__typeof__(f_dequantize))(uintptr_t)f[4];
    f_group = (__typeof__(f_group))(uintptr_t)f[5];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, NULL},
    {"linear_q8", (PyCFunction)(void (*)(void))linear_q8, METH_FASTCALL, NULL},
    {"group_linear_q8", (PyCFunction)(void (*)(void))group_linear_q8, METH_FASTCALL, NULL},
    {"quantize_q8", (PyCFunction)(void (*)(void))quantize_q8, METH_FASTCALL, NULL},
    {"rmsnorm_q8", (PyCFunction)(void (*)(void))rmsnorm_q8, METH_FASTCALL, NULL},
    {"silu_mul_q8", (PyCFunction)(void (*)(void))silu_mul_q8, METH_FASTCALL, NULL},
    {"dequantize_q8", (PyCFunction)(void (*)(void))dequantize_q8, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_get_device = PyUnicode_InternFromString("get_device");
    if (!s_dtype || !s_shape || !s_stride || !s_data_ptr || !s_get_device) return NULL;
    return PyModule_Create(&module);
}
