/*
 * Argument marshalling of the norm, 8-bit quantiser and 8-bit Linear layer for
 * Python: torch tensors to the C ABI of include/vnm.h.
 *
 * These calls stand in decode loops, where one takes a few microseconds on the
 * GPU. Reading a tensor's shape, type, device, strides and address from Python
 * and passing two dozen arguments through ctypes costs 7 us a call; the same reads
 * from C cost 2. Nothing is computed here: every check is of a tensor's description,
 * and the functions called are the library's exported ones, whose addresses
 * setup() is given.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/vnm.h"

static __typeof__(&vnm_rmsnorm) fn_rmsnorm;
static __typeof__(&vnm_rmsnorm_backward) fn_rmsnorm_backward;
static __typeof__(&vnm_rmsnorm_backward_workspace_size) fn_rmsnorm_workspace;
static __typeof__(&vnm_fp8_quantize) fn_quantize;
static __typeof__(&vnm_fp8_linear) fn_linear;
typedef vnm_status (*testing_linear_t)(const void*, int64_t, vnm_fp8, const float*, int64_t, int64_t, const void*, int64_t,
                                       vnm_fp8, const float*, int64_t, int64_t, int32_t, int64_t, int64_t, int64_t,
                                       const void*, vnm_dtype, vnm_activation, void*, int64_t, vnm_dtype, int32_t*, int32_t,
                                       vnm_stream_t);
static testing_linear_t fn_linear_skip;

static PyObject *py_f16, *py_f32, *py_bf16, *py_e4m3, *py_e5m2, *py_i32; /* torch dtypes */
static PyObject *py_current_device, *py_current_stream;
static PyObject *s_shape, *s_dtype, *s_get_device, *s_stride, *s_data_ptr, *s_cuda_stream;

/* A tensor's description. */
typedef struct {
    int64_t rows, cols; /* a vector: cols = its length, rows = -1 */
    PyObject* dtype;    /* borrowed: torch's dtype objects live for good */
} Desc;

static int long_of(PyObject* o, int64_t* out) {
    if (o == NULL) return -1;
    *out = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int ints_of(PyObject* t, int64_t* v, Py_ssize_t* n) { /* up to two whole numbers of a tuple; steals t */
    if (t == NULL) return -1;
    if (!PyTuple_Check(t)) {
        Py_DECREF(t);
        PyErr_SetString(PyExc_TypeError, "expected a torch tensor");
        return -1;
    }
    *n = PyTuple_GET_SIZE(t);
    for (Py_ssize_t i = 0; i < *n && i < 2; ++i) {
        v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
        if (v[i] == -1 && PyErr_Occurred()) {
            Py_DECREF(t);
            return -1;
        }
    }
    Py_DECREF(t);
    return 0;
}

static int describe(PyObject* t, Desc* d, int64_t* device) {
    int64_t v[2] = {0, 0};
    Py_ssize_t n = 0;
    if (ints_of(PyObject_GetAttr(t, s_shape), v, &n) < 0) return -1;
    d->rows = n == 2 ? v[0] : -1;
    d->cols = n == 2 ? v[1] : n == 1 ? v[0] : -1;
    if (n != 1 && n != 2) d->rows = -2;
    d->dtype = PyObject_GetAttr(t, s_dtype);
    if (d->dtype == NULL) return -1;
    Py_DECREF(d->dtype);
    return long_of(PyObject_CallMethodNoArgs(t, s_get_device), device);
}

static int refuse(PyObject* t, const char* name, int64_t rows, int64_t cols, PyObject* dtype, int64_t device) {
    PyObject* shape = PyObject_GetAttr(t, s_shape);
    PyObject* got = PyObject_GetAttr(t, s_dtype);
    PyObject* want = dtype ? PyObject_Str(dtype) : PyUnicode_FromString("any type served");
    if (shape && got && want) {
        if (rows >= 0)
            PyErr_Format(PyExc_ValueError, "%s must be a row-major tensor of shape (%lld, %lld), %U, on cuda:%lld; got %S, %S", name,
                         (long long)rows, (long long)cols, want, (long long)device, shape, got);
        else
            PyErr_Format(PyExc_ValueError, "%s must be a contiguous tensor of shape (%lld,), %U, on cuda:%lld; got %S, %S", name,
                         (long long)cols, want, (long long)device, shape, got);
    }
    Py_XDECREF(shape);
    Py_XDECREF(got);
    Py_XDECREF(want);
    return -1;
}

static int address(PyObject* t, void** p) {
    int64_t v;
    if (long_of(PyObject_CallMethodNoArgs(t, s_data_ptr), &v) < 0) return -1;
    *p = (void*)(intptr_t)v;
    return 0;
}

/* Row-major rows x cols (rows = -1: a contiguous vector), of a type or (dtype NULL) any. */
static int tensor(PyObject* t, const char* name, int64_t rows, int64_t cols, PyObject* dtype, int64_t device, void** p,
                  int64_t* ld) {
    *p = NULL;
    *ld = 1;
    if (t == Py_None) return 0;
    Desc d;
    int64_t dev, st[2] = {1, 1};
    Py_ssize_t n;
    if (describe(t, &d, &dev) < 0 || ints_of(PyObject_CallMethodNoArgs(t, s_stride), st, &n) < 0) return -1;
    if (d.rows != rows || d.cols != cols || dev != device || (dtype != NULL && d.dtype != dtype) ||
        (cols > 1 && st[n - 1] != 1))
        return refuse(t, name, rows, cols, dtype, device);
    /* (a matrix of one row may carry any stride) */
    if (rows >= 0) *ld = st[0] >= cols && st[0] > 0 ? st[0] : cols > 0 ? cols : 1;
    return address(t, p);
}

/* fp32 scales of any strides. */
static int scales(PyObject* t, const char* name, int64_t rows, int64_t cols, int64_t device, float** p, int64_t* rs,
                  int64_t* cs) {
    *p = NULL;
    *rs = *cs = 0;
    if (t == Py_None) return 0;
    Desc d;
    int64_t dev, st[2] = {0, 0};
    Py_ssize_t n;
    if (describe(t, &d, &dev) < 0 || ints_of(PyObject_CallMethodNoArgs(t, s_stride), st, &n) < 0) return -1;
    if (d.rows != rows || d.cols != cols || dev != device || d.dtype != py_f32)
        return refuse(t, name, rows, cols, py_f32, device);
    *rs = st[0];
    *cs = st[1];
    void* v;
    if (address(t, &v) < 0) return -1;
    *p = v;
    return 0;
}

static int dtype_of(PyObject* dtype, const char* name, vnm_dtype* out) {
    if (dtype == py_f16)
        *out = VNM_F16;
    else if (dtype == py_bf16)
        *out = VNM_BF16;
    else if (dtype == py_f32)
        *out = VNM_F32;
    else {
        PyErr_Format(PyExc_ValueError, "%s must be fp16, bf16 or fp32", name);
        return -1;
    }
    return 0;
}

static int fp8_of(PyObject* dtype, const char* name, vnm_fp8* out) {
    if (dtype == py_e4m3)
        *out = VNM_E4M3;
    else if (dtype == py_e5m2)
        *out = VNM_E5M2;
    else {
        PyErr_Format(PyExc_ValueError, "%s must be float8_e4m3fn or float8_e5m2", name);
        return -1;
    }
    return 0;
}

/* The type of a tensor argument that may be None (then `none`). */
static PyObject* type_of(PyObject* t) {
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    Py_XDECREF(d);
    return d;
}

/* The call's first tensor: a matrix on the current CUDA device. */
static int first(PyObject* t, const char* name, Desc* d, int64_t* device) {
    int64_t cur;
    if (describe(t, d, device) < 0) return -1;
    if (d->rows < 0 || *device < 0) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA matrix", name);
        return -1;
    }
    if (long_of(PyObject_CallNoArgs(py_current_device), &cur) < 0) return -1;
    if (cur != *device) {
        PyErr_Format(PyExc_ValueError, "%s must be on the current CUDA device", name);
        return -1;
    }
    return 0;
}

/* The stream's handle: of the given one, or torch's current one on the device. */
static int stream_of(PyObject* stream, int64_t device, vnm_stream_t* out) {
    int64_t v;
    if (stream == Py_None) {
        PyObject* i = PyLong_FromLongLong(device);
        if (i == NULL) return -1;
        PyObject* r = PyObject_CallOneArg(py_current_stream, i);
        Py_DECREF(i);
        if (long_of(r, &v) < 0) return -1;
    } else if (long_of(PyObject_GetAttr(stream, s_cuda_stream), &v) < 0) {
        return -1;
    }
    *out = (vnm_stream_t)(intptr_t)v;
    return 0;
}

static int64_t groups(int64_t n) { return (n + 127) / 128; }

static int count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return 0;
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return -1;
}

/* x, weight, eps, residual, h, y, rstd, q, q_scale, stream -> status */
static PyObject* rmsnorm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Desc x, dq;
    int64_t dev, ld_x, ld_r, ld_h, ld_y, ld_q, one, rs, cs, q_dev;
    void *xp, *rp, *wp, *hp, *yp, *sp, *qp;
    float* cp;
    vnm_dtype type;
    vnm_fp8 q_type = VNM_E4M3;
    vnm_stream_t stream;
    if (count(n, 10) < 0 || first(a[0], "x", &x, &dev) < 0 || dtype_of(x.dtype, "x", &type) < 0) return NULL;
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) return NULL;
    const int64_t T = x.rows, D = x.cols;
    if (tensor(a[0], "x", T, D, NULL, dev, &xp, &ld_x) < 0 || tensor(a[1], "weight", -1, D, x.dtype, dev, &wp, &one) < 0 ||
        tensor(a[3], "residual", T, D, x.dtype, dev, &rp, &ld_r) < 0 || tensor(a[4], "h", T, D, x.dtype, dev, &hp, &ld_h) < 0 ||
        tensor(a[5], "y", T, D, x.dtype, dev, &yp, &ld_y) < 0 || tensor(a[6], "rstd", -1, T, py_f32, dev, &sp, &one) < 0 ||
        tensor(a[7], "q", T, D, NULL, dev, &qp, &ld_q) < 0 || scales(a[8], "q_scale", T, groups(D), dev, &cp, &rs, &cs) < 0)
        return NULL;
    if (a[7] != Py_None && (describe(a[7], &dq, &q_dev) < 0 || fp8_of(dq.dtype, "q", &q_type) < 0)) return NULL;
    if (stream_of(a[9], dev, &stream) < 0) return NULL;
    vnm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn_rmsnorm(xp, ld_x, rp, ld_r, wp, (float)eps, T, D, type, hp, ld_h, yp, ld_y, sp, qp, ld_q, q_type, cp, rs, cs, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* dy, h, weight, rstd, dh, dweight, dresidual, workspace address, workspace bytes, stream -> status */
static PyObject* rmsnorm_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Desc x;
    int64_t dev, ld_dy, ld_h, ld_r, ld_o, one, ws, bytes;
    void *yp, *hp, *wp, *sp, *rp, *op, *gp;
    vnm_dtype type;
    vnm_stream_t stream;
    if (count(n, 10) < 0 || first(a[0], "dy", &x, &dev) < 0 || dtype_of(x.dtype, "dy", &type) < 0) return NULL;
    const int64_t T = x.rows, D = x.cols;
    if (tensor(a[0], "dy", T, D, NULL, dev, &yp, &ld_dy) < 0 || tensor(a[1], "h", T, D, x.dtype, dev, &hp, &ld_h) < 0 ||
        tensor(a[2], "weight", -1, D, x.dtype, dev, &wp, &one) < 0 || tensor(a[3], "rstd", -1, T, py_f32, dev, &sp, &one) < 0 ||
        tensor(a[4], "dh", T, D, x.dtype, dev, &op, &ld_o) < 0 || tensor(a[5], "dweight", -1, D, py_f32, dev, &gp, &one) < 0 ||
        tensor(a[6], "dresidual", T, D, x.dtype, dev, &rp, &ld_r) < 0)
        return NULL;
    ws = PyLong_AsLongLong(a[7]);
    bytes = PyLong_AsLongLong(a[8]);
    if (PyErr_Occurred() || stream_of(a[9], dev, &stream) < 0) return NULL;
    vnm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn_rmsnorm_backward(yp, ld_dy, hp, ld_h, wp, sp, rp, ld_r, T, D, type, op, ld_o, gp, (void*)(intptr_t)ws,
                             (size_t)bytes, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* X, q, s, qt, st, block_rows, stream -> status */
static PyObject* fp8_quantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Desc x;
    int64_t dev, ld_x, ld_q, ld_t, rs, cs, trs, tcs;
    void *xp, *qp, *tp;
    float *sp, *up;
    vnm_dtype type;
    vnm_fp8 q_type = VNM_E4M3, t_type = VNM_E4M3;
    vnm_stream_t stream;
    PyObject* d;
    if (count(n, 7) < 0 || first(a[0], "X", &x, &dev) < 0 || dtype_of(x.dtype, "X", &type) < 0) return NULL;
    const long block = PyLong_AsLong(a[5]);
    if (block == -1 && PyErr_Occurred()) return NULL;
    const int64_t R = x.rows, C = x.cols, per = block > 0 ? block : 1;
    if (a[1] != Py_None && ((d = type_of(a[1])) == NULL || fp8_of(d, "q", &q_type) < 0)) return NULL;
    if (a[3] != Py_None && ((d = type_of(a[3])) == NULL || fp8_of(d, "qt", &t_type) < 0)) return NULL;
    if (a[1] != Py_None && a[3] != Py_None && q_type != t_type) {
        PyErr_SetString(PyExc_ValueError, "q and qt must have the same type");
        return NULL;
    }
    if (tensor(a[0], "X", R, C, NULL, dev, &xp, &ld_x) < 0 || tensor(a[1], "q", R, C, NULL, dev, &qp, &ld_q) < 0 ||
        scales(a[2], "s", (R + per - 1) / per, groups(C), dev, &sp, &rs, &cs) < 0 ||
        tensor(a[3], "qt", C, R, NULL, dev, &tp, &ld_t) < 0 ||
        scales(a[4], "st", (C + per - 1) / per, groups(R), dev, &up, &trs, &tcs) < 0 || stream_of(a[6], dev, &stream) < 0)
        return NULL;
    vnm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn_quantize(xp, ld_x, R, C, type, (int32_t)block, a[1] != Py_None ? q_type : t_type, qp, ld_q, sp, rs, cs, tp,
                     ld_t, up, trs, tcs, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* xq, x_scale, wq, w_scale, Y, bias, act, status, skip_stage (-1: none), stream -> status */
static PyObject* fp8_linear(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    Desc x, w, ws, y, b;
    int64_t dev, d2, ld_x, ld_w, ld_y, one, xrs, xcs, wrs, wcs;
    void *xp, *wp, *yp, *bp, *sp;
    float *xs, *wsp;
    vnm_fp8 x_type, w_type;
    vnm_dtype y_type, b_type = VNM_F32;
    vnm_stream_t stream;
    if (count(n, 10) < 0 || first(a[0], "xq", &x, &dev) < 0 || fp8_of(x.dtype, "xq", &x_type) < 0 ||
        describe(a[2], &w, &d2) < 0 || fp8_of(w.dtype, "wq", &w_type) < 0 || describe(a[3], &ws, &d2) < 0 ||
        describe(a[4], &y, &d2) < 0 || dtype_of(y.dtype, "Y", &y_type) < 0)
        return NULL;
    const long act = PyLong_AsLong(a[6]), skip = PyLong_AsLong(a[8]);
    if (PyErr_Occurred()) return NULL;
    const int64_t T = x.rows, K = x.cols, R = w.rows >= 0 ? w.rows : 0;
    /* the scales tell a scale a row from one for 128 rows (the same thing for one row) */
    const int32_t block = ws.rows == R ? 1 : 128;
    if (tensor(a[0], "xq", T, K, NULL, dev, &xp, &ld_x) < 0 || tensor(a[2], "wq", R, K, NULL, dev, &wp, &ld_w) < 0 ||
        tensor(a[4], "Y", T, R, NULL, dev, &yp, &ld_y) < 0 ||
        scales(a[1], "x_scale", T, groups(K), dev, &xs, &xrs, &xcs) < 0 ||
        scales(a[3], "w_scale", block == 1 ? R : groups(R), groups(K), dev, &wsp, &wrs, &wcs) < 0 ||
        tensor(a[5], "bias", -1, R, NULL, dev, &bp, &one) < 0)
        return NULL;
    if (a[5] != Py_None && (describe(a[5], &b, &d2) < 0 || dtype_of(b.dtype, "bias", &b_type) < 0)) return NULL;
    sp = NULL;
    if (a[7] != Py_None) {
        Desc s;
        if (describe(a[7], &s, &d2) < 0) return NULL;
        if (s.dtype != py_i32 || d2 != dev || s.rows != -1 || s.cols < 3) {
            PyErr_SetString(PyExc_ValueError, "status must be a CUDA int32 tensor of at least 3 words");
            return NULL;
        }
        if (address(a[7], &sp) < 0) return NULL;
    }
    if (stream_of(a[9], dev, &stream) < 0) return NULL;
    vnm_status st;
    Py_BEGIN_ALLOW_THREADS
    if (skip >= 0)
        st = fn_linear_skip(xp, ld_x, x_type, xs, xrs, xcs, wp, ld_w, w_type, wsp, wrs, wcs, block, T, R, K, bp, b_type,
                            (vnm_activation)act, yp, ld_y, y_type, sp, (int32_t)skip, stream);
    else
        st = fn_linear(xp, ld_x, x_type, xs, xrs, xcs, wp, ld_w, w_type, wsp, wrs, wcs, block, T, R, K, bp, b_type,
                       (vnm_activation)act, yp, ld_y, y_type, sp, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* T, D -> bytes of workspace of rmsnorm_backward, or minus the status */
static PyObject* rmsnorm_workspace(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    if (count(n, 2) < 0) return NULL;
    const int64_t T = PyLong_AsLongLong(a[0]), D = PyLong_AsLongLong(a[1]);
    if (PyErr_Occurred()) return NULL;
    size_t bytes = 0;
    const vnm_status st = fn_rmsnorm_workspace(T, D, &bytes);
    return PyLong_FromLongLong(st == VNM_OK ? (int64_t)bytes : -(int64_t)st);
}

/* The six functions' addresses, torch's six types, current device and current stream. */
static PyObject* setup(PyObject* self, PyObject* args) {
    unsigned long long f[6];
    PyObject *t[6], *device, *stream;
    if (!PyArg_ParseTuple(args, "(KKKKKK)(OOOOOO)OO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &t[0], &t[1], &t[2], &t[3],
                          &t[4], &t[5], &device, &stream))
        return NULL;
    fn_rmsnorm = (__typeof__(fn_rmsnorm))(uintptr_t)f[0];
    fn_rmsnorm_backward = (__typeof__(fn_rmsnorm_backward))(uintptr_t)f[1];
    fn_rmsnorm_workspace = (__typeof__(fn_rmsnorm_workspace))(uintptr_t)f[2];
    fn_quantize = (__typeof__(fn_quantize))(uintptr_t)f[3];
    fn_linear = (__typeof__(fn_linear))(uintptr_t)f[4];
    fn_linear_skip = (testing_linear_t)(uintptr_t)f[5];
    PyObject** to[8] = {&py_f16, &py_bf16, &py_f32, &py_e4m3, &py_e5m2, &py_i32, &py_current_device, &py_current_stream};
    PyObject* from[8] = {t[0], t[1], t[2], t[3], t[4], t[5], device, stream};
    for (int i = 0; i < 8; ++i) {
        Py_INCREF(from[i]);
        Py_XSETREF(*to[i], from[i]);
    }
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "Addresses of the library's functions, and torch's types and queries."},
    {"rmsnorm", (PyCFunction)(void (*)(void))rmsnorm, METH_FASTCALL, "vnm_rmsnorm"},
    {"rmsnorm_backward", (PyCFunction)(void (*)(void))rmsnorm_backward, METH_FASTCALL, "vnm_rmsnorm_backward"},
    {"rmsnorm_workspace", (PyCFunction)(void (*)(void))rmsnorm_workspace, METH_FASTCALL, "vnm_rmsnorm_backward_workspace_size"},
    {"fp8_quantize", (PyCFunction)(void (*)(void))fp8_quantize, METH_FASTCALL, "vnm_fp8_quantize"},
    {"fp8_linear", (PyCFunction)(void (*)(void))fp8_linear, METH_FASTCALL, "vnm_fp8_linear"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_vnm_binding", "Argument marshalling for libvnm.", -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__vnm_binding(void) {
    s_shape = PyUnicode_InternFromString("shape");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!s_shape || !s_dtype || !s_get_device || !s_stride || !s_data_ptr || !s_cuda_stream) return NULL;
    return PyModule_Create(&module);
}
