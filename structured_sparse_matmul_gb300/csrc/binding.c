/*
 * Argument marshalling of the norm, 8-bit quantiser and 8-bit Linear layer for
 * Python: torch tensors to the C ABI of include/vnm.h.
 *
 * These calls stand in decode loops, where one takes a few microseconds on the
 * GPU. Reading a tensor's shape, type, device, strides and address from Python
 * and passing two dozen arguments through ctypes costs 7 us a call; the same reads
 * from C cost 2, each attribute read once. Nothing is computed here: every check
 * is of a tensor's description, and the functions called are the library's
 * exported ones, whose addresses setup() is given.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <string.h>

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
typedef vnm_status (*testing_linear_no_status_t)(const void*, int64_t, vnm_fp8, const float*, int64_t, int64_t, const void*,
                                                 int64_t, vnm_fp8, const float*, int64_t, int64_t, int32_t, int64_t, int64_t,
                                                 int64_t, void*, int64_t, vnm_dtype, int32_t, vnm_stream_t);
static testing_linear_no_status_t fn_linear_skip_no_status;

static PyObject *py_f16, *py_f32, *py_bf16, *py_e4m3, *py_e5m2, *py_i32; /* torch dtypes */
static PyObject *py_current_device, *py_current_stream;
static PyObject *s_shape, *s_dtype, *s_get_device, *s_stride, *s_data_ptr, *s_cuda_stream, *s_nbytes;

/* A tensor's description, each attribute read once; dims = -1 for None. */
typedef struct {
    PyObject* object;   /* borrowed from the call's arguments */
    PyObject* dtype;    /* borrowed: torch's dtype objects live for good */
    Py_ssize_t dims;
    int64_t size[2], stride[2], device;
    void* p;
} Tensor;

static int long_of(PyObject* o, int64_t* out) { /* steals o */
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

static int read_tensor(PyObject* o, Tensor* t) {
    memset(t, 0, sizeof(*t));
    t->object = o;
    t->dims = -1;
    t->device = -1;
    if (o == Py_None) return 0;
    Py_ssize_t strides;
    int64_t address;
    if (ints_of(PyObject_GetAttr(o, s_shape), t->size, &t->dims) < 0 ||
        ints_of(PyObject_CallMethodNoArgs(o, s_stride), t->stride, &strides) < 0 ||
        long_of(PyObject_CallMethodNoArgs(o, s_get_device), &t->device) < 0 ||
        long_of(PyObject_CallMethodNoArgs(o, s_data_ptr), &address) < 0)
        return -1;
    t->dtype = PyObject_GetAttr(o, s_dtype);
    if (t->dtype == NULL) return -1;
    Py_DECREF(t->dtype);
    t->p = (void*)(intptr_t)address;
    return 0;
}

static int read_all(PyObject* const* o, const int* which, int n, Tensor* t) {
    for (int i = 0; i < n; ++i)
        if (read_tensor(o[which[i]], &t[i]) < 0) return -1;
    return 0;
}

static int refuse(const Tensor* t, const char* name, int64_t rows, int64_t cols, PyObject* dtype, int64_t device) {
    PyObject* shape = PyObject_GetAttr(t->object, s_shape);
    PyObject* want = dtype ? PyObject_Str(dtype) : PyUnicode_FromString("any type served");
    if (shape && want) {
        if (rows >= 0)
            PyErr_Format(PyExc_ValueError, "%s must be a row-major tensor of shape (%lld, %lld), %U, on cuda:%lld; got %S, %S", name,
                         (long long)rows, (long long)cols, want, (long long)device, shape, t->dtype);
        else
            PyErr_Format(PyExc_ValueError, "%s must be a contiguous tensor of shape (%lld,), %U, on cuda:%lld; got %S, %S", name,
                         (long long)cols, want, (long long)device, shape, t->dtype);
    }
    Py_XDECREF(shape);
    Py_XDECREF(want);
    return -1;
}

/* Row-major rows x cols, of a type or (dtype NULL) any; *ld its leading dimension (1 for None). */
static int matrix(const Tensor* t, const char* name, int64_t rows, int64_t cols, PyObject* dtype, int64_t device, int64_t* ld) {
    *ld = 1;
    if (t->dims < 0) return 0;
    if (t->dims != 2 || t->size[0] != rows || t->size[1] != cols || t->device != device ||
        (dtype != NULL && t->dtype != dtype) || (cols > 1 && t->stride[1] != 1))
        return refuse(t, name, rows, cols, dtype, device);
    /* Rows that overlap (an expanded tensor's) have no leading dimension; one row may carry any stride. */
    const int64_t least = cols > 0 ? cols : 1;
    if (rows > 1 && cols > 0 && t->stride[0] < least) return refuse(t, name, rows, cols, dtype, device);
    *ld = t->stride[0] >= least ? t->stride[0] : least;
    return 0;
}

/* A contiguous vector. */
static int vector(const Tensor* t, const char* name, int64_t n, PyObject* dtype, int64_t device) {
    if (t->dims < 0) return 0;
    if (t->dims != 1 || t->size[0] != n || t->device != device || (dtype != NULL && t->dtype != dtype) ||
        (n > 1 && t->stride[0] != 1))
        return refuse(t, name, -1, n, dtype, device);
    return 0;
}

/* fp32 scales of any strides. */
static int scales(const Tensor* t, const char* name, int64_t rows, int64_t cols, int64_t device) {
    if (t->dims < 0) return 0;
    if (t->dims != 2 || t->size[0] != rows || t->size[1] != cols || t->device != device || t->dtype != py_f32)
        return refuse(t, name, rows, cols, py_f32, device);
    return 0;
}

static int dtype_of(const Tensor* t, const char* name, vnm_dtype* out) {
    if (t->dims >= 0 && t->dtype == py_f16)
        *out = VNM_F16;
    else if (t->dims >= 0 && t->dtype == py_bf16)
        *out = VNM_BF16;
    else if (t->dims >= 0 && t->dtype == py_f32)
        *out = VNM_F32;
    else {
        PyErr_Format(PyExc_ValueError, "%s must be fp16, bf16 or fp32", name);
        return -1;
    }
    return 0;
}

static int fp8_of(const Tensor* t, const char* name, vnm_fp8* out) {
    if (t->dims >= 0 && t->dtype == py_e4m3)
        *out = VNM_E4M3;
    else if (t->dims >= 0 && t->dtype == py_e5m2)
        *out = VNM_E5M2;
    else {
        PyErr_Format(PyExc_ValueError, "%s must be float8_e4m3fn or float8_e5m2", name);
        return -1;
    }
    return 0;
}

/* The call's first tensor: a matrix on the current CUDA device. */
static int first(const Tensor* t, const char* name) {
    int64_t cur;
    if (t->dims != 2 || t->device < 0) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA matrix", name);
        return -1;
    }
    if (long_of(PyObject_CallNoArgs(py_current_device), &cur) < 0) return -1;
    if (cur != t->device) {
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

/* A number of the C ABI's 32 bits; -1, which every such argument refuses, for one that does not fit. */
static int32_t narrow(long v) { return v >= INT32_MIN && v <= INT32_MAX ? (int32_t)v : -1; }

static int64_t groups(int64_t n) { return (n + 127) / 128; }

static int count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return 0;
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return -1;
}

/* x, weight, eps, residual, h, y, rstd, q, q_scale, stream -> status */
static PyObject* rmsnorm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    static const int which[8] = {0, 1, 3, 4, 5, 6, 7, 8};
    Tensor t[8];
    const Tensor *x = &t[0], *w = &t[1], *r = &t[2], *h = &t[3], *y = &t[4], *rstd = &t[5], *q = &t[6], *s = &t[7];
    int64_t ld_x, ld_r, ld_h, ld_y, ld_q;
    vnm_dtype type;
    vnm_fp8 q_type = VNM_E4M3;
    vnm_stream_t stream;
    if (count(n, 10) < 0 || read_all(a, which, 8, t) < 0 || first(x, "x") < 0 || dtype_of(x, "x", &type) < 0) return NULL;
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) return NULL;
    const int64_t T = x->size[0], D = x->size[1], dev = x->device;
    if (matrix(x, "x", T, D, NULL, dev, &ld_x) < 0 || vector(w, "weight", D, x->dtype, dev) < 0 ||
        matrix(r, "residual", T, D, x->dtype, dev, &ld_r) < 0 || matrix(h, "h", T, D, x->dtype, dev, &ld_h) < 0 ||
        matrix(y, "y", T, D, x->dtype, dev, &ld_y) < 0 || vector(rstd, "rstd", T, py_f32, dev) < 0 ||
        matrix(q, "q", T, D, NULL, dev, &ld_q) < 0 || scales(s, "q_scale", T, groups(D), dev) < 0 ||
        (q->dims >= 0 && fp8_of(q, "q", &q_type) < 0) || stream_of(a[9], dev, &stream) < 0)
        return NULL;
    vnm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn_rmsnorm(x->p, ld_x, r->p, ld_r, w->p, (float)eps, T, D, type, h->p, ld_h, y->p, ld_y, rstd->p, q->p, ld_q, q_type,
                    s->p, s->stride[0], s->stride[1], stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* dy, h, weight, rstd, dh, dweight, dresidual, workspace, stream -> status */
static PyObject* rmsnorm_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    static const int which[8] = {0, 1, 2, 3, 4, 5, 6, 7};
    Tensor t[8];
    const Tensor *dy = &t[0], *h = &t[1], *w = &t[2], *rstd = &t[3], *dh = &t[4], *dw = &t[5], *dr = &t[6], *ws = &t[7];
    int64_t ld_dy, ld_h, ld_r, ld_o, bytes = 0;
    vnm_dtype type;
    vnm_stream_t stream;
    if (count(n, 9) < 0 || read_all(a, which, 8, t) < 0 || first(dy, "dy") < 0 || dtype_of(dy, "dy", &type) < 0) return NULL;
    const int64_t T = dy->size[0], D = dy->size[1], dev = dy->device;
    if (matrix(dy, "dy", T, D, NULL, dev, &ld_dy) < 0 || matrix(h, "h", T, D, dy->dtype, dev, &ld_h) < 0 ||
        vector(w, "weight", D, dy->dtype, dev) < 0 || vector(rstd, "rstd", T, py_f32, dev) < 0 ||
        matrix(dh, "dh", T, D, dy->dtype, dev, &ld_o) < 0 || vector(dw, "dweight", D, py_f32, dev) < 0 ||
        matrix(dr, "dresidual", T, D, dy->dtype, dev, &ld_r) < 0)
        return NULL;
    if (ws->dims >= 0) {
        if (ws->device != dev || ws->dims != 1 || (ws->size[0] > 1 && ws->stride[0] != 1)) {
            PyErr_SetString(PyExc_ValueError, "workspace must be a contiguous vector on dy's device");
            return NULL;
        }
        if (long_of(PyObject_GetAttr(ws->object, s_nbytes), &bytes) < 0) return NULL;
    }
    if (stream_of(a[8], dev, &stream) < 0) return NULL;
    vnm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn_rmsnorm_backward(dy->p, ld_dy, h->p, ld_h, w->p, rstd->p, dr->p, ld_r, T, D, type, dh->p, ld_o, dw->p, ws->p,
                             (size_t)bytes, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* X, q, s, qt, st, block_rows, stream -> status */
static PyObject* fp8_quantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    static const int which[5] = {0, 1, 2, 3, 4};
    Tensor t[5];
    const Tensor *x = &t[0], *q = &t[1], *s = &t[2], *qt = &t[3], *u = &t[4];
    int64_t ld_x, ld_q, ld_t;
    vnm_dtype type;
    vnm_fp8 q_type = VNM_E4M3, t_type = VNM_E4M3;
    vnm_stream_t stream;
    if (count(n, 7) < 0 || read_all(a, which, 5, t) < 0 || first(x, "X") < 0 || dtype_of(x, "X", &type) < 0) return NULL;
    const long block = PyLong_AsLong(a[5]);
    if (block == -1 && PyErr_Occurred()) return NULL;
    const int64_t R = x->size[0], C = x->size[1], dev = x->device, per = block > 0 ? block : 1;
    if ((q->dims >= 0 && fp8_of(q, "q", &q_type) < 0) || (qt->dims >= 0 && fp8_of(qt, "qt", &t_type) < 0)) return NULL;
    if (q->dims >= 0 && qt->dims >= 0 && q_type != t_type) {
        PyErr_SetString(PyExc_ValueError, "q and qt must have the same type");
        return NULL;
    }
    if (matrix(x, "X", R, C, NULL, dev, &ld_x) < 0 || matrix(q, "q", R, C, NULL, dev, &ld_q) < 0 ||
        scales(s, "s", (R + per - 1) / per, groups(C), dev) < 0 || matrix(qt, "qt", C, R, NULL, dev, &ld_t) < 0 ||
        scales(u, "st", (C + per - 1) / per, groups(R), dev) < 0 || stream_of(a[6], dev, &stream) < 0)
        return NULL;
    vnm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn_quantize(x->p, ld_x, R, C, type, narrow(block), q->dims >= 0 ? q_type : t_type, q->p, ld_q, s->p, s->stride[0],
                     s->stride[1], qt->p, ld_t, u->p, u->stride[0], u->stride[1], stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* xq, x_scale, wq, w_scale, Y, bias, act, status, skip_stage (-1: none), stream -> status */
static PyObject* fp8_linear(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    static const int which[7] = {0, 1, 2, 3, 4, 5, 7};
    Tensor t[7];
    const Tensor *x = &t[0], *xs = &t[1], *w = &t[2], *ws = &t[3], *y = &t[4], *b = &t[5], *status = &t[6];
    int64_t ld_x, ld_w, ld_y;
    vnm_fp8 x_type, w_type;
    vnm_dtype y_type, b_type = VNM_F32;
    vnm_stream_t stream;
    if (count(n, 10) < 0 || read_all(a, which, 7, t) < 0 || first(x, "xq") < 0 || fp8_of(x, "xq", &x_type) < 0 ||
        fp8_of(w, "wq", &w_type) < 0 || dtype_of(y, "Y", &y_type) < 0)
        return NULL;
    const long act = PyLong_AsLong(a[6]), skip = PyLong_AsLong(a[8]);
    if (PyErr_Occurred()) return NULL;
    const int64_t T = x->size[0], K = x->size[1], R = w->size[0], dev = x->device;
    /* the scales tell a scale a row from one for 128 rows (the same thing for one row) */
    const int32_t block = ws->dims == 2 && ws->size[0] == R ? 1 : 128;
    if (matrix(x, "xq", T, K, NULL, dev, &ld_x) < 0 || matrix(w, "wq", R, K, NULL, dev, &ld_w) < 0 ||
        matrix(y, "Y", T, R, NULL, dev, &ld_y) < 0 || scales(xs, "x_scale", T, groups(K), dev) < 0 ||
        scales(ws, "w_scale", block == 1 ? R : groups(R), groups(K), dev) < 0 || vector(b, "bias", R, NULL, dev) < 0 ||
        (b->dims >= 0 && dtype_of(b, "bias", &b_type) < 0))
        return NULL;
    if (status->dims >= 0 && (status->dtype != py_i32 || status->device != dev || status->dims != 1 || status->size[0] < 3 ||
                              status->stride[0] != 1)) {
        PyErr_SetString(PyExc_ValueError, "status must be a CUDA int32 tensor of at least 3 words");
        return NULL;
    }
    if (stream_of(a[9], dev, &stream) < 0) return NULL;
    vnm_status st;
    Py_BEGIN_ALLOW_THREADS
    if (skip >= 0 && status->dims < 0)
        st = fn_linear_skip_no_status(x->p, ld_x, x_type, xs->p, xs->stride[0], xs->stride[1], w->p, ld_w, w_type, ws->p,
                                      ws->stride[0], ws->stride[1], block, T, R, K, y->p, ld_y, y_type, narrow(skip), stream);
    else if (skip >= 0)
        st = fn_linear_skip(x->p, ld_x, x_type, xs->p, xs->stride[0], xs->stride[1], w->p, ld_w, w_type, ws->p, ws->stride[0],
                            ws->stride[1], block, T, R, K, b->p, b_type, (vnm_activation)narrow(act), y->p, ld_y, y_type, status->p,
                            narrow(skip), stream);
    else
        st = fn_linear(x->p, ld_x, x_type, xs->p, xs->stride[0], xs->stride[1], w->p, ld_w, w_type, ws->p, ws->stride[0],
                       ws->stride[1], block, T, R, K, b->p, b_type, (vnm_activation)narrow(act), y->p, ld_y, y_type, status->p, stream);
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

/* The seven functions' addresses, torch's six types, current device and current stream. */
static PyObject* setup(PyObject* self, PyObject* args) {
    unsigned long long f[7];
    PyObject *t[6], *device, *stream;
    if (!PyArg_ParseTuple(args, "(KKKKKKK)(OOOOOO)OO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &t[0], &t[1], &t[2], &t[3],
                          &t[4], &t[5], &device, &stream))
        return NULL;
    fn_rmsnorm = (__typeof__(fn_rmsnorm))(uintptr_t)f[0];
    fn_rmsnorm_backward = (__typeof__(fn_rmsnorm_backward))(uintptr_t)f[1];
    fn_rmsnorm_workspace = (__typeof__(fn_rmsnorm_workspace))(uintptr_t)f[2];
    fn_quantize = (__typeof__(fn_quantize))(uintptr_t)f[3];
    fn_linear = (__typeof__(fn_linear))(uintptr_t)f[4];
    fn_linear_skip = (testing_linear_t)(uintptr_t)f[5];
    fn_linear_skip_no_status = (testing_linear_no_status_t)(uintptr_t)f[6];
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
    s_nbytes = PyUnicode_InternFromString("nbytes");
    if (!s_shape || !s_dtype || !s_get_device || !s_stride || !s_data_ptr || !s_cuda_stream || !s_nbytes) return NULL;
    return PyModule_Create(&module);
}
