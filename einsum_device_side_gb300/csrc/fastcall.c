/*
 * fastcall.c -- CPython binding of the hot entry points of include/tropical.h.
 *
 * Argument marshalling only: each function takes plain Python integers
 * (device addresses, extents, strides, dtype and semiring codes, the stream
 * handle) and tuples of them, fills the C descriptors and calls the C ABI,
 * returning its status code.  It exists because a ctypes call converting
 * twenty arguments costs about 2 us of host time per call, more than the
 * library's own planning; the vectorcall convention (METH_FASTCALL) used here
 * passes the arguments without building a tuple.  No torch type crosses it.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <string.h>

#include "tropical.h"

/* a Python int (or None = 0) as a pointer-sized integer */
static int as_ptr(PyObject* o, void** out)
{
    if (o == Py_None) {
        *out = NULL;
        return 0;
    }
    *out = PyLong_AsVoidPtr(o);
    return (*out == NULL && PyErr_Occurred()) ? -1 : 0;
}

static int as_i64(PyObject* o, int64_t* out)
{
    *out = (int64_t)PyLong_AsLongLong(o);
    return (*out == -1 && PyErr_Occurred()) ? -1 : 0;
}

/* descriptor from (address, dtype code, shape tuple, stride tuple) */
static int fill_tensor(trop_tensor* t, PyObject* ptr, PyObject* dtype, PyObject* shape, PyObject* stride)
{
    if (!PyTuple_Check(shape) || !PyTuple_Check(stride)) {
        PyErr_SetString(PyExc_TypeError, "shape and stride must be tuples");
        return -1;
    }
    const Py_ssize_t n = PyTuple_GET_SIZE(shape);
    if (n > TROP_MAX_RANK || PyTuple_GET_SIZE(stride) != n) {
        PyErr_SetString(PyExc_ValueError, "rank above 32 or shape/stride lengths differ");
        return -1;
    }
    if (as_ptr(ptr, &t->data) < 0) return -1;
    const long dt = PyLong_AsLong(dtype);
    if (dt == -1 && PyErr_Occurred()) return -1;
    t->dtype = (int32_t)dt;
    t->rank = (int32_t)n;
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (as_i64(PyTuple_GET_ITEM(shape, i), &t->shape[i]) < 0) return -1;
        if (as_i64(PyTuple_GET_ITEM(stride, i), &t->stride[i]) < 0) return -1;
    }
    return 0;
}

static int check_nargs(Py_ssize_t nargs, Py_ssize_t want, const char* name)
{
    if (nargs == want) return 0;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name, want, nargs);
    return -1;
}

/* Every tensor is passed as four arguments: address (int or None), dtype code, shape tuple,
 * stride tuple (elements). */

/* permute_trace(in x4, spec: bytes, semiring, out x4, argmax_ptr, stream, no_alloc) -> status */
static PyObject* fc_permute_trace(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 13, "permute_trace") < 0) return NULL;
    trop_tensor in, out;
    void *argmax, *stream;
    if (fill_tensor(&in, a[0], a[1], a[2], a[3]) < 0 || fill_tensor(&out, a[6], a[7], a[8], a[9]) < 0 ||
        as_ptr(a[10], &argmax) < 0 || as_ptr(a[11], &stream) < 0)
        return NULL;
    const char* spec = PyBytes_AsString(a[4]);
    const long sr = PyLong_AsLong(a[5]);
    const int no_alloc = PyObject_IsTrue(a[12]);
    if (!spec || (sr == -1 && PyErr_Occurred()) || no_alloc < 0) return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = no_alloc ? tropical_permute_trace_noalloc(&in, spec, (int)sr, &out, (int32_t*)argmax, stream)
                  : tropical_permute_trace(&in, spec, (int)sr, &out, (int32_t*)argmax, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* permute_pair(val_in x4, arg_in x4, spec: bytes, val_out x4, arg_out x4, stream) -> status */
static PyObject* fc_permute_pair(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 18, "permute_pair") < 0) return NULL;
    trop_tensor vi, ai, vo, ao;
    void* stream;
    if (fill_tensor(&vi, a[0], a[1], a[2], a[3]) < 0 || fill_tensor(&ai, a[4], a[5], a[6], a[7]) < 0 ||
        fill_tensor(&vo, a[9], a[10], a[11], a[12]) < 0 || fill_tensor(&ao, a[13], a[14], a[15], a[16]) < 0 ||
        as_ptr(a[17], &stream) < 0)
        return NULL;
    const char* spec = PyBytes_AsString(a[8]);
    if (!spec) return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = tropical_permute_pair(&vi, &ai, spec, &vo, &ao, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* gemm(semiring, dtype, batch, M, N, K, A, sAb, sAm, sAk, B, sBb, sBk, sBn, C, sCb, sCm, sCn,
 *      argmax, stream): the twenty arguments of tropical_gemm_strided_batched_argmax */
static PyObject* fc_gemm(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 20, "gemm") < 0) return NULL;
    int64_t v[20];
    void* p[20];
    for (int i = 0; i < 20; ++i) {
        const int is_ptr = i == 6 || i == 10 || i == 14 || i == 18 || i == 19;
        if (is_ptr ? as_ptr(a[i], &p[i]) < 0 : as_i64(a[i], &v[i]) < 0) return NULL;
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = tropical_gemm_strided_batched_argmax((int)v[0], (int)v[1], v[2], v[3], v[4], v[5], p[6], v[7], v[8], v[9],
                                              p[10], v[11], v[12], v[13], p[14], v[15], v[16], v[17],
                                              (int32_t*)p[18], p[19]);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* einsum(spec: bytes, A x4, B x4, semiring, out x4, argmax_ptr, stream) -> status */
static PyObject* fc_einsum(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 16, "einsum") < 0) return NULL;
    trop_tensor A, B, out;
    void *argmax, *stream;
    if (fill_tensor(&A, a[1], a[2], a[3], a[4]) < 0 || fill_tensor(&B, a[5], a[6], a[7], a[8]) < 0 ||
        fill_tensor(&out, a[10], a[11], a[12], a[13]) < 0 || as_ptr(a[14], &argmax) < 0 ||
        as_ptr(a[15], &stream) < 0)
        return NULL;
    const char* spec = PyBytes_AsString(a[0]);
    const long sr = PyLong_AsLong(a[9]);
    if (!spec || (sr == -1 && PyErr_Occurred())) return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = tropical_einsum_pairwise(spec, &A, &B, (int)sr, &out, (int32_t*)argmax, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* ---- tensor-taking variants: the same calls, reading each tensor's data_ptr(), dtype, shape and
 * stride() through the C API (the tensors are treated as plain Python objects with those
 * attributes), so the Python wrapper does no per-argument work.  set_torch_handles() gives the
 * dtype objects (matched by identity: float32, int32, int64, float64, bfloat16, float16 -> the
 * trop_dtype codes) and the function returning a device's current raw stream. */
#define N_DTYPES 8       /* f32, i32, i64, f64, bf16, f16, i8, u8: the trop_dtype codes */
#define N_TROPICAL 4     /* the ones that the tropical operations know */
static PyObject* g_dtype_obj[N_DTYPES];
static PyObject* g_raw_stream;
static PyObject *s_data_ptr, *s_shape, *s_stride, *s_dtype, *s_get_device, *s_cuda_stream;

static PyObject* fc_set_torch_handles(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, N_DTYPES + 1, "set_torch_handles") < 0) return NULL;
    for (int i = 0; i < N_DTYPES; ++i) {
        Py_XDECREF(g_dtype_obj[i]);
        Py_INCREF(a[i]);
        g_dtype_obj[i] = a[i];
    }
    Py_XDECREF(g_raw_stream);
    Py_INCREF(a[N_DTYPES]);
    g_raw_stream = a[N_DTYPES];
    Py_RETURN_NONE;
}

/* the descriptor of a tensor object whose dtype is one of the first n_dtypes */
static int obj_tensor_of(trop_tensor* t, PyObject* obj, int n_dtypes)
{
    PyObject* p = PyObject_CallMethodNoArgs(obj, s_data_ptr);
    if (!p) return -1;
    const int bad = as_ptr(p, &t->data) < 0;
    Py_DECREF(p);
    if (bad) return -1;
    PyObject* dt = PyObject_GetAttr(obj, s_dtype);
    if (!dt) return -1;
    t->dtype = -1;  /* unknown dtypes reach the C ABI as -1, which it refuses */
    for (int i = 0; i < n_dtypes; ++i)
        if (dt == g_dtype_obj[i]) t->dtype = i;
    Py_DECREF(dt);
    PyObject* shape = PyObject_GetAttr(obj, s_shape);
    if (!shape) return -1;
    PyObject* stride = PyObject_CallMethodNoArgs(obj, s_stride);
    if (!stride) {
        Py_DECREF(shape);
        return -1;
    }
    int rc = 0;
    const Py_ssize_t n = PyTuple_Check(shape) && PyTuple_Check(stride) ? PyTuple_GET_SIZE(shape) : -1;
    if (n < 0 || n > TROP_MAX_RANK || PyTuple_GET_SIZE(stride) != n) {
        PyErr_SetString(PyExc_ValueError, "tensor rank above 32 or unreadable shape/stride");
        rc = -1;
    } else {
        t->rank = (int32_t)n;
        for (Py_ssize_t i = 0; i < n && rc == 0; ++i)
            if (as_i64(PyTuple_GET_ITEM(shape, i), &t->shape[i]) < 0 || as_i64(PyTuple_GET_ITEM(stride, i), &t->stride[i]) < 0)
                rc = -1;
    }
    Py_DECREF(shape);
    Py_DECREF(stride);
    return rc;
}

static int obj_tensor(trop_tensor* t, PyObject* obj) { return obj_tensor_of(t, obj, N_TROPICAL); }

/* the stream handle: stream.cuda_stream, or the current raw stream of obj's device */
static int obj_stream(PyObject* stream, PyObject* obj, void** out)
{
    PyObject* h;
    if (stream != Py_None) {
        h = PyObject_GetAttr(stream, s_cuda_stream);
    } else {
        if (!g_raw_stream) {
            PyErr_SetString(PyExc_RuntimeError, "set_torch_handles was not called");
            return -1;
        }
        PyObject* dev = PyObject_CallMethodNoArgs(obj, s_get_device);
        if (!dev) return -1;
        h = PyObject_CallOneArg(g_raw_stream, dev);
        Py_DECREF(dev);
    }
    if (!h) return -1;
    const int rc = as_ptr(h, out);
    Py_DECREF(h);
    return rc;
}

static int obj_semiring(PyObject* o, long* sr)
{
    if (PyUnicode_Check(o)) {
        *sr = PyUnicode_CompareWithASCIIString(o, "maxplus") == 0    ? 0
              : PyUnicode_CompareWithASCIIString(o, "minplus") == 0  ? 1
              : PyUnicode_CompareWithASCIIString(o, "maxtimes") == 0 ? 2
                                                                      : -1;
        if (*sr < 0) {
            PyErr_SetString(PyExc_KeyError, "semiring must be 'maxplus', 'minplus' or 'maxtimes'");
            return -1;
        }
        return 0;
    }
    *sr = PyLong_AsLong(o);
    return (*sr == -1 && PyErr_Occurred()) ? -1 : 0;
}

/* permute_trace_t(x, spec: str, semiring, out, argmax tensor or None, stream or None, no_alloc) */
static PyObject* fc_permute_trace_t(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 7, "permute_trace_t") < 0) return NULL;
    trop_tensor in, out;
    void *argmax = NULL, *stream;
    long sr;
    if (obj_tensor(&in, a[0]) < 0 || obj_tensor(&out, a[3]) < 0 || obj_semiring(a[2], &sr) < 0 ||
        obj_stream(a[5], a[0], &stream) < 0)
        return NULL;
    if (a[4] != Py_None) {
        PyObject* p = PyObject_CallMethodNoArgs(a[4], s_data_ptr);
        if (!p) return NULL;
        const int bad = as_ptr(p, &argmax) < 0;
        Py_DECREF(p);
        if (bad) return NULL;
    }
    const char* spec = PyUnicode_AsUTF8(a[1]);
    const int no_alloc = PyObject_IsTrue(a[6]);
    if (!spec || no_alloc < 0) return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = no_alloc ? tropical_permute_trace_noalloc(&in, spec, (int)sr, &out, (int32_t*)argmax, stream)
                  : tropical_permute_trace(&in, spec, (int)sr, &out, (int32_t*)argmax, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* permute_pair_t(val, arg, spec: str, out_val, out_arg, stream or None) */
static PyObject* fc_permute_pair_t(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 6, "permute_pair_t") < 0) return NULL;
    trop_tensor vi, ai, vo, ao;
    void* stream;
    if (obj_tensor(&vi, a[0]) < 0 || obj_tensor(&ai, a[1]) < 0 || obj_tensor(&vo, a[3]) < 0 ||
        obj_tensor(&ao, a[4]) < 0 || obj_stream(a[5], a[0], &stream) < 0)
        return NULL;
    const char* spec = PyUnicode_AsUTF8(a[2]);
    if (!spec) return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = tropical_permute_pair(&vi, &ai, spec, &vo, &ao, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* ---- training operators.  Tensors as objects; "or None" leaves one out. */

/* address of a tensor object, NULL for None */
static int obj_ptr(PyObject* obj, void** out)
{
    *out = NULL;
    if (obj == Py_None) return 0;
    PyObject* p = PyObject_CallMethodNoArgs(obj, s_data_ptr);
    if (!p) return -1;
    const int bad = as_ptr(p, out) < 0;
    Py_DECREF(p);
    return bad ? -1 : 0;
}
static int as_double(PyObject* o, double* out)
{
    *out = PyFloat_AsDouble(o);
    return (*out == -1.0 && PyErr_Occurred()) ? -1 : 0;
}

/* The device number of a tensor object, -1 for the host's; -2 on error. */
static long obj_device(PyObject* obj)
{
    PyObject* d = PyObject_CallMethodNoArgs(obj, s_get_device);
    if (!d) return -2;
    const long v = PyLong_AsLong(d);
    Py_DECREF(d);
    return v == -1 && PyErr_Occurred() ? -2 : v;
}

/* A function below that is given something out of the ordinary (a vector that is strided, of another
 * length or type, on another device) returns PLAIN_PATH and launches nothing: the Python wrapper
 * then checks every argument by itself and says which it was. */
#define PLAIN_PATH 1

/* A vector of n contiguous elements of `dtype` on `device`, or None: 0 with its address, PLAIN_PATH, or -1. */
static int obj_vector(PyObject* obj, int64_t n, int32_t dtype, long device, void** out)
{
    *out = NULL;
    if (obj == Py_None) return 0;
    trop_tensor t;
    if (obj_tensor_of(&t, obj, N_DTYPES) < 0) return -1;
    const long d = obj_device(obj);
    if (d == -2) return -1;
    int64_t count = 1;
    for (int i = t.rank - 1; i >= 0; --i) {
        if (t.shape[i] != 1 && t.stride[i] != count) return PLAIN_PATH;
        count *= t.shape[i];
    }
    *out = t.data;
    return count == n && t.dtype == dtype && d == device ? 0 : PLAIN_PATH;
}
#define VECTOR(obj, n, dtype, out)                                        \
    do {                                                                  \
        const int v_ = obj_vector((obj), (n), (dtype), device, (out));    \
        if (v_ < 0) return NULL;                                          \
        if (v_ > 0) return PyLong_FromLong(PLAIN_PATH);                   \
    } while (0)

/* [..., C] as a matrix: the leading axes merged where they make one stride, else PLAIN_PATH. */
static int as_rows(trop_tensor* t)
{
    if (t->rank == 2) return 0;
    if (t->rank < 2) return PLAIN_PATH;
    int64_t rows = 1, stride = 0;
    for (int i = t->rank - 2; i >= 0; --i) {
        if (t->shape[i] == 1) continue;
        if (t->shape[i] == 0) return PLAIN_PATH;
        if (rows > 1 && t->stride[i] != rows * stride) return PLAIN_PATH;
        if (rows == 1) stride = t->stride[i];
        rows *= t->shape[i];
    }
    const int64_t c = t->shape[t->rank - 1], sc = t->stride[t->rank - 1];
    t->shape[0] = rows;
    t->stride[0] = rows > 1 ? stride : c;
    t->shape[1] = c;
    t->stride[1] = sc;
    t->rank = 2;
    return 0;
}
static int32_t dtype_or(PyObject* obj, int32_t other)
{
    if (obj == Py_None) return other;
    PyObject* dt = PyObject_GetAttr(obj, s_dtype);
    if (!dt) return -2;
    int32_t code = -1;
    for (int i = 0; i < N_DTYPES; ++i)
        if (dt == g_dtype_obj[i]) code = i;
    Py_DECREF(dt);
    return code;
}

/* Results allocated here rather than in the Python wrapper, which saves its interpreter several us per
 * call: torch.empty(n, dtype=, device=) and torch.empty_like(t), by the handles set_torch_allocators
 * was given. */
static PyObject *g_empty, *g_empty_like, *g_f32, *g_empty_kw, *s_device;

static PyObject* fc_set_torch_allocators(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 3, "set_torch_allocators") < 0) return NULL;
    if (!g_empty_kw) g_empty_kw = Py_BuildValue("(ss)", "dtype", "device");
    if (!g_empty_kw) return NULL;
    PyObject** to[3] = {&g_empty, &g_empty_like, &g_f32};
    for (int i = 0; i < 3; ++i) {
        Py_INCREF(a[i]);
        Py_XSETREF(*to[i], a[i]);
    }
    Py_RETURN_NONE;
}
/* an uninitialised vector of n elements beside `like` */
static PyObject* new_vector(int64_t n, PyObject* dtype, PyObject* like)
{
    PyObject* size = PyLong_FromLongLong((long long)n);
    PyObject* device = size ? PyObject_GetAttr(like, s_device) : NULL;
    PyObject* r = NULL;
    if (device) {
        PyObject* args[3] = {size, dtype, device};
        r = PyObject_Vectorcall(g_empty, args, 1, g_empty_kw);
    }
    Py_XDECREF(size);
    Py_XDECREF(device);
    return r;
}
/* an uninitialised f32 scalar beside `like` */
static PyObject* new_scalar(PyObject* like)
{
    PyObject* size = PyTuple_New(0);
    PyObject* device = size ? PyObject_GetAttr(like, s_device) : NULL;
    PyObject* r = NULL;
    if (device) {
        PyObject* args[3] = {size, g_f32, device};
        r = PyObject_Vectorcall(g_empty, args, 1, g_empty_kw);
    }
    Py_XDECREF(size);
    Py_XDECREF(device);
    return r;
}
/* data pointer of a tensor made here */
static int fresh_ptr(PyObject* t, void** out) { return t ? obj_ptr(t, out) : -1; }

/* layer_norm(x, weight or None, bias or None, eps, stream or None) -> (y, mean, rstd) of a matrix x,
 * or a status: PLAIN_PATH or an error code */
static PyObject* fc_layer_norm(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 5, "layer_norm") < 0) return NULL;
    trop_tensor x, y;
    void *w, *b, *mean, *rstd, *stream;
    double eps;
    if (obj_tensor_of(&x, a[0], N_DTYPES) < 0 || as_double(a[3], &eps) < 0 || obj_stream(a[4], a[0], &stream) < 0) return NULL;
    if (!g_empty || x.rank != 2 || x.dtype < 0) return PyLong_FromLong(PLAIN_PATH);
    const long device = obj_device(a[0]);
    const int32_t wdtype = dtype_or(a[1] != Py_None ? a[1] : a[2], x.dtype);
    if (device == -2 || wdtype == -2) return NULL;
    if (device < 0) return PyLong_FromLong(PLAIN_PATH);
    VECTOR(a[1], x.shape[1], wdtype, &w);
    VECTOR(a[2], x.shape[1], wdtype, &b);
    PyObject* oy = PyObject_CallOneArg(g_empty_like, a[0]);
    PyObject* om = oy ? new_vector(x.shape[0], g_f32, a[0]) : NULL;
    PyObject* orr = om ? PyObject_CallOneArg(g_empty_like, om) : NULL;
    PyObject* out = NULL;
    if (orr && obj_tensor_of(&y, oy, N_DTYPES) == 0 && fresh_ptr(om, &mean) == 0 && fresh_ptr(orr, &rstd) == 0) {
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = tropical_layer_norm(&x, w, b, wdtype, eps, &y, (float*)mean, (float*)rstd, stream);
        Py_END_ALLOW_THREADS
        out = rc == 0 ? PyTuple_Pack(3, oy, om, orr) : PyLong_FromLong(rc);
    }
    Py_XDECREF(oy);
    Py_XDECREF(om);
    Py_XDECREF(orr);
    return out;
}

/* layer_norm_backward(dy, x, mean, rstd, weight, stream or None) -> (dx, dweight, dbias) of a matrix x, all
 * three wanted, or a status */
static PyObject* fc_layer_norm_backward(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 6, "layer_norm_backward") < 0) return NULL;
    trop_tensor dy, x, dx;
    void *mean, *rstd, *w, *dw, *db, *stream;
    if (obj_tensor_of(&dy, a[0], N_DTYPES) < 0 || obj_tensor_of(&x, a[1], N_DTYPES) < 0 || obj_stream(a[5], a[1], &stream) < 0)
        return NULL;
    const long device = obj_device(a[1]), other = obj_device(a[0]);
    const int32_t wdtype = dtype_or(a[4], x.dtype);
    if (device == -2 || other == -2 || wdtype == -2) return NULL;
    if (!g_empty || a[4] == Py_None || x.rank != 2 || dy.rank != 2 || x.dtype < 0 || device < 0 || device != other ||
        dy.shape[0] != x.shape[0] || dy.shape[1] != x.shape[1])
        return PyLong_FromLong(PLAIN_PATH);
    VECTOR(a[2], x.shape[0], TROP_F32, &mean);
    VECTOR(a[3], x.shape[0], TROP_F32, &rstd);
    VECTOR(a[4], x.shape[1], wdtype, &w);
    PyObject* ox = PyObject_CallOneArg(g_empty_like, a[1]);
    PyObject* ow = ox ? PyObject_CallOneArg(g_empty_like, a[4]) : NULL;
    PyObject* ob = ow ? PyObject_CallOneArg(g_empty_like, a[4]) : NULL;
    PyObject* out = NULL;
    if (ob && obj_tensor_of(&dx, ox, N_DTYPES) == 0 && fresh_ptr(ow, &dw) == 0 && fresh_ptr(ob, &db) == 0) {
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = tropical_layer_norm_backward(&dy, &x, (float*)mean, (float*)rstd, w, wdtype, &dx, dw, db, stream);
        Py_END_ALLOW_THREADS
        out = rc == 0 ? PyTuple_Pack(3, ox, ow, ob) : PyLong_FromLong(rc);
    }
    Py_XDECREF(ox);
    Py_XDECREF(ow);
    Py_XDECREF(ob);
    return out;
}

/* layer_norm_t(x, weight or None, bias or None, eps, y, mean, rstd, stream or None) */
static PyObject* fc_layer_norm_t(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 8, "layer_norm_t") < 0) return NULL;
    trop_tensor x, y;
    void *w, *b, *mean, *rstd, *stream;
    double eps;
    if (obj_tensor_of(&x, a[0], N_DTYPES) < 0 || as_double(a[3], &eps) < 0 || obj_tensor_of(&y, a[4], N_DTYPES) < 0 ||
        obj_stream(a[7], a[0], &stream) < 0)
        return NULL;
    if (as_rows(&x) || as_rows(&y)) return PyLong_FromLong(PLAIN_PATH);
    const long device = obj_device(a[0]);
    const int32_t wdtype = dtype_or(a[1] != Py_None ? a[1] : a[2], x.dtype);
    if (device == -2 || wdtype == -2) return NULL;
    VECTOR(a[1], x.shape[1], wdtype, &w);
    VECTOR(a[2], x.shape[1], wdtype, &b);
    VECTOR(a[5], x.shape[0], TROP_F32, &mean);
    VECTOR(a[6], x.shape[0], TROP_F32, &rstd);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = tropical_layer_norm(&x, w, b, wdtype, eps, &y, (float*)mean, (float*)rstd, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* layer_norm_backward_t(dy, x, mean, rstd, weight or None, dx or None, dweight or None, dbias or None,
 * stream or None) */
static PyObject* fc_layer_norm_backward_t(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 9, "layer_norm_backward_t") < 0) return NULL;
    trop_tensor dy, x, dx;
    void *mean, *rstd, *w, *dw, *db, *stream;
    if (obj_tensor_of(&dy, a[0], N_DTYPES) < 0 || obj_tensor_of(&x, a[1], N_DTYPES) < 0 ||
        (a[5] != Py_None && obj_tensor_of(&dx, a[5], N_DTYPES) < 0) || obj_stream(a[8], a[1], &stream) < 0)
        return NULL;
    if (as_rows(&dy) || as_rows(&x) || (a[5] != Py_None && as_rows(&dx))) return PyLong_FromLong(PLAIN_PATH);
    const long device = obj_device(a[1]), other = obj_device(a[0]);
    const int32_t wdtype = dtype_or(a[4] != Py_None ? a[4] : a[6] != Py_None ? a[6] : a[7], x.dtype);
    if (device == -2 || other == -2 || wdtype == -2) return NULL;
    if (device != other) return PyLong_FromLong(PLAIN_PATH);
    VECTOR(a[2], x.shape[0], TROP_F32, &mean);
    VECTOR(a[3], x.shape[0], TROP_F32, &rstd);
    VECTOR(a[4], x.shape[1], wdtype, &w);
    VECTOR(a[6], x.shape[1], wdtype, &dw);
    VECTOR(a[7], x.shape[1], wdtype, &db);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = tropical_layer_norm_backward(&dy, &x, (float*)mean, (float*)rstd, w, wdtype, a[5] == Py_None ? NULL : &dx, dw,
                                      db, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* x, w and target of the head's loss on one device: 0, PLAIN_PATH, or -1 */
static int head_operands(PyObject* const* a, trop_tensor* x, trop_tensor* w, trop_tensor* t, long* device)
{
    if (obj_tensor_of(x, a[0], N_DTYPES) < 0 || obj_tensor_of(w, a[1], N_DTYPES) < 0 || obj_tensor_of(t, a[2], N_DTYPES) < 0)
        return -1;
    const long d = obj_device(a[0]), e = obj_device(a[1]), f = obj_device(a[2]);
    if (d == -2 || e == -2 || f == -2) return -1;
    *device = d;
    return d == e && d == f && x->rank == 2 ? 0 : PLAIN_PATH;
}

/* linear_ce_t(x, w, target, ignore_index, mean, loss or None, lse, total or None, kept, stream or None) */
static PyObject* fc_linear_ce_t(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 10, "linear_ce_t") < 0) return NULL;
    trop_tensor x, w, t;
    void *loss, *lse, *total, *kept, *stream;
    int64_t ignore;
    long device;
    const int mean = PyObject_IsTrue(a[4]);
    const int usual = head_operands(a, &x, &w, &t, &device);
    if (usual < 0 || as_i64(a[3], &ignore) < 0 || mean < 0 || obj_stream(a[9], a[0], &stream) < 0) return NULL;
    if (usual > 0) return PyLong_FromLong(PLAIN_PATH);
    VECTOR(a[5], x.shape[0], TROP_F32, &loss);
    VECTOR(a[6], x.shape[0], TROP_F32, &lse);
    VECTOR(a[7], 1, TROP_F32, &total);
    VECTOR(a[8], 1, TROP_F32, &kept);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = tropical_linear_cross_entropy(&x, &w, &t, ignore, mean, (float*)loss, (float*)lse, (float*)total,
                                       (float*)kept, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* linear_ce(x, w, target, ignore_index, reduction: 0 none, 1 mean, 2 sum, stream or None) ->
 * (loss, lse, kept), or a status */
static PyObject* fc_linear_ce(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 6, "linear_ce") < 0) return NULL;
    trop_tensor x, w, t;
    void *loss = NULL, *lse, *total = NULL, *kept, *stream;
    int64_t ignore, reduction;
    long device;
    const int usual = head_operands(a, &x, &w, &t, &device);
    if (usual < 0 || as_i64(a[3], &ignore) < 0 || as_i64(a[4], &reduction) < 0 || obj_stream(a[5], a[0], &stream) < 0) return NULL;
    if (!g_empty || usual > 0 || device < 0) return PyLong_FromLong(PLAIN_PATH);
    /* the loss and the count are tensors of their own: as views of one they could not be changed in place */
    PyObject* ol = new_vector(x.shape[0], g_f32, a[0]);
    PyObject* ov = !ol ? NULL : reduction == 0 ? PyObject_CallOneArg(g_empty_like, ol) : new_scalar(a[0]);
    PyObject* ok = ov ? new_scalar(a[0]) : NULL;
    PyObject* out = NULL;
    if (ok && fresh_ptr(ol, &lse) == 0 && fresh_ptr(ov, reduction == 0 ? &loss : &total) == 0 && fresh_ptr(ok, &kept) == 0) {
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = tropical_linear_cross_entropy(&x, &w, &t, ignore, reduction == 1, (float*)loss, (float*)lse, (float*)total,
                                           (float*)kept, stream);
        Py_END_ALLOW_THREADS
        out = rc == 0 ? PyTuple_Pack(3, ov, ol, ok) : PyLong_FromLong(rc);
    }
    Py_XDECREF(ol);
    Py_XDECREF(ov);
    Py_XDECREF(ok);
    return out;
}

/* linear_ce_backward_t(x, w, target, ignore_index, dloss, lse, kept or None, dx or None, dw or None, stream or None) */
static PyObject* fc_linear_ce_backward_t(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 10, "linear_ce_backward_t") < 0) return NULL;
    trop_tensor x, w, t, g, dx, dw;
    void *lse, *kept, *stream;
    int64_t ignore;
    long device;
    const int usual = head_operands(a, &x, &w, &t, &device);
    if (usual < 0 || as_i64(a[3], &ignore) < 0 || obj_tensor_of(&g, a[4], N_DTYPES) < 0 ||
        (a[7] != Py_None && obj_tensor_of(&dx, a[7], N_DTYPES) < 0) ||
        (a[8] != Py_None && obj_tensor_of(&dw, a[8], N_DTYPES) < 0) || obj_stream(a[9], a[0], &stream) < 0)
        return NULL;
    const long other = obj_device(a[4]);
    if (other == -2) return NULL;
    if (usual > 0 || other != device || g.dtype != TROP_F32 || g.rank > 1 || (g.rank == 1 && g.shape[0] != x.shape[0]))
        return PyLong_FromLong(PLAIN_PATH);
    VECTOR(a[5], x.shape[0], TROP_F32, &lse);
    VECTOR(a[6], 1, TROP_F32, &kept);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = tropical_linear_cross_entropy_backward((float*)g.data, g.rank ? g.stride[0] : 0, &x, &w, &t, ignore, (float*)lse,
                                                (float*)kept, a[7] == Py_None ? NULL : &dx, a[8] == Py_None ? NULL : &dw,
                                                stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* adamw_plan_step(plan address, lr, beta1, beta2, eps, weight_decay, grad_scale, step, tensor, stream or None) */
static PyObject* fc_adamw_plan_step(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 10, "adamw_plan_step") < 0) return NULL;
    trop_adamw_options o;
    void *plan, *stream;
    if (as_ptr(a[0], &plan) < 0 || as_double(a[1], &o.lr) < 0 || as_double(a[2], &o.beta1) < 0 ||
        as_double(a[3], &o.beta2) < 0 || as_double(a[4], &o.eps) < 0 || as_double(a[5], &o.weight_decay) < 0 ||
        as_double(a[6], &o.grad_scale) < 0 || as_i64(a[7], &o.step) < 0 || obj_stream(a[9], a[8], &stream) < 0)
        return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = tropical_adamw_plan_step((trop_adamw_plan)plan, &o, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* adamw_plan_values(plan address, tensor, stream or None) */
static PyObject* fc_adamw_plan_values(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 3, "adamw_plan_values") < 0) return NULL;
    void *plan, *stream;
    if (as_ptr(a[0], &plan) < 0 || obj_stream(a[2], a[1], &stream) < 0) return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = tropical_adamw_plan_values((trop_adamw_plan)plan, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* ---- operators of a residual block.  Their results are allocated by the Python wrapper, which goes through its own
 * checks and the plain path wherever one of these returns anything but 0. */

/* a matrix on `device` (rows merged): 0, PLAIN_PATH, or -1 */
static int obj_rows(PyObject* obj, long device, trop_tensor* t)
{
    if (obj_tensor_of(t, obj, N_DTYPES) < 0) return -1;
    const long d = obj_device(obj);
    return d == -2 ? -1 : d != device || d < 0 || as_rows(t) ? PLAIN_PATH : 0;
}
#define ROWS(obj, t)                                          \
    do {                                                      \
        const int v_ = obj_rows((obj), device, (t));          \
        if (v_ < 0) return NULL;                              \
        if (v_ > 0) return PyLong_FromLong(PLAIN_PATH);       \
    } while (0)

#define DEVICE_OR_PLAIN                                       \
    do {                                                      \
        if (device == -2) return NULL;                        \
        if (device < 0) return PyLong_FromLong(PLAIN_PATH);   \
    } while (0)

/* activation_pack_t(x, codes, scales), activation_values_t(codes, scales, x) */
static PyObject* activation_t(PyObject* const* a, Py_ssize_t nargs, int pack)
{
    if (check_nargs(nargs, 3, pack ? "activation_pack_t" : "activation_values_t") < 0) return NULL;
    trop_tensor x, codes, scales;
    void* stream;
    PyObject *ox = a[pack ? 0 : 2], *oc = a[pack ? 1 : 0], *os = a[pack ? 2 : 1];
    const long device = obj_device(ox);
    DEVICE_OR_PLAIN;
    if (obj_stream(Py_None, ox, &stream) < 0) return NULL;
    ROWS(ox, &x);
    ROWS(oc, &codes);
    ROWS(os, &scales);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = pack ? tropical_activation_pack(&x, &codes, &scales, stream) : tropical_activation_values(&codes, &scales, &x, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}
static PyObject* fc_activation_pack_t(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    return activation_t(a, nargs, 1);
}
static PyObject* fc_activation_values_t(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    return activation_t(a, nargs, 0);
}

/* activation_weight_grad_t(dy, codes, scales, dw, db or None) */
static PyObject* fc_activation_weight_grad_t(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 5, "activation_weight_grad_t") < 0) return NULL;
    trop_tensor dy, codes, scales, dw;
    void *db, *stream;
    const long device = obj_device(a[0]);
    DEVICE_OR_PLAIN;
    if (obj_stream(Py_None, a[0], &stream) < 0 || obj_ptr(a[4], &db) < 0) return NULL;
    ROWS(a[0], &dy);
    ROWS(a[1], &codes);
    ROWS(a[2], &scales);
    ROWS(a[3], &dw);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = tropical_activation_weight_grad(&dy, &codes, &scales, &dw, db, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* The options (norm, post_norm, gate_act, alpha, scale, eps, weight, bias, post_weight, post_bias, scale vector) at a[0..10], the
 * vectors each a tensor or None and of one type (y's where there is none): 0, PLAIN_PATH, or -1 */
static int residual_options(PyObject* const* a, int64_t n, int32_t dtype, long device, trop_residual_options* o)
{
    int64_t v[3];
    for (int i = 0; i < 3; ++i)
        if (as_i64(a[i], &v[i]) < 0) return -1;
    if (as_double(a[3], &o->alpha) < 0 || as_double(a[4], &o->scale) < 0 || as_double(a[5], &o->eps) < 0) return -1;
    int32_t wdtype = dtype;
    for (int i = 10; i >= 6; --i) wdtype = dtype_or(a[i], wdtype);
    if (wdtype == -2) return -1;
    void* p[5];
    for (int i = 0; i < 5; ++i) {
        const int rc = obj_vector(a[6 + i], n, wdtype, device, &p[i]);
        if (rc != 0) return rc;
    }
    o->norm = (int)v[0], o->post_norm = (int)v[1], o->gate_act = (int)v[2], o->wdtype = wdtype;
    o->weight = p[0], o->bias = p[1], o->post_weight = p[2], o->post_bias = p[3], o->scale_vector = p[4];
    return 0;
}
#define OPTIONS(a, n, dtype, o)                                             \
    do {                                                                    \
        const int v_ = residual_options((a), (n), (dtype), device, (o));    \
        if (v_ < 0) return NULL;                                            \
        if (v_ > 0) return PyLong_FromLong(PLAIN_PATH);                     \
    } while (0)

/* u's, the gate's and r's 8-bit copies at a[0..5] (codes, scales; None: not kept) */
static int residual_kept(PyObject* const* a, long device, trop_tensor* t, trop_kept* kept)
{
    for (int i = 0; i < 3; ++i) {
        kept[i].codes = kept[i].scales = NULL;
        if (a[2 * i] == Py_None) continue;
        int rc = obj_rows(a[2 * i], device, &t[2 * i]);
        if (rc == 0) rc = obj_rows(a[2 * i + 1], device, &t[2 * i + 1]);
        if (rc != 0) return rc;
        kept[i].codes = &t[2 * i];
        kept[i].scales = &t[2 * i + 1];
    }
    return 0;
}
#define KEPT(a, t, kept)                                      \
    do {                                                      \
        const int v_ = residual_kept((a), device, (t), (kept)); \
        if (v_ < 0) return NULL;                              \
        if (v_ > 0) return PyLong_FromLong(PLAIN_PATH);       \
    } while (0)

/* two tensor objects of one shape, or (but > 0) of one but for `but` in the last place: 0, PLAIN_PATH, or -1 */
static int same_shape(PyObject* p, PyObject* q, int64_t but)
{
    PyObject* s = PyObject_GetAttr(p, s_shape);
    PyObject* t = s ? PyObject_GetAttr(q, s_shape) : NULL;
    int rc = t ? 0 : -1;
    if (rc == 0) {
        const Py_ssize_t n = PyTuple_Check(s) && PyTuple_Check(t) ? PyTuple_GET_SIZE(s) : -1;
        if (n < 1 || PyTuple_GET_SIZE(t) != n) rc = PLAIN_PATH;
        for (Py_ssize_t i = 0; i < n && rc == 0; ++i) {
            int64_t x, y;
            if (as_i64(PyTuple_GET_ITEM(s, i), &x) < 0 || as_i64(PyTuple_GET_ITEM(t, i), &y) < 0) rc = -1;
            else if (x != y && !(i == n - 1 && but > 0 && y == but)) rc = PLAIN_PATH;
        }
    }
    Py_XDECREF(s);
    Py_XDECREF(t);
    return rc;
}
#define SAME(p, q, but)                                       \
    do {                                                      \
        const int v_ = same_shape((p), (q), (but));           \
        if (v_ < 0) return NULL;                              \
        if (v_ > 0) return PyLong_FromLong(PLAIN_PATH);       \
    } while (0)

/* residual_norm_t(options x11, x, u, gate or None, y, r, stats, copies x6) */
static PyObject* fc_residual_norm_t(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 23, "residual_norm_t") < 0) return NULL;
    trop_tensor x, u, g, y, r, t[6];
    trop_residual_options o;
    trop_kept kept[3];
    void *stats, *stream;
    const long device = obj_device(a[11]);
    DEVICE_OR_PLAIN;
    if (obj_stream(Py_None, a[11], &stream) < 0 || obj_ptr(a[16], &stats) < 0) return NULL;
    SAME(a[11], a[12], 0);
    if (a[13] != Py_None) SAME(a[11], a[13], 1);
    ROWS(a[11], &x);
    ROWS(a[12], &u);
    if (a[13] != Py_None) ROWS(a[13], &g);
    ROWS(a[14], &y);
    ROWS(a[15], &r);
    OPTIONS(a, x.shape[1], x.dtype, &o);
    KEPT(a + 17, t, kept);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = tropical_residual_norm(&o, &x, &u, a[13] == Py_None ? NULL : &g, &y, &r, (float*)stats, a[17] == Py_None ? NULL : kept, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* residual_norm_backward_t(options x11, dy, dr, r, u, gate, stats, copies x6, dx, du, dgate, dscale, dweight, dbias, dpost_weight,
 * dpost_bias, x's dtype, u's dtype): None where a tensor is not given or not wanted */
static PyObject* fc_residual_norm_backward_t(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    if (check_nargs(nargs, 33, "residual_norm_backward_t") < 0) return NULL;
    trop_tensor in[5], t[6], out[3];
    trop_residual_options o;
    trop_residual_grads grads;
    trop_kept kept[3];
    void *stats, *stream, *v[5];
    const long device = obj_device(a[11]);
    DEVICE_OR_PLAIN;
    if (obj_stream(Py_None, a[11], &stream) < 0) return NULL;
    for (int i = 0; i < 5; ++i) {
        if (a[11 + i] == Py_None) continue;
        SAME(a[11], a[11 + i], i == 4 ? 1 : 0);
        ROWS(a[11 + i], &in[i]);
    }
    for (int i = 0; i < 3; ++i) {
        if (a[17 + 2 * i] != Py_None) {  /* codes, and a scale for each 32 of a row's */
            SAME(a[11], a[17 + 2 * i], 0);
            SAME(a[11], a[18 + 2 * i], (in[0].shape[1] + 31) / 32);
        }
        if (a[23 + i] != Py_None) ROWS(a[23 + i], &out[i]);
    }
    VECTOR(a[16], 4 * in[0].shape[0], TROP_F32, &stats);
    OPTIONS(a, in[0].shape[1], in[0].dtype, &o);
    KEPT(a + 17, t, kept);
    for (int i = 0; i < 5; ++i)
        if (obj_ptr(a[26 + i], &v[i]) < 0) return NULL;
    grads.dx = a[23] == Py_None ? NULL : &out[0];
    grads.du = a[24] == Py_None ? NULL : &out[1];
    grads.dgate = a[25] == Py_None ? NULL : &out[2];
    grads.dscale = v[0], grads.dweight = v[1], grads.dbias = v[2], grads.dpost_weight = v[3], grads.dpost_bias = v[4];
    int64_t xt, ut;
    if (as_i64(a[31], &xt) < 0 || as_i64(a[32], &ut) < 0) return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = tropical_residual_norm_backward(&o, &in[0], a[12] == Py_None ? NULL : &in[1], a[13] == Py_None ? NULL : &in[2],
                                         a[14] == Py_None ? NULL : &in[3], a[15] == Py_None ? NULL : &in[4], (const float*)stats,
                                         a[17] == Py_None ? NULL : kept, (int)xt, (int)ut, &grads, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* fc_last_error(PyObject* self, PyObject* const* a, Py_ssize_t nargs)
{
    (void)self;
    (void)a;
    if (check_nargs(nargs, 0, "last_error") < 0) return NULL;
    return PyUnicode_DecodeUTF8(tropical_last_error(), (Py_ssize_t)strlen(tropical_last_error()), "replace");
}

static PyMethodDef methods[] = {
    {"permute_trace", (PyCFunction)(void (*)(void))fc_permute_trace, METH_FASTCALL, "tropical_permute_trace"},
    {"permute_pair", (PyCFunction)(void (*)(void))fc_permute_pair, METH_FASTCALL, "tropical_permute_pair"},
    {"gemm", (PyCFunction)(void (*)(void))fc_gemm, METH_FASTCALL, "tropical_gemm_strided_batched_argmax"},
    {"einsum", (PyCFunction)(void (*)(void))fc_einsum, METH_FASTCALL, "tropical_einsum_pairwise"},
    {"last_error", (PyCFunction)(void (*)(void))fc_last_error, METH_FASTCALL, "tropical_last_error"},
    {"set_torch_handles", (PyCFunction)(void (*)(void))fc_set_torch_handles, METH_FASTCALL,
     "dtype objects (float32, int32, int64, float64, bfloat16, float16, int8, uint8) and the current-raw-stream function"},
    {"permute_trace_t", (PyCFunction)(void (*)(void))fc_permute_trace_t, METH_FASTCALL,
     "tropical_permute_trace on tensor objects"},
    {"permute_pair_t", (PyCFunction)(void (*)(void))fc_permute_pair_t, METH_FASTCALL,
     "tropical_permute_pair on tensor objects"},
    {"set_torch_allocators", (PyCFunction)(void (*)(void))fc_set_torch_allocators, METH_FASTCALL,
     "torch.empty, torch.empty_like, torch.float32"},
    {"layer_norm", (PyCFunction)(void (*)(void))fc_layer_norm, METH_FASTCALL, "tropical_layer_norm, its results allocated"},
    {"layer_norm_backward", (PyCFunction)(void (*)(void))fc_layer_norm_backward, METH_FASTCALL,
     "tropical_layer_norm_backward, its results allocated"},
    {"linear_ce", (PyCFunction)(void (*)(void))fc_linear_ce, METH_FASTCALL,
     "tropical_linear_cross_entropy, its results allocated"},
    {"layer_norm_t", (PyCFunction)(void (*)(void))fc_layer_norm_t, METH_FASTCALL,
     "tropical_layer_norm on tensor objects"},
    {"layer_norm_backward_t", (PyCFunction)(void (*)(void))fc_layer_norm_backward_t, METH_FASTCALL,
     "tropical_layer_norm_backward on tensor objects"},
    {"linear_ce_t", (PyCFunction)(void (*)(void))fc_linear_ce_t, METH_FASTCALL,
     "tropical_linear_cross_entropy on tensor objects"},
    {"linear_ce_backward_t", (PyCFunction)(void (*)(void))fc_linear_ce_backward_t, METH_FASTCALL,
     "tropical_linear_cross_entropy_backward on tensor objects"},
    {"adamw_plan_step", (PyCFunction)(void (*)(void))fc_adamw_plan_step, METH_FASTCALL, "tropical_adamw_plan_step"},
    {"adamw_plan_values", (PyCFunction)(void (*)(void))fc_adamw_plan_values, METH_FASTCALL, "tropical_adamw_plan_values"},
    {"activation_pack_t", (PyCFunction)(void (*)(void))fc_activation_pack_t, METH_FASTCALL, "tropical_activation_pack on tensor objects"},
    {"activation_values_t", (PyCFunction)(void (*)(void))fc_activation_values_t, METH_FASTCALL, "tropical_activation_values on tensor objects"},
    {"activation_weight_grad_t", (PyCFunction)(void (*)(void))fc_activation_weight_grad_t, METH_FASTCALL, "tropical_activation_weight_grad on tensor objects"},
    {"residual_norm_t", (PyCFunction)(void (*)(void))fc_residual_norm_t, METH_FASTCALL, "tropical_residual_norm on tensor objects"},
    {"residual_norm_backward_t", (PyCFunction)(void (*)(void))fc_residual_norm_backward_t, METH_FASTCALL, "tropical_residual_norm_backward on tensor objects"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", "hot entry points of the C ABI", -1,
                                    methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void)
{
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_device = PyUnicode_InternFromString("device");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!s_data_ptr || !s_shape || !s_stride || !s_dtype || !s_get_device || !s_cuda_stream) return NULL;
    return PyModule_Create(&module);
}
