/*
 * binding.c -- argument marshalling of the context-free operators for Python:
 * takes CUDA tensors apart (device, type, shape, stride, address) and makes
 * the C call.  No compute.  A call's host time is most of a small operator's:
 * the same checks in Python with ctypes took 2.5 to 4 us a call beside the
 * launch, here well under one.
 *
 * Tensors are read through their Python attributes only, so this depends on
 * neither PyTorch's headers nor its version.  Every function returns the C
 * call's status; a tensor that does not fit raises ValueError.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "moe.h"

int moe_binding_device(void); /* the current device, -1 where there is none; not part of the C interface */

static PyObject *s_get_device, *s_device, *s_dtype, *s_is_contiguous, *s_numel, *s_data_ptr, *s_shape, *s_stride, *s_cuda_stream;
static PyObject *t_f32, *t_bf16, *t_i32, *t_u8; /* torch dtypes */

static int bad(PyObject* t, const char* what, const char* expected) {
    if (!PyErr_Occurred() || PyErr_ExceptionMatches(PyExc_AttributeError)) {
        PyErr_Clear();
        PyObject *shape = PyObject_GetAttr(t, s_shape), *type = shape ? PyObject_GetAttr(t, s_dtype) : NULL;
        PyErr_Clear();
        if (shape && type) {
            PyObject* plain = PySequence_Tuple(shape);
            if (plain) PyErr_Format(PyExc_ValueError, "%s: expected %s, got %R %S", what, expected, plain, type);
            Py_XDECREF(plain);
        } else {
            PyErr_Format(PyExc_ValueError, "%s: expected %s, got %R", what, expected, (PyObject*)Py_TYPE(t));
        }
        Py_XDECREF(shape);
        Py_XDECREF(type);
    }
    return -1;
}

static int has_type(PyObject* t, PyObject* type) {
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    const int yes = d == type;
    Py_XDECREF(d);
    return yes;
}
/* the method's result as a whole number; -1 and an exception set if there is none */
static long long number(PyObject* t, PyObject* method) {
    PyObject* v = PyObject_CallMethodNoArgs(t, method);
    if (!v) return -1;
    const long long n = PyLong_AsLongLong(v);
    Py_DECREF(v);
    return n;
}
static int address(PyObject* t, void** out) {
    PyObject* v = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!v) return -1;
    *out = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return PyErr_Occurred() ? -1 : 0;
}

/*
 * A call's kernels run on the current device, and everything it is given has
 * to be there: an address of another GPU would be a fault.  *dev is that
 * device; where there is none to be told, the first tensor's.
 */
static int same_device(long long d, const char* what, int* dev) {
    if (*dev < 0) *dev = (int)d;
    if (d == *dev) return 0;
    PyErr_Format(PyExc_ValueError, "%s: is on GPU %lld, the call is for GPU %d", what, d, *dev);
    return -1;
}
/* 0: a CUDA tensor of that device; -1 and an exception if not */
static int on_device(PyObject* t, const char* what, const char* expected, int* dev) {
    const long long d = number(t, s_get_device); /* -1 for a tensor of the host */
    return d < 0 ? bad(t, what, expected) : same_device(d, what, dev);
}

/* contiguous CUDA tensor of at least n elements of the type; None gives NULL */
static int flat(PyObject* t, PyObject* type, long long n, const char* what, const char* expected, int* dev, void** out) {
    *out = NULL;
    if (t == Py_None) return 0;
    if (on_device(t, what, expected, dev)) return -1;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    const int contiguous = c == Py_True;
    Py_XDECREF(c);
    if (!contiguous || !has_type(t, type) || number(t, s_numel) < n) return bad(t, what, expected);
    return address(t, out);
}
static int flat_i32(PyObject* t, long long n, const char* what, int* dev, void** out) {
    return flat(t, t_i32, n, what, "a contiguous int32 CUDA tensor that is long enough", dev, out);
}
static int flat_f32(PyObject* t, long long n, const char* what, int* dev, void** out) {
    return flat(t, t_f32, n, what, "a contiguous float32 CUDA tensor that is long enough", dev, out);
}

typedef struct {
    void* p;
    int32_t type;
    int64_t rows, cols, ld;
} matrix_t;

/* 2D CUDA tensor of fp32 or bf16 with contiguous rows */
static int matrix(PyObject* t, const char* what, int* dev, matrix_t* m) {
    static const char* expected = "a 2D CUDA tensor of float32 or bfloat16 with contiguous rows";
    PyObject *d = PyObject_GetAttr(t, s_dtype), *shape = NULL, *stride = NULL;
    int rc = -1;
    const int ok = d == t_f32 || d == t_bf16;
    m->type = d == t_f32 ? MOE_F32 : MOE_BF16;
    Py_XDECREF(d);
    if (!ok) return bad(t, what, expected);
    if (on_device(t, what, expected, dev)) return -1;
    shape = PyObject_GetAttr(t, s_shape);
    if (shape) stride = PyObject_CallMethodNoArgs(t, s_stride);
    if (shape && stride && PyTuple_Check(shape) && PyTuple_Check(stride) && PyTuple_GET_SIZE(shape) == 2 &&
        PyTuple_GET_SIZE(stride) == 2) {
        m->rows = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
        m->cols = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 1));
        m->ld = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 0));
        if (m->rows <= 1) m->ld = m->cols; /* one row's stride means nothing */
        if (m->cols <= 1 || PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 1)) == 1) rc = address(t, &m->p);
    }
    Py_XDECREF(shape);
    Py_XDECREF(stride);
    return rc ? bad(t, what, expected) : 0;
}

/* rows and columns of a 2D tensor */
static int sides(PyObject* t, const char* what, int64_t* rows, int64_t* cols) {
    PyObject* shape = PyObject_GetAttr(t, s_shape);
    int rc = -1;
    if (shape && PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 2) {
        *rows = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
        *cols = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 1));
        rc = 0;
    }
    Py_XDECREF(shape);
    return rc ? bad(t, what, "a 2D tensor") : 0;
}

/* None, a raw cudaStream_t, or an object with one as cuda_stream */
static int stream_of(PyObject* s, void** out) {
    *out = NULL;
    if (s == Py_None) return 0;
    if (PyLong_Check(s)) {
        *out = PyLong_AsVoidPtr(s);
    } else {
        PyObject* v = PyObject_GetAttr(s, s_cuda_stream);
        if (!v) return -1;
        *out = PyLong_AsVoidPtr(v);
        Py_DECREF(v);
    }
    return PyErr_Occurred() ? -1 : 0;
}

/* copy of a ctypes structure */
static int structure(PyObject* o, void* out, size_t size, const char* what) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE)) return -1;
    const int ok = (size_t)b.len == size;
    if (ok) memcpy(out, b.buf, size);
    PyBuffer_Release(&b);
    if (!ok) PyErr_Format(PyExc_ValueError, "%s: not the library's structure", what);
    return ok ? 0 : -1;
}

/* copy of a matrix's descriptor, whose data is on the call's device as far as that is known (attribute device >= 0) */
static int descriptor(PyObject* o, moe_mx* out, const char* what, int* dev) {
    if (structure(o, out, sizeof *out, what)) return -1;
    PyObject* v = PyObject_GetAttr(o, s_device);
    const long d = v ? PyLong_AsLong(v) : -1;
    Py_XDECREF(v);
    if (PyErr_Occurred()) PyErr_Clear(); /* a structure of another make */
    return d < 0 ? 0 : same_device(d, what, dev);
}

static int count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return 0;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return -1;
}
#define ARGS PyObject *self, PyObject *const *v, Py_ssize_t n
#define STATUS(call)                 \
    do {                             \
        int rc_;                     \
        Py_BEGIN_ALLOW_THREADS       \
        rc_ = (call);                \
        Py_END_ALLOW_THREADS         \
        return PyLong_FromLong(rc_); \
    } while (0)
#define CHECK(cond, ...)                                \
    do {                                                \
        if (!(cond)) {                                  \
            PyErr_Format(PyExc_ValueError, __VA_ARGS__); \
            return NULL;                                \
        }                                               \
    } while (0)

/* cfg, logits, bias, idx, w, stream */
static PyObject* route(ARGS) {
    moe_route_config c;
    matrix_t l;
    void *bias, *idx, *w, *st;
    int dev = moe_binding_device();
    (void)self;
    if (count(n, 6) || structure(v[0], &c, sizeof c, "cfg") || matrix(v[1], "logits", &dev, &l)) return NULL;
    CHECK(l.cols == c.n_experts, "logits have %lld columns, the config %d experts", (long long)l.cols, c.n_experts);
    const long long out = l.rows * (long long)c.top_k;
    if (flat_f32(v[2], c.n_experts, "bias", &dev, &bias) || flat_i32(v[3], out, "idx", &dev, &idx) ||
        flat_f32(v[4], out, "w", &dev, &w) || stream_of(v[5], &st))
        return NULL;
    STATUS(moe_route(&c, l.p, l.type, l.ld, bias, l.rows, idx, w, st));
}

/* idx, n_experts, offsets, row_of_pair, token_of_row, group_of_row, workspace, stream */
static PyObject* dispatch(ARGS) {
    int64_t T, k;
    void *idx, *off, *rop, *tor, *gor, *ws, *st;
    long long bytes = 0;
    int dev = moe_binding_device();
    (void)self;
    if (count(n, 8) || sides(v[0], "idx", &T, &k)) return NULL;
    const long E = PyLong_AsLong(v[1]);
    if (E == -1 && PyErr_Occurred()) return NULL;
    CHECK(k <= INT32_MAX && E >= INT32_MIN && E < INT32_MAX, "idx has too many columns, or n_experts is out of range");
    if (flat_i32(v[0], T * k, "idx", &dev, &idx) || flat_i32(v[2], E + 1, "offsets", &dev, &off) ||
        flat_i32(v[3], T * k, "row_of_pair", &dev, &rop) || flat_i32(v[4], T * k, "token_of_row", &dev, &tor) ||
        flat_i32(v[5], T * k, "group_of_row", &dev, &gor) ||
        flat(v[6], t_u8, 0, "workspace", "a contiguous uint8 CUDA tensor", &dev, &ws) || stream_of(v[7], &st))
        return NULL;
    if (v[6] != Py_None && (bytes = number(v[6], s_numel)) < 0) return NULL;
    STATUS(moe_dispatch(idx, T, (int32_t)k, (int32_t)E, off, rop, tor, gor, ws, (size_t)bytes, st));
}

static int64_t rows_of(const moe_mx* m) { return m->ragged ? m->rows : m->rows * m->groups; }

/* m, src, act, src_row, group_of_row, offsets, tensor_scale, stream */
static PyObject* quantise(ARGS) {
    moe_mx m;
    matrix_t s;
    void *row, *gor, *off, *ts, *st;
    int dev = moe_binding_device();
    (void)self;
    if (count(n, 8) || descriptor(v[0], &m, "m", &dev) || matrix(v[1], "src", &dev, &s)) return NULL;
    const long act = PyLong_AsLong(v[2]);
    if (act == -1 && PyErr_Occurred()) return NULL;
    const int64_t rows = rows_of(&m), cols = act == MOE_ACT_SWIGLU ? 2 * (int64_t)m.cols : m.cols;
    CHECK(s.cols == cols, "src has %lld columns, the matrix needs %lld", (long long)s.cols, (long long)cols);
    CHECK(v[3] != Py_None || s.rows >= rows, "src has %lld rows, the matrix %lld", (long long)s.rows, (long long)rows);
    if (flat_i32(v[3], rows, "src_row", &dev, &row) || flat_i32(v[4], rows, "group_of_row", &dev, &gor) ||
        flat_i32(v[5], (long long)m.groups + 1, "offsets", &dev, &off) ||
        flat_f32(v[6], m.groups, "tensor_scale", &dev, &ts) || stream_of(v[7], &st))
        return NULL;
    STATUS(moe_mx_quantise_rows(&m, s.p, s.rows, s.type, s.ld, (int32_t)act, row, gor, off, ts, st));
}

/* m, dst, group_of_row, offsets, tensor_scale, stream */
static PyObject* dequantise(ARGS) {
    moe_mx m;
    matrix_t d;
    void *gor, *off, *ts, *st;
    int dev = moe_binding_device();
    (void)self;
    if (count(n, 6) || descriptor(v[0], &m, "m", &dev) || matrix(v[1], "dst", &dev, &d)) return NULL;
    const int64_t rows = rows_of(&m);
    CHECK(d.cols == m.cols && d.rows >= rows, "dst is %lld x %lld, the matrix %lld x %d", (long long)d.rows,
          (long long)d.cols, (long long)rows, m.cols);
    if (flat_i32(v[2], rows, "group_of_row", &dev, &gor) ||
        flat_i32(v[3], (long long)m.groups + 1, "offsets", &dev, &off) || flat_f32(v[4], m.groups, "tensor_scale", &dev, &ts) || stream_of(v[5], &st))
        return NULL;
    STATUS(moe_mx_dequantise(&m, gor, off, ts, d.p, d.type, d.ld, st));
}

/* x, w, y, offsets, alpha, stream */
static PyObject* product(ARGS) {
    moe_mx x, w;
    matrix_t y;
    void *off, *alpha, *st;
    int dev = moe_binding_device();
    (void)self;
    if (count(n, 6) || descriptor(v[0], &x, "x", &dev) || descriptor(v[1], &w, "w", &dev) ||
        matrix(v[2], "y", &dev, &y))
        return NULL;
    CHECK(y.rows >= x.rows && y.cols == w.rows, "y is %lld x %lld, the product %lld x %lld", (long long)y.rows,
          (long long)y.cols, (long long)x.rows, (long long)w.rows);
    if (flat_i32(v[3], (long long)x.groups + 1, "offsets", &dev, &off) ||
        flat_f32(v[4], w.groups, "alpha", &dev, &alpha) || stream_of(v[5], &st))
        return NULL;
    STATUS(moe_mx_product(&x, &w, off, alpha, y.p, y.type, y.ld, st));
}

/* rows, row_of_pair, w, y, stream */
static PyObject* combine(ARGS) {
    matrix_t r, y;
    int64_t T, k;
    void *rop, *w, *st;
    int dev = moe_binding_device();
    (void)self;
    if (count(n, 5) || matrix(v[0], "rows", &dev, &r) || sides(v[1], "row_of_pair", &T, &k) ||
        matrix(v[3], "y", &dev, &y))
        return NULL;
    CHECK(y.cols == r.cols && y.rows == T, "y is %lld x %lld, expected %lld x %lld", (long long)y.rows, (long long)y.cols,
          (long long)T, (long long)r.cols);
    CHECK(k <= INT32_MAX && r.cols <= INT32_MAX, "row_of_pair or rows has too many columns");
    if (flat_i32(v[1], T * k, "row_of_pair", &dev, &rop) || flat_f32(v[2], T * k, "w", &dev, &w) ||
        stream_of(v[4], &st))
        return NULL;
    STATUS(moe_combine_rows(r.p, r.rows, r.type, r.ld, rop, w, T, (int32_t)k, (int32_t)r.cols, y.p, y.type, y.ld, st));
}

/* the torch dtypes float32, bfloat16, int32, uint8 */
static PyObject* dtypes(ARGS) {
    (void)self;
    if (count(n, 4)) return NULL;
    PyObject** to[4] = {&t_f32, &t_bf16, &t_i32, &t_u8};
    for (int i = 0; i < 4; ++i) {
        Py_INCREF(v[i]);
        Py_XSETREF(*to[i], v[i]);
    }
    Py_RETURN_NONE;
}

#define FN(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FN(route),   FN(dispatch), FN(quantise), FN(dequantise),
                                FN(product), FN(combine),  FN(dtypes),   {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__call(void) {
    struct {
        PyObject** at;
        const char* name;
    } names[] = {{&s_get_device, "get_device"}, {&s_device, "device"},     {&s_dtype, "dtype"},
                 {&s_is_contiguous, "is_contiguous"}, {&s_numel, "numel"}, {&s_data_ptr, "data_ptr"},
                 {&s_shape, "shape"}, {&s_stride, "stride"}, {&s_cuda_stream, "cuda_stream"}};
    for (size_t i = 0; i < sizeof names / sizeof names[0]; ++i)
        if (!(*names[i].at = PyUnicode_InternFromString(names[i].name))) return NULL;
    return PyModule_Create(&module);
}
