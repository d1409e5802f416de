/*
 * binding.c -- argument marshalling of the context-free operators for Python:
 * takes CUDA tensors apart (device, type, shape, stride, address) and makes
 * the C call.  No compute.  A call's host time is most of a small operator's:
 * the same checks in Python with ctypes took 2.5 to 4 us a call beside the
 * launch, here well under one.
 *
 * A torch tensor is read by tensor.cc; any other object that has a tensor's
 * attributes through those.  A function returns the C call's
 * status; those with names raise what it stands for, and are the package's
 * functions themselves (a Python function around them would cost a tenth of a
 * small call).  A tensor that does not fit raises ValueError.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "moe.h"
#include "tensor.h"

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

/* the method's result as a whole number; -1 and an exception set if there is none */
static long long number(PyObject* t, PyObject* method) {
    PyObject* v = PyObject_CallMethodNoArgs(t, method);
    if (!v) return -1;
    const long long n = PyLong_AsLongLong(v);
    Py_DECREF(v);
    return n;
}
/* a tuple's first MOE_TENSOR_DIMS numbers; its length, or -1 */
static int numbers(PyObject* tuple, int64_t* out) {
    const int n = tuple && PyTuple_Check(tuple) ? (int)PyTuple_GET_SIZE(tuple) : -1;
    for (int i = 0; i < n && i < MOE_TENSOR_DIMS; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    Py_XDECREF(tuple);
    return PyErr_Occurred() ? -1 : n;
}
/* a tensor, or what has its attributes; -1 (an exception may be set) if that lacks one */
static int look(PyObject* t, moe_tensor* v) {
    if (moe_tensor_of(t, v)) return 0;
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    Py_XDECREF(d);
    if (!d) return -1;
    v->type = d == t_f32 ? MOE_TENSOR_F32 : d == t_bf16 ? MOE_TENSOR_BF16 : d == t_i32 ? MOE_TENSOR_I32 : d == t_u8 ? MOE_TENSOR_U8 : MOE_TENSOR_OTHER;
    v->device = (int)number(t, s_get_device);
    if (PyErr_Occurred()) return -1;
    v->dims = numbers(PyObject_GetAttr(t, s_shape), v->shape);
    if (PyErr_Occurred() || v->dims != numbers(PyObject_CallMethodNoArgs(t, s_stride), v->stride)) return -1;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    v->contiguous = c == Py_True;
    Py_XDECREF(c);
    v->numel = c ? number(t, s_numel) : -1;
    PyObject* p = PyErr_Occurred() ? NULL : PyObject_CallMethodNoArgs(t, s_data_ptr);
    v->p = p ? PyLong_AsVoidPtr(p) : NULL;
    Py_XDECREF(p);
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
static int on_device(PyObject* t, const moe_tensor* v, const char* what, const char* expected, int* dev) {
    return v->device < 0 ? bad(t, what, expected) : same_device(v->device, what, dev);
}

/* contiguous CUDA tensor of at least n elements of the type; None gives NULL */
static int flat(PyObject* t, int type, long long n, const char* what, const char* expected, int* dev, void** out) {
    moe_tensor v;
    *out = NULL;
    if (t == Py_None) return 0;
    if (look(t, &v)) return bad(t, what, expected);
    if (on_device(t, &v, what, expected, dev)) return -1;
    if (!v.contiguous || v.type != type || v.numel < n) return bad(t, what, expected);
    *out = v.p;
    return 0;
}
static int flat_i32(PyObject* t, long long n, const char* what, int* dev, void** out) {
    return flat(t, MOE_TENSOR_I32, n, what, "a contiguous int32 CUDA tensor that is long enough", dev, out);
}
static int flat_f32(PyObject* t, long long n, const char* what, int* dev, void** out) {
    return flat(t, MOE_TENSOR_F32, n, what, "a contiguous float32 CUDA tensor that is long enough", dev, out);
}

/* a uint8 tensor's bytes; None has none */
static int room(PyObject* t, int* dev, void** p, long long* bytes) {
    moe_tensor v;
    if (flat(t, MOE_TENSOR_U8, 0, "workspace", "a contiguous uint8 CUDA tensor", dev, p)) return -1;
    *bytes = t == Py_None || look(t, &v) ? 0 : v.numel;
    return PyErr_Occurred() ? -1 : 0;
}

typedef struct {
    void* p;
    int32_t type;
    int64_t rows, cols, ld;
} matrix_t;

/* 2D CUDA tensor of fp32 or bf16 with contiguous rows */
static int matrix(PyObject* t, const char* what, int* dev, matrix_t* m) {
    static const char* expected = "a 2D CUDA tensor of float32 or bfloat16 with contiguous rows";
    moe_tensor v;
    if (look(t, &v) || (v.type != MOE_TENSOR_F32 && v.type != MOE_TENSOR_BF16)) return bad(t, what, expected);
    if (on_device(t, &v, what, expected, dev)) return -1;
    if (v.dims != 2 || (v.shape[1] > 1 && v.stride[1] != 1)) return bad(t, what, expected);
    m->p = v.p;
    m->type = v.type == MOE_TENSOR_F32 ? MOE_F32 : MOE_BF16;
    m->rows = v.shape[0], m->cols = v.shape[1];
    m->ld = m->rows <= 1 ? m->cols : v.stride[0]; /* one row's stride means nothing */
    return 0;
}

typedef struct {
    void* p;
    int32_t type;
    int64_t n, heads, dim, ld, head; /* element (t, h, i) at t * ld + h * head + i */
} heads_t;

/* 3D CUDA tensor [tokens, heads, values] of fp32 or bf16, its values contiguous */
static int heads_of(PyObject* t, const char* what, int* dev, heads_t* m) {
    static const char* expected = "a 3D CUDA tensor of float32 or bfloat16 with contiguous heads";
    moe_tensor v;
    if (look(t, &v) || (v.type != MOE_TENSOR_F32 && v.type != MOE_TENSOR_BF16)) return bad(t, what, expected);
    if (on_device(t, &v, what, expected, dev)) return -1;
    if (v.dims != 3 || v.shape[1] > INT32_MAX || v.shape[2] > INT32_MAX || (v.shape[2] > 1 && v.stride[2] != 1))
        return bad(t, what, expected);
    m->p = v.p;
    m->type = v.type == MOE_TENSOR_F32 ? MOE_F32 : MOE_BF16;
    m->n = v.shape[0], m->heads = v.shape[1], m->dim = v.shape[2];
    m->head = m->heads <= 1 ? m->dim : v.stride[1]; /* one head's or token's stride means nothing */
    m->ld = m->n <= 1 ? m->heads * m->dim : v.stride[0];
    return 0;
}

/* rows and columns of a 2D tensor */
static int sides(PyObject* t, const char* what, int64_t* rows, int64_t* cols) {
    moe_tensor v;
    if (look(t, &v) || v.dims != 2) return bad(t, what, "a 2D tensor");
    *rows = v.shape[0], *cols = v.shape[1];
    return 0;
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

/*
 * Arguments by place and by name into v[0..n-1], in the order of the names; the first `required` have to be given, the
 * others stay None.  The names are interned, as the ones in a caller's code are.
 */
static int arguments(PyObject* const* given, Py_ssize_t n_given, PyObject* kwnames, PyObject* const* names, int n,
                     int required, const char* what, PyObject** v) {
    if (n_given > n) {
        PyErr_Format(PyExc_TypeError, "%s: at most %d arguments, got %zd", what, n, n_given);
        return -1;
    }
    for (int i = 0; i < n; ++i) v[i] = i < n_given ? given[i] : NULL;
    const Py_ssize_t kw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t k = 0; k < kw; ++k) {
        PyObject* name = PyTuple_GET_ITEM(kwnames, k);
        int i = 0;
        while (i < n && names[i] != name) ++i;
        if (i == n)
            for (i = 0; i < n && PyUnicode_Compare(names[i], name) != 0; ++i)
                if (PyErr_Occurred()) return -1;
        if (i == n || v[i]) {
            PyErr_Format(PyExc_TypeError, i == n ? "%s: no argument %R" : "%s: %R is given twice", what, name);
            return -1;
        }
        v[i] = given[n_given + k];
    }
    for (int i = 0; i < n; ++i) {
        if (!v[i] && i < required) {
            PyErr_Format(PyExc_TypeError, "%s: %S is required", what, names[i]);
            return -1;
        }
        if (!v[i]) v[i] = Py_None;
    }
    return 0;
}
#define KWARGS PyObject *self, PyObject *const *given, Py_ssize_t n_given, PyObject *kwnames
static PyObject* failed; /* the package's function that raises what a status stands for */
#define NONE_OR_RAISE(call)                                     \
    do {                                                        \
        int rc_;                                                \
        Py_BEGIN_ALLOW_THREADS                                  \
        rc_ = (call);                                           \
        Py_END_ALLOW_THREADS                                    \
        if (rc_ >= 0) Py_RETURN_NONE;                           \
        return PyObject_CallFunction(failed, "i", rc_);         \
    } while (0)

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
        room(v[6], &dev, &ws, &bytes) || stream_of(v[7], &st))
        return NULL;
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

/* copy of a batch's descriptor, its lists on the call's device; None gives NULL */
static int batch(PyObject* o, moe_seqs* out, const moe_seqs** p, int* dev) {
    *p = NULL;
    if (o == Py_None) return 0;
    if (structure(o, out, sizeof *out, "seqs")) return -1;
    PyObject* v = PyObject_GetAttr(o, s_device);
    const long d = v ? PyLong_AsLong(v) : -1;
    Py_XDECREF(v);
    if (PyErr_Occurred()) PyErr_Clear();
    *p = out;
    return d < 0 ? 0 : same_device(d, "seqs", dev);
}

/*
 * A state [slots, d[0], .., d[n - 1]] of the type, contiguous: its slots, and -1 and an exception if it is another tensor.
 * Every extent is looked at: one with its dimensions exchanged has as many values.
 */
static long long state_of(PyObject* t, int type, int n, const int64_t* d, const char* expected, int* dev, void** out) {
    moe_tensor v;
    if (look(t, &v)) return bad(t, "state", expected);
    if (on_device(t, &v, "state", expected, dev)) return -1;
    if (v.dims != n + 1 || v.type != type || !v.contiguous) return bad(t, "state", expected);
    for (int i = 0; i < n; ++i)
        if (v.shape[1 + i] != d[i]) return bad(t, "state", expected);
    *out = v.p;
    return v.shape[0];
}
/* contiguous fp32 [at least n, heads]; one of [heads, n] has as many values */
static int gates_of(PyObject* t, int64_t n, int64_t heads, const char* what, int* dev, void** out) {
    static const char* expected = "a contiguous float32 CUDA tensor [T, v_heads]";
    moe_tensor v;
    if (look(t, &v)) return bad(t, what, expected);
    if (on_device(t, &v, what, expected, dev)) return -1;
    if (v.dims != 2 || v.type != MOE_TENSOR_F32 || !v.contiguous || v.shape[0] < n || v.shape[1] != heads)
        return bad(t, what, expected);
    *out = v.p;
    return 0;
}
/* the address of a state without slots, which is never read or written */
static _Alignas(16) char no_slots[16];

static PyObject* conv_names[8];
static const char conv_doc[] =
    "moe_conv(x, w, y, bias=None, act=MOE_ACT_SILU, seqs=None, state=None, stream=None)\n--\n\n"
    "Causal convolution of each column of x [T, channels] by w [channels, width], into y; state [slots, width - 1,\n"
    "channels], of x's type, is read and replaced.";
static PyObject* conv(KWARGS) {
    PyObject* v[8];
    matrix_t x, w, y;
    moe_seqs q;
    const moe_seqs* qp;
    void *bias, *state = NULL, *st;
    long long slots = 0;
    int dev = moe_binding_device();
    (void)self;
    if (arguments(given, n_given, kwnames, conv_names, 8, 3, "moe_conv", v) || matrix(v[0], "x", &dev, &x) ||
        matrix(v[1], "w", &dev, &w) || matrix(v[2], "y", &dev, &y))
        return NULL;
    const long act = v[4] == Py_None ? MOE_ACT_SILU : PyLong_AsLong(v[4]);
    if (act == -1 && PyErr_Occurred()) return NULL;
    CHECK(x.cols <= INT32_MAX && w.rows == x.cols && w.cols <= INT32_MAX && w.ld == w.cols,
          "w is %lld x %lld, expected contiguous rows of each of %lld channels", (long long)w.rows, (long long)w.cols,
          (long long)x.cols);
    CHECK(y.cols == x.cols && y.rows >= x.rows && y.type == x.type, "y is %lld x %lld, x %lld x %lld, of one type",
          (long long)y.rows, (long long)y.cols, (long long)x.rows, (long long)x.cols);
    if (flat_f32(v[3], x.cols, "bias", &dev, &bias) || batch(v[5], &q, &qp, &dev) || stream_of(v[7], &st)) return NULL;
    if (v[6] != Py_None) {
        const int64_t rest[] = {w.cols - 1, x.cols};
        slots = state_of(v[6], x.type == MOE_F32 ? MOE_TENSOR_F32 : MOE_TENSOR_BF16, 2, rest,
                         "a contiguous CUDA tensor [slots, width - 1, channels] of x's type", &dev, &state);
        if (slots < 0) return NULL;
        if (!slots) state = no_slots; /* which torch gives no address: every sequence is left out */
    }
    NONE_OR_RAISE(moe_conv(qp, x.p, x.type, x.ld, x.rows, (int32_t)x.cols, w.p, w.type, (int32_t)w.cols, bias, (int32_t)act,
                           state, slots, y.p, y.ld, st));
}

static PyObject* head_norm_names[11];
static const char head_norm_doc[] =
    "moe_head_norm(cfg, x, y, weight=None, gate=None, x2=None, y2=None, weight2=None, pos=None, inv_freq=None, "
    "stream=None)\n--\n\n"
    "Norm of each head of x [T, heads, dim], then the rotation or the gate, into y (which may be x); x2, y2: a second\n"
    "tensor in the same pass.  pos [T] int32, inv_freq [rot_dim / 2] fp32.";
static PyObject* head_norm(KWARGS) {
    PyObject* v[11];
    moe_head_norm_config c;
    moe_heads t[2];
    heads_t x, y, gate;
    void *pos, *freq, *weight, *st;
    int dev = moe_binding_device();
    (void)self;
    if (arguments(given, n_given, kwnames, head_norm_names, 11, 3, "moe_head_norm", v) || structure(v[0], &c, sizeof c, "cfg"))
        return NULL;
    const int second = v[5] != Py_None;
    CHECK(second || v[6] == Py_None, "y2 goes with x2");
    memset(t, 0, sizeof t);
    long long tokens = 0;
    for (int i = 0; i <= second; ++i) {
        const char *xn = i ? "x2" : "x", *yn = i ? "y2" : "y";
        if (heads_of(v[i ? 5 : 1], xn, &dev, &x) || heads_of(v[i ? 6 : 2], yn, &dev, &y)) return NULL;
        if (!i) {
            tokens = x.n;
            c.dim = (int32_t)x.dim;
        }
        CHECK(x.n == tokens && x.dim == c.dim, "%s is %lld x %lld x %lld, expected %lld tokens and heads of %d", xn,
              (long long)x.n, (long long)x.heads, (long long)x.dim, tokens, c.dim);
        CHECK(y.n == x.n && y.heads == x.heads && y.dim == x.dim && y.type == x.type,
              "%s is %lld x %lld x %lld, expected %lld x %lld x %lld of %s's type", yn, (long long)y.n, (long long)y.heads,
              (long long)y.dim, (long long)x.n, (long long)x.heads, (long long)x.dim, xn);
        if (flat_f32(v[i ? 7 : 3], x.dim, "weight", &dev, &weight)) return NULL;
        t[i].x_dev = x.p, t[i].x_ld = x.ld, t[i].x_head = x.head;
        t[i].y_dev = y.p, t[i].y_ld = y.ld, t[i].y_head = y.head;
        t[i].weight_dev = weight;
        t[i].heads = (int32_t)x.heads;
        t[i].type = x.type;
        if (!i && v[4] != Py_None) {
            if (heads_of(v[4], "gate", &dev, &gate)) return NULL;
            CHECK(gate.n == x.n && gate.heads == x.heads && gate.dim == x.dim && gate.type == x.type,
                  "gate is %lld x %lld x %lld, expected %lld x %lld x %lld of x's type", (long long)gate.n,
                  (long long)gate.heads, (long long)gate.dim, (long long)x.n, (long long)x.heads, (long long)x.dim);
            t[i].gate_dev = gate.p, t[i].gate_ld = gate.ld, t[i].gate_head = gate.head;
        }
    }
    CHECK(second || v[7] == Py_None, "weight2 goes with x2");
    if (flat_i32(v[8], tokens, "pos", &dev, &pos) || flat_f32(v[9], c.rot_dim / 2, "inv_freq", &dev, &freq) ||
        stream_of(v[10], &st))
        return NULL;
    NONE_OR_RAISE(moe_head_norm(&c, &t[0], second ? &t[1] : NULL, pos, freq, tokens, st));
}

static PyObject* delta_names[11];
static const char delta_doc[] =
    "moe_delta(q, k, v, g, beta, state, o, scale=1.0, seqs=None, workspace=None, stream=None)\n--\n\n"
    "The gated delta rule: q, k [T, k_heads, k_dim], v, o [T, v_heads, v_dim] bf16, g, beta [T, v_heads] fp32, state\n"
    "[slots, v_heads, v_dim, k_dim] fp32 (read and replaced) or None; workspace: uint8, moe_delta_workspace() bytes,\n"
    "not looked at where that is 0.";
static PyObject* delta(KWARGS) {
    PyObject* v[11];
    moe_delta_config c;
    heads_t q, k, val, o;
    moe_seqs b;
    const moe_seqs* bp;
    void *g, *beta, *state = NULL, *ws = NULL, *st;
    long long slots = 0, bytes = 0;
    int dev = moe_binding_device();
    (void)self;
    if (arguments(given, n_given, kwnames, delta_names, 11, 7, "moe_delta", v) || heads_of(v[0], "q", &dev, &q) || heads_of(v[1], "k", &dev, &k) ||
        heads_of(v[2], "v", &dev, &val) || heads_of(v[6], "o", &dev, &o))
        return NULL;
    const double scale = v[7] == Py_None ? 1.0 : PyFloat_AsDouble(v[7]);
    if (scale == -1.0 && PyErr_Occurred()) return NULL;
    CHECK(q.type == MOE_BF16 && k.type == MOE_BF16 && val.type == MOE_BF16 && o.type == MOE_BF16,
          "q, k, v and o: expected bfloat16");
    CHECK(q.n == val.n && k.n == val.n && k.heads == q.heads && k.dim == q.dim,
          "q is %lld x %lld x %lld, k %lld x %lld x %lld, v has %lld tokens", (long long)q.n, (long long)q.heads,
          (long long)q.dim, (long long)k.n, (long long)k.heads, (long long)k.dim, (long long)val.n);
    CHECK(o.n >= val.n && o.heads == val.heads && o.dim == val.dim, "o is %lld x %lld x %lld, v %lld x %lld x %lld",
          (long long)o.n, (long long)o.heads, (long long)o.dim, (long long)val.n, (long long)val.heads, (long long)val.dim);
    CHECK(q.head == q.dim && k.head == k.dim && val.head == val.dim && o.head == o.dim,
          "q, k, v and o: the heads of a token have to stand side by side");
    c.k_heads = (int32_t)q.heads, c.v_heads = (int32_t)val.heads;
    c.k_dim = (int32_t)q.dim, c.v_dim = (int32_t)val.dim;
    c.scale = (float)scale;
    CHECK(v[3] != Py_None && v[4] != Py_None, "g and beta are required");
    if (gates_of(v[3], val.n, val.heads, "g", &dev, &g) || gates_of(v[4], val.n, val.heads, "beta", &dev, &beta) ||
        batch(v[8], &b, &bp, &dev) || stream_of(v[10], &st))
        return NULL;
    if (v[9] != Py_None && moe_delta_workspace(&c, val.n, bp ? bp->n : 1, bp ? bp->offsets_dev ? bp->max_len : 1 : 0) &&
        room(v[9], &dev, &ws, &bytes))
        return NULL;
    if (v[5] != Py_None) {
        const int64_t rest[] = {val.heads, val.dim, q.dim};
        slots = state_of(v[5], MOE_TENSOR_F32, 3, rest, "a contiguous float32 CUDA tensor [slots, v_heads, v_dim, k_dim]", &dev,
                         &state);
        if (slots < 0) return NULL;
        if (!slots) state = no_slots;
    }
    NONE_OR_RAISE(moe_delta(&c, bp, q.p, q.ld, k.p, k.ld, val.p, val.ld, g, beta, state, slots, o.p, o.ld, val.n, ws,
                            (size_t)bytes, st));
}

/* the package's function for a failed call's status */
static PyObject* on_failure(ARGS) {
    (void)self;
    if (count(n, 1)) return NULL;
    Py_INCREF(v[0]);
    Py_XSETREF(failed, v[0]);
    Py_RETURN_NONE;
}

/* the torch and Python that the module was compiled for */
static PyObject* built_for(PyObject* self, PyObject* none) {
    (void)self, (void)none;
    return PyUnicode_FromString(moe_tensor_built_for());
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
#define KWFN(name) {"moe_" #name, (PyCFunction)(void (*)(void))name, METH_FASTCALL | METH_KEYWORDS, name##_doc}
static PyMethodDef methods[] = {FN(route),   FN(dispatch), FN(quantise), FN(dequantise),
                                FN(product), FN(combine),  FN(dtypes),   FN(on_failure),
                                KWFN(conv),  KWFN(head_norm), KWFN(delta), {"built_for", built_for, METH_NOARGS, NULL}, {NULL, NULL, 0, NULL}};
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
    static const char* const conv_args[] = {"x", "w", "y", "bias", "act", "seqs", "state", "stream"};
    static const char* const head_norm_args[] = {"cfg", "x", "y", "weight", "gate", "x2", "y2", "weight2", "pos", "inv_freq", "stream"};
    static const char* const delta_args[] = {"q", "k", "v", "g", "beta", "state", "o", "scale", "seqs", "workspace", "stream"};
    for (int i = 0; i < 8; ++i)
        if (!(conv_names[i] = PyUnicode_InternFromString(conv_args[i]))) return NULL;
    for (int i = 0; i < 11; ++i)
        if (!(head_norm_names[i] = PyUnicode_InternFromString(head_norm_args[i])) ||
            !(delta_names[i] = PyUnicode_InternFromString(delta_args[i])))
            return NULL;
    return PyModule_Create(&module);
}
