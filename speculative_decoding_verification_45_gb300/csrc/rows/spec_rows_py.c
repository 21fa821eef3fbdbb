/* spec_rows_py.c -- the common calls of 8-bit rows without the interpreter's share.
 *
 * One row through a norm is 2 us of work for the GPU and was 14 us of Python: a
 * third of that reading tensors' attributes, a third converting arguments.  The
 * functions here take the same tensors, and make the call where everything is as
 * usual: tensors on the current device, of the types and shapes that belong
 * together, rows at one stride of a multiple of 16 bytes, outputs to be made, the
 * current stream.  Anything else, an error among it, is left to rows.py: they
 * return None, with nothing enqueued, and its checks say what is wrong.
 *
 * Python's C API only: tensors are read through their methods, and made by torch. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <math.h>
#include <stdint.h>

#include "spec_verify.h"

static PyObject *s_dtype, *s_shape, *s_get_device, *s_data_ptr, *s_is_contiguous, *s_stride, *s_numel;
static PyObject *t_float32, *t_bfloat16, *t_e4m3, *t_e5m2, *t_e8m0, *t_int32; /* dtypes */
static PyObject *c_coded, *f_empty, *f_current, *f_stream;

static spec_status (*call_quantise)(const void *, int64_t, spec_dtype, const spec_coded *, int, void *);
static spec_status (*call_norm)(const void *, int64_t, spec_dtype, const void *, int64_t, spec_dtype, const void *,
                                spec_dtype, float, void *, int64_t, const spec_coded *, void *);
static spec_status (*call_gate)(const void *, int64_t, const void *, int64_t, spec_dtype, spec_act, const spec_coded *, void *);
static spec_status (*call_product)(const spec_coded *, const spec_coded *, void *, int64_t, spec_dtype, uint32_t *, void *);

/* A method's result as a number; -1 with an error set where it has none. */
static long long number_of(PyObject *t, PyObject *name)
{
    PyObject *r = PyObject_CallMethodNoArgs(t, name);
    if (!r)
        return -1;
    const long long v = (long long)PyLong_AsUnsignedLongLongMask(r);
    Py_DECREF(r);
    return v;
}

typedef struct {
    void *at;
    int64_t rows, dim, step;
    PyObject *dtype; /* borrowed: torch keeps its dtypes */
    PyObject *shape; /* owned */
} matrix;

static void drop(matrix *m) { Py_CLEAR(m->shape); }

/* A tensor of rows on device `index`, `size` bytes an element, rows beginning at multiples of `align` bytes; 0: not as usual. */
static int read_matrix(PyObject *t, long long index, int align, matrix *m)
{
    m->shape = NULL;
    m->dtype = PyObject_GetAttr(t, s_dtype);
    if (!m->dtype)
        return 0;
    Py_DECREF(m->dtype);
    const int size = m->dtype == t_float32 ? 4 : m->dtype == t_bfloat16 ? 2 : 1;
    if (size == 1 && m->dtype != t_e4m3 && m->dtype != t_e5m2 && m->dtype != t_e8m0)
        return 0;
    if (number_of(t, s_get_device) != index)
        return 0;
    m->at = (void *)(uintptr_t)number_of(t, s_data_ptr);
    m->shape = PyObject_GetAttr(t, s_shape);
    PyObject *dense = m->shape && !PyErr_Occurred() ? PyObject_CallMethodNoArgs(t, s_is_contiguous) : NULL;
    if (!dense)
        return 0;
    const int contiguous = dense == Py_True;
    Py_DECREF(dense);
    if (!PyTuple_Check(m->shape))
        return 0;
    const Py_ssize_t n = PyTuple_GET_SIZE(m->shape);
    if (n < 1)
        return 0;
    m->rows = 1;
    for (Py_ssize_t i = 0; i + 1 < n; ++i)
        m->rows *= PyLong_AsLongLong(PyTuple_GET_ITEM(m->shape, i));
    m->dim = m->step = PyLong_AsLongLong(PyTuple_GET_ITEM(m->shape, n - 1));
    if (!contiguous) {
        PyObject *stride = PyObject_CallMethodNoArgs(t, s_stride);
        if (!stride || !PyTuple_Check(stride) || PyTuple_GET_SIZE(stride) != n ||
            PyLong_AsLongLong(PyTuple_GET_ITEM(stride, n - 1)) != 1) {
            Py_XDECREF(stride);
            return 0;
        }
        int64_t below = 1;
        int known = 0, one = 1;
        for (Py_ssize_t i = n - 2; i >= 0; --i) {
            const int64_t size_i = PyLong_AsLongLong(PyTuple_GET_ITEM(m->shape, i)), step = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, i));
            if (size_i == 1)
                continue;
            if (!known)
                m->step = step;
            else if (step != m->step * below)
                one = 0;
            known = 1;
            below *= size_i;
        }
        Py_DECREF(stride);
        if (!one)
            return 0;
    }
    if (PyErr_Occurred() || m->rows < 1 || m->rows > SPEC_MAX_CODED_ROWS || m->dim < 1 || m->dim > SPEC_MAX_ROW || m->step < 0)
        return 0;
    return (((uintptr_t)m->at | (uintptr_t)(m->step * size)) & (uintptr_t)(align - 1)) == 0;
}

static int floating(const matrix *m, spec_dtype *type)
{
    *type = m->dtype == t_bfloat16 ? SPEC_BF16 : SPEC_F32;
    return m->dtype == t_bfloat16 || m->dtype == t_float32;
}

static int same_shape(const matrix *a, const matrix *b) { return PyObject_RichCompareBool(a->shape, b->shape, Py_EQ) == 1; }

/* The device of the first tensor of a call, if it is the current one; else -1. */
static long long device_of(PyObject *t)
{
    const long long index = number_of(t, s_get_device);
    if (index < 0 || PyErr_Occurred())
        return -1;
    PyObject *r = PyObject_CallNoArgs(f_current);
    if (!r)
        return -1;
    const long long current = PyLong_AsLongLong(r);
    Py_DECREF(r);
    return current == index ? index : -1;
}

static int stream_of(long long index, void **stream)
{
    PyObject *i = PyLong_FromLongLong(index), *r = i ? PyObject_CallOneArg(f_stream, i) : NULL;
    Py_XDECREF(i);
    if (!r)
        return 0;
    *stream = (void *)(uintptr_t)PyLong_AsUnsignedLongLongMask(r);
    Py_DECREF(r);
    return !PyErr_Occurred();
}

/* A new dense tensor of like's shape but for its last dimension (`last`), or, with above >= 0, of two dimensions. */
static PyObject *make(PyObject *like, int64_t above, int64_t last, PyObject *dtype, void **at)
{
    const Py_ssize_t n = above >= 0 ? 2 : PyTuple_GET_SIZE(like);
    PyObject *shape = PyTuple_New(n), *stride = PyTuple_New(n), *t = NULL;
    int64_t step = 1;
    for (Py_ssize_t i = n - 1; shape && stride && i >= 0; --i) {
        const int64_t size = i == n - 1 ? last : above >= 0 ? above : PyLong_AsLongLong(PyTuple_GET_ITEM(like, i));
        PyObject *a = PyLong_FromLongLong(size), *b = PyLong_FromLongLong(step);
        PyTuple_SET_ITEM(shape, i, a);
        PyTuple_SET_ITEM(stride, i, b);
        step *= size;
    }
    if (shape && stride && !PyErr_Occurred()) {
        PyObject *args[] = {shape, stride, dtype};
        t = PyObject_Vectorcall(f_empty, args, 3, NULL);
    }
    Py_XDECREF(shape);
    Py_XDECREF(stride);
    if (t) {
        *at = (void *)(uintptr_t)number_of(t, s_data_ptr);
        if (PyErr_Occurred())
            Py_CLEAR(t);
    }
    return t;
}

typedef struct {
    PyObject *codes, *scale;
    spec_coded c;
} output;

static int make_coded(const matrix *like, PyObject *code, int block_rows, output *o)
{
    const int64_t blocks = (like->dim + 127) / 128;
    void *scale = NULL;
    o->codes = o->scale = NULL;
    if ((code != t_e4m3 && code != t_e5m2) || like->dim % 16)
        return 0;
    o->codes = make(like->shape, -1, like->dim, code, &o->c.codes);
    o->scale = o->codes ? make(like->shape, block_rows == 1 ? -1 : (like->rows + 127) / 128, blocks, t_e8m0, &scale) : NULL;
    if (!o->scale)
        return 0;
    o->c.scale = scale;
    o->c.stride = like->dim;
    o->c.scale_stride = blocks;
    o->c.rows = (int32_t)like->rows;
    o->c.dim = (int32_t)like->dim;
    o->c.code = code == t_e4m3 ? SPEC_E4M3 : SPEC_E5M2;
    return 1;
}

/* The named tuple of an output, whose tensors it takes over. */
static PyObject *coded(output *o)
{
    PyObject *two = PyTuple_Pack(2, o->codes, o->scale), *args = two ? PyTuple_Pack(1, two) : NULL;
    PyObject *r = args ? PyTuple_Type.tp_new((PyTypeObject *)c_coded, args, NULL) : NULL;
    Py_XDECREF(two);
    Py_XDECREF(args);
    return r;
}

static void drop_output(output *o)
{
    Py_CLEAR(o->codes);
    Py_CLEAR(o->scale);
}

/* A call of the library, other threads running meanwhile (it may have to wait for room among the launches). */
#define WITHOUT_LOCK(status, call)  \
    do {                            \
        Py_BEGIN_ALLOW_THREADS      \
        (status) = (call);          \
        Py_END_ALLOW_THREADS        \
    } while (0)

/* What a call gives: the result, or None for all that is not as usual. */
static PyObject *finish(PyObject *r)
{
    if (r)
        return r;
    PyErr_Clear();
    Py_RETURN_NONE;
}

/* quantise(x, code, block_rows) */
static PyObject *py_quantise(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    PyObject *r = NULL;
    matrix x = {0};
    output o = {0};
    spec_dtype type;
    void *stream;
    const long long index = n == 3 ? device_of(args[0]) : -1;
    const long block = index >= 0 ? PyLong_AsLong(args[2]) : 0;
    if (index >= 0 && read_matrix(args[0], index, 16, &x) && floating(&x, &type) &&
        (block == 1 || PyTuple_GET_SIZE(x.shape) == 2) && make_coded(&x, args[1], (int)block, &o) && stream_of(index, &stream)) {
        spec_status status;
        WITHOUT_LOCK(status, call_quantise(x.at, x.step, type, &o.c, (int)block, stream));
        if (status == SPEC_OK)
            r = coded(&o);
    }
    drop(&x);
    drop_output(&o);
    return finish(r);
}

/* norm(x, weight or None, residual or None, eps, code) */
static PyObject *py_norm(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    PyObject *r = NULL, *sum = NULL;
    matrix x = {0}, w = {0}, res = {0};
    output o = {0};
    spec_dtype type, w_type = SPEC_F32, r_type = SPEC_F32;
    void *stream, *sum_at = NULL;
    const long long index = n == 5 ? device_of(args[0]) : -1;
    const double eps = index >= 0 ? PyFloat_AsDouble(args[3]) : 0.0;
    int ok = index >= 0 && eps >= 0x1p-126 && eps <= 3e38 && read_matrix(args[0], index, 16, &x) && floating(&x, &type) &&
             x.dim <= SPEC_MAX_NORM_ROW;
    if (ok && args[1] != Py_None)
        ok = read_matrix(args[1], index, 16, &w) && floating(&w, &w_type) && PyTuple_GET_SIZE(w.shape) == 1 && w.dim == x.dim;
    if (ok && args[2] != Py_None) {
        ok = read_matrix(args[2], index, 16, &res) && floating(&res, &r_type) && same_shape(&res, &x);
        if (ok)
            ok = (sum = make(x.shape, -1, x.dim, res.dtype, &sum_at)) != NULL;
    }
    spec_status status = SPEC_ERR_INVALID_ARG;
    if (ok && make_coded(&x, args[4], 1, &o) && stream_of(index, &stream))
        WITHOUT_LOCK(status, call_norm(x.at, x.step, type, res.at, res.step, r_type, w.at, w_type, (float)eps, sum_at, x.dim, &o.c, stream));
    if (status == SPEC_OK) {
        PyObject *c = coded(&o);
        r = c ? PyTuple_Pack(2, c, sum ? sum : Py_None) : NULL;
        Py_XDECREF(c);
    }
    Py_XDECREF(sum);
    drop(&x);
    drop(&w);
    drop(&res);
    drop_output(&o);
    return finish(r);
}

/* gate(gate, up, act, code) */
static PyObject *py_gate(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    PyObject *r = NULL;
    matrix g = {0}, u = {0};
    output o = {0};
    spec_dtype type;
    void *stream;
    const long long index = n == 4 ? device_of(args[0]) : -1;
    const long act = index >= 0 ? PyLong_AsLong(args[2]) : 0;
    if (index >= 0 && read_matrix(args[0], index, 16, &g) && floating(&g, &type) && read_matrix(args[1], index, 16, &u) &&
        u.dtype == g.dtype && same_shape(&u, &g) && make_coded(&g, args[3], 1, &o) && stream_of(index, &stream)) {
        spec_status status;
        WITHOUT_LOCK(status, call_gate(g.at, g.step, u.at, u.step, type, (spec_act)act, &o.c, stream));
        if (status == SPEC_OK)
            r = coded(&o);
    }
    drop(&g);
    drop(&u);
    drop_output(&o);
    return finish(r);
}

/* Codes and scales that a product reads; the codes' shape is kept in m. */
static int read_coded(PyObject *pair, long long index, int weight, matrix *m, spec_coded *c)
{
    matrix s = {0};
    if (!PyTuple_Check(pair) || PyTuple_GET_SIZE(pair) != 2 || !read_matrix(PyTuple_GET_ITEM(pair, 0), index, 16, m) ||
        (m->dtype != t_e4m3 && m->dtype != t_e5m2) || m->dim % 16 || m->step < m->dim)
        return 0;
    const int64_t blocks = (m->dim + 127) / 128;
    const Py_ssize_t n = PyTuple_GET_SIZE(m->shape);
    int ok = read_matrix(PyTuple_GET_ITEM(pair, 1), index, 1, &s) && s.dtype == t_e8m0 && s.dim == blocks && s.step >= blocks &&
             PyTuple_GET_SIZE(s.shape) == n;
    if (ok && weight)
        ok = n == 2 && s.rows == (m->rows + 127) / 128;
    for (Py_ssize_t i = 0; ok && !weight && i + 1 < n; ++i)
        ok = PyObject_RichCompareBool(PyTuple_GET_ITEM(s.shape, i), PyTuple_GET_ITEM(m->shape, i), Py_EQ) == 1;
    c->codes = m->at;
    c->scale = s.at;
    c->stride = m->step;
    c->scale_stride = s.step;
    c->rows = (int32_t)m->rows;
    c->dim = (int32_t)m->dim;
    c->code = m->dtype == t_e4m3 ? SPEC_E4M3 : SPEC_E5M2;
    drop(&s);
    return ok;
}

/* The address of a status word, or NULL for None; 0: not as usual. */
static int read_status(PyObject *t, long long index, uint32_t **at)
{
    *at = NULL;
    if (t == Py_None)
        return 1;
    PyObject *dtype = PyObject_GetAttr(t, s_dtype);
    if (!dtype)
        return 0;
    Py_DECREF(dtype);
    if (dtype != t_int32 || number_of(t, s_get_device) != index || number_of(t, s_numel) < 1 || PyErr_Occurred())
        return 0;
    PyObject *dense = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    Py_XDECREF(dense);
    if (dense != Py_True)
        return 0;
    *at = (uint32_t *)(uintptr_t)number_of(t, s_data_ptr);
    return !PyErr_Occurred();
}

/* product(rows, weight, dtype, status or None) */
static PyObject *py_product(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    PyObject *r = NULL, *out = NULL;
    matrix a = {0}, w = {0};
    spec_coded rows, weight;
    uint32_t *word;
    void *stream, *at;
    const long long index =
        n == 4 && PyTuple_Check(args[0]) && PyTuple_GET_SIZE(args[0]) == 2 ? device_of(PyTuple_GET_ITEM(args[0], 0)) : -1;
    if (index >= 0 && (args[2] == t_bfloat16 || args[2] == t_float32) && read_coded(args[0], index, 0, &a, &rows) &&
        read_coded(args[1], index, 1, &w, &weight) && a.dim == w.dim && read_status(args[3], index, &word) && (out = make(a.shape, -1, w.rows, args[2], &at)) &&
        stream_of(index, &stream)) {
        const spec_dtype type = args[2] == t_bfloat16 ? SPEC_BF16 : SPEC_F32;
        spec_status status;
        WITHOUT_LOCK(status, call_product(&rows, &weight, at, w.rows, type, word, stream));
        if (status == SPEC_OK)
            r = Py_NewRef(out);
    }
    Py_XDECREF(out);
    drop(&a);
    drop(&w);
    return finish(r);
}

/* setup((float32, bfloat16, e4m3, e5m2, e8m0, int32), Coded, empty, current, stream, (addresses of the four calls)) */
static PyObject *py_setup(PyObject *self, PyObject *args)
{
    (void)self;
    PyObject *types[6], *more[4];
    unsigned long long at[4];
    if (!PyArg_ParseTuple(args, "(OOOOOO)OOOO(KKKK)", &types[0], &types[1], &types[2], &types[3], &types[4], &types[5], &more[0], &more[1],
                          &more[2], &more[3], &at[0], &at[1], &at[2], &at[3]))
        return NULL;
    if (!PyType_Check(more[0]) || !PyType_IsSubtype((PyTypeObject *)more[0], &PyTuple_Type)) {
        PyErr_SetString(PyExc_TypeError, "Coded must be a named tuple");
        return NULL;
    }
    PyObject **const to[] = {&t_float32, &t_bfloat16, &t_e4m3, &t_e5m2, &t_e8m0, &t_int32, &c_coded, &f_empty, &f_current, &f_stream};
    for (int i = 0; i < 10; ++i)
        Py_XSETREF(*to[i], Py_NewRef(i < 6 ? types[i] : more[i - 6]));
    call_quantise = (spec_status(*)(const void *, int64_t, spec_dtype, const spec_coded *, int, void *))(uintptr_t)at[0];
    call_norm = (spec_status(*)(const void *, int64_t, spec_dtype, const void *, int64_t, spec_dtype, const void *, spec_dtype, float,
                                void *, int64_t, const spec_coded *, void *))(uintptr_t)at[1];
    call_gate = (spec_status(*)(const void *, int64_t, const void *, int64_t, spec_dtype, spec_act, const spec_coded *,
                                void *))(uintptr_t)at[2];
    call_product = (spec_status(*)(const spec_coded *, const spec_coded *, void *, int64_t, spec_dtype, uint32_t *,
                                   void *))(uintptr_t)at[3];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", py_setup, METH_VARARGS, "dtypes, the named tuple, torch's functions and the library's calls"},
    {"quantise", (PyCFunction)(void (*)(void))py_quantise, METH_FASTCALL, "quantise(x, code, block_rows): Coded or None"},
    {"norm", (PyCFunction)(void (*)(void))py_norm, METH_FASTCALL, "norm(x, weight, residual, eps, code): (Coded, sum) or None"},
    {"gate", (PyCFunction)(void (*)(void))py_gate, METH_FASTCALL, "gate(gate, up, act, code): Coded or None"},
    {"product", (PyCFunction)(void (*)(void))py_product, METH_FASTCALL, "product(rows, weight, dtype, status): the product or None"},
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "spec_rows_py", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_spec_rows_py(void)
{
    PyObject **const names[] = {&s_dtype, &s_shape, &s_get_device, &s_data_ptr, &s_is_contiguous, &s_stride, &s_numel};
    static const char *const text[] = {"dtype", "shape", "get_device", "data_ptr", "is_contiguous", "stride", "numel"};
    for (int i = 0; i < 7; ++i)
        if (!(*names[i] = PyUnicode_InternFromString(text[i])))
            return NULL;
    return PyModule_Create(&module);
}
