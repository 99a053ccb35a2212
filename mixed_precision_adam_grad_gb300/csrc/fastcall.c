/*
 * fastcall.c — CPython module `_fastcall`: the calls of the entry points that a
 * program makes for single tokens and small matrices, where marshalling a
 * dozen arguments through ctypes (6 us on a Grace core) costs more than the
 * kernel.  No behaviour of its own: it converts the arguments by the binding's
 * rules and calls the library's function, whose address the binding hands over
 * with bind() once the library is loaded, without the interpreter's lock: a
 * launch waits where the device's queue is full, and other threads run then.
 *   pointers: None, an int, or an object with data_ptr() or .ctypes.data
 *   structs:  a ctypes structure (its buffer)
 *   streams:  None, an int, or an object with .cuda_stream
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>

#include "slide.h"

static PyObject *s_data_ptr, *s_ctypes, *s_data, *s_cuda_stream;

enum { F_ROUTE, F_ROUTE_BACK, F_ROUTE_BIAS, F_ORTHO, F_MUON, F_COUNT };
static const char *const names[F_COUNT] = {"slide_route_experts", "slide_route_experts_backward", "slide_route_bias_step",
                                           "slide_orthogonalize", "slide_muon_step"};
static void *functions[F_COUNT];

static int to_i64(PyObject *o, int64_t *v)
{
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred())
        return 0;
    *v = x;
    return 1;
}

static int to_i32(PyObject *o, int32_t *v)
{
    int64_t x;
    if (!to_i64(o, &x))
        return 0;
    if (x < INT32_MIN || x > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "value does not fit in 32 bits");
        return 0;
    }
    *v = (int32_t)x;
    return 1;
}

static int to_ptr(PyObject *o, void **p)
{
    PyObject *r;
    if (o == Py_None) {
        *p = NULL;
        return 1;
    }
    if (PyLong_Check(o)) {
        *p = PyLong_AsVoidPtr(o);
        return !PyErr_Occurred();
    }
    r = PyObject_CallMethodNoArgs(o, s_data_ptr);
    if (!r) {
        PyObject *c;
        if (!PyErr_ExceptionMatches(PyExc_AttributeError))
            return 0;
        PyErr_Clear();
        c = PyObject_GetAttr(o, s_ctypes);
        r = c ? PyObject_GetAttr(c, s_data) : NULL;
        Py_XDECREF(c);
        if (!r) {
            PyErr_Format(PyExc_TypeError, "cannot take a pointer of %s", Py_TYPE(o)->tp_name);
            return 0;
        }
    }
    *p = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return !PyErr_Occurred();
}

static int to_stream(PyObject *o, slide_stream_t *s)
{
    PyObject *r;
    if (o == Py_None) {
        *s = NULL;
        return 1;
    }
    if (PyLong_Check(o)) {
        *s = (slide_stream_t)PyLong_AsVoidPtr(o);
        return !PyErr_Occurred();
    }
    r = PyObject_GetAttr(o, s_cuda_stream);
    if (!r)
        return 0;
    *s = (slide_stream_t)PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return !PyErr_Occurred();
}

/* The structure's bytes; the caller holds the object for the call. */
static int to_struct(PyObject *o, size_t size, const void **p)
{
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0)
        return 0;
    *p = b.buf;
    if ((size_t)b.len != size) {
        PyBuffer_Release(&b);
        PyErr_SetString(PyExc_TypeError, "structure of another size");
        return 0;
    }
    PyBuffer_Release(&b);
    return 1;
}

static int ready(int f, Py_ssize_t n, Py_ssize_t want)
{
    if (!functions[f]) {
        PyErr_Format(PyExc_RuntimeError, "%s is not bound", names[f]);
        return 0;
    }
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%s: %zd arguments expected", names[f], want);
        return 0;
    }
    return 1;
}

static PyObject *bind(PyObject *self, PyObject *args)
{
    const char *name;
    unsigned long long at;
    int f;
    (void)self;
    if (!PyArg_ParseTuple(args, "sK", &name, &at))
        return NULL;
    for (f = 0; f < F_COUNT; ++f) {
        if (strcmp(name, names[f]) == 0) {
            functions[f] = (void *)(uintptr_t)at;
            Py_RETURN_NONE;
        }
    }
    PyErr_Format(PyExc_ValueError, "unknown entry point %s", name);
    return NULL;
}

static PyObject *route_experts(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int64_t tokens, stride;
    int32_t type;
    void *logits, *bias, *mask, *w, *e, *load;
    const void *cfg;
    slide_stream_t s;
    slide_status rc;
    (void)self;
    if (!ready(F_ROUTE, n, 11) || !to_i64(a[0], &tokens) || !to_ptr(a[1], &logits) || !to_i32(a[2], &type) ||
        !to_i64(a[3], &stride) || !to_ptr(a[4], &bias) || !to_ptr(a[5], &mask) ||
        !to_struct(a[6], sizeof(slide_route_config), &cfg) || !to_ptr(a[7], &w) || !to_ptr(a[8], &e) ||
        !to_ptr(a[9], &load) || !to_stream(a[10], &s))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    rc = ((__typeof__(slide_route_experts) *)functions[F_ROUTE])(tokens, logits, type, stride, bias, mask, cfg, w,
         e, load, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject *route_experts_backward(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int64_t tokens, stride, d_stride;
    int32_t type;
    void *logits, *e, *dw, *mask, *dx;
    const void *cfg;
    slide_stream_t s;
    slide_status rc;
    (void)self;
    if (!ready(F_ROUTE_BACK, n, 11) || !to_i64(a[0], &tokens) || !to_ptr(a[1], &logits) || !to_i32(a[2], &type) ||
        !to_i64(a[3], &stride) || !to_ptr(a[4], &e) || !to_ptr(a[5], &dw) || !to_ptr(a[6], &mask) ||
        !to_struct(a[7], sizeof(slide_route_config), &cfg) || !to_ptr(a[8], &dx) || !to_i64(a[9], &d_stride) ||
        !to_stream(a[10], &s))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    rc = ((__typeof__(slide_route_experts_backward) *)functions[F_ROUTE_BACK])(tokens, logits, type, stride, e, dw,
         mask, cfg, dx, d_stride, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject *route_bias_step(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int32_t experts;
    void *load, *bias;
    double rate;
    slide_stream_t s;
    slide_status rc;
    (void)self;
    if (!ready(F_ROUTE_BIAS, n, 5) || !to_i32(a[0], &experts) || !to_ptr(a[1], &load) || !to_ptr(a[2], &bias))
        return NULL;
    rate = PyFloat_AsDouble(a[3]);
    if ((rate == -1.0 && PyErr_Occurred()) || !to_stream(a[4], &s))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    rc = ((__typeof__(slide_route_bias_step) *)functions[F_ROUTE_BIAS])(experts, load, bias, (float)rate, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject *orthogonalize(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int32_t batch, rows, cols, type;
    int64_t xr, xb, outr, outb, bytes;
    void *x, *out, *ws;
    const void *params;
    slide_stream_t s;
    slide_status rc;
    (void)self;
    if (!ready(F_ORTHO, n, 14) || !to_i32(a[0], &batch) || !to_i32(a[1], &rows) || !to_i32(a[2], &cols) ||
        !to_ptr(a[3], &x) || !to_i32(a[4], &type) || !to_i64(a[5], &xr) || !to_i64(a[6], &xb) || !to_ptr(a[7], &out) ||
        !to_i64(a[8], &outr) || !to_i64(a[9], &outb) || !to_struct(a[10], sizeof(slide_ortho_params), &params) ||
        !to_ptr(a[11], &ws) || !to_i64(a[12], &bytes) || !to_stream(a[13], &s))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    rc = ((__typeof__(slide_orthogonalize) *)functions[F_ORTHO])(batch, rows, cols, x, type, xr, xb, out, outr,
         outb, params, ws, bytes, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject *muon_step(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    int32_t batch, rows, cols, type;
    int64_t bytes;
    void *th, *mom, *w, *ws;
    const void *grads[SLIDE_MAX_REPLICAS] = {0}, *hp;
    slide_stream_t s;
    slide_status rc;
    PyObject *seq;
    Py_ssize_t r, count;
    (void)self;
    if (!ready(F_MUON, n, 12) || !to_i32(a[0], &batch) || !to_i32(a[1], &rows) || !to_i32(a[2], &cols))
        return NULL;
    seq = PySequence_Fast(a[3], "grad_replicas is not a sequence");
    if (!seq)
        return NULL;
    count = PySequence_Fast_GET_SIZE(seq);
    for (r = 0; r < count && r < SLIDE_MAX_REPLICAS; ++r) {  /* the library refuses more */
        if (!to_ptr(PySequence_Fast_GET_ITEM(seq, r), (void **)&grads[r])) {
            Py_DECREF(seq);
            return NULL;
        }
    }
    Py_DECREF(seq);
    if (!to_i32(a[4], &type) || !to_ptr(a[5], &th) || !to_ptr(a[6], &mom) || !to_ptr(a[7], &w) ||
        !to_struct(a[8], sizeof(slide_muon_hparams), &hp) || !to_ptr(a[9], &ws) || !to_i64(a[10], &bytes) ||
        !to_stream(a[11], &s))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    rc = ((__typeof__(slide_muon_step) *)functions[F_MUON])(batch, rows, cols, count > INT32_MAX ? INT32_MAX :
         (int32_t)count, grads, type, th, mom, w, hp, ws, bytes, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "bind(name, address)"},
    {"route_experts", (PyCFunction)(void (*)(void))route_experts, METH_FASTCALL, NULL},
    {"route_experts_backward", (PyCFunction)(void (*)(void))route_experts_backward, METH_FASTCALL, NULL},
    {"route_bias_step", (PyCFunction)(void (*)(void))route_bias_step, METH_FASTCALL, NULL},
    {"orthogonalize", (PyCFunction)(void (*)(void))orthogonalize, METH_FASTCALL, NULL},
    {"muon_step", (PyCFunction)(void (*)(void))muon_step, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void)
{
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_ctypes = PyUnicode_InternFromString("ctypes");
    s_data = PyUnicode_InternFromString("data");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!s_data_ptr || !s_ctypes || !s_data || !s_cuda_stream)
        return NULL;
    return PyModule_Create(&module);
}
