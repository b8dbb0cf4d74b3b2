/* bind.c - the Python side of the calls that sit between a layer's larger
 * kernels (routing, norms, 8-bit products).  Their GPU work is a few
 * microseconds, so marshalling counts: one native call checks the operands,
 * takes their addresses and calls the library, where ctypes and checks in
 * Python took 7 us a call.
 *
 * call(index, arg, ...): an argument is a whole number, None (0) or an operand,
 * a tuple of a name, a tensor or an address or None, a kind, and what the call
 * reads or writes:
 *   (name, t, kind, rows, cols): rows * cols elements without a gap;
 *   (name, t, kind, rows, cols, ld, whole): rows of cols elements that start ld
 *   elements apart, of which memory holds `whole` (what stands behind cols does
 *   not count).
 * A tensor is one of the current CUDA device and of the kind's type, and has
 * those elements where the call expects them.  A raw device address is the
 * caller's word.  A failed check or call raises HfqError.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <stdint.h>

#include "hfq4moe.h"

#define MAX_ARGS 24
#define MAX_KINDS 8

static PyObject *g_error, *g_tensor, *g_get_device, *g_layout, *g_kinds[MAX_KINDS];
static PyObject *s_shape, *s_dtype, *s_get_device, *s_is_contiguous, *s_numel, *s_data_ptr;

typedef int64_t V;
#define P(i) ((void *)(uintptr_t)v[i])
#define I(i) ((int)v[i])
#define Z(i) ((size_t)v[i])

static hfq_status do_route(const V *v)
{
    return moe_route_scored(P(0), (hfq_dtype)I(1), I(2), I(3), I(4), P(5), P(6), I(7), P(8), P(9), P(10), P(11), P(12),
                            P(13), Z(14), P(15));
}

static hfq_status do_norm(const V *v)
{
    return moe_norm_residual(P(0), I(1), I(2), P(3), (hfq_dtype)I(4), I(5), P(6), P(7), (hfq_dtype)I(8), I(9), P(10),
                             P(11), P(12), P(13), (hfq_dtype)I(14), P(15), P(16), P(17));
}

static hfq_status do_quantize(const V *v)
{
    return q8_quantize_rows(P(0), (hfq_dtype)I(1), I(2), I(3), I(4), I(5), P(6), I(7), P(8), P(9));
}

static hfq_status do_matmul(const V *v)
{
    return q8_matmul(P(0), I(1), P(2), I(3), I(4), P(5), I(6), P(7), I(8), P(9), (hfq_dtype)I(10), I(11), P(12));
}

static hfq_status do_linear(const V *v)
{
    return q8_linear(P(0), (hfq_dtype)I(1), I(2), I(3), I(4), P(5), I(6), P(7), I(8), P(9), (hfq_dtype)I(10), I(11), P(12),
                     Z(13), P(14));
}

/* argument types: p pointer, i int, z size_t */
static const struct {
    const char *sig;
    hfq_status (*fn)(const V *);
} g_calls[] = {
    {"piiiippippppppzp", do_route}, {"piipiippiippppippp", do_norm}, {"piiiiipipp", do_quantize},
    {"pipiipipipiip", do_matmul},   {"piiiipipipiipzp", do_linear},
};

static int fail_arg(PyObject *name, const char *why)
{
    PyObject *msg = PyUnicode_FromFormat("%U %s", name, why);
    PyObject *args = msg ? Py_BuildValue("(iN)", (int)HFQ_ERR_ARG, msg) : NULL;
    if (args) {
        PyErr_SetObject(g_error, args);
        Py_DECREF(args);
    }
    return -1;
}

static int to_word(PyObject *o, V *v)
{
    *v = PyLong_AsLongLong(o);
    if (*v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        *v = (V)PyLong_AsUnsignedLongLong(o);
        if (PyErr_Occurred()) return -1;
    }
    return 0;
}

/* The whole number that a method without arguments returns. */
static int ask(PyObject *t, PyObject *method, V *v)
{
    PyObject *r = PyObject_CallMethodNoArgs(t, method);
    if (!r) return -1;
    const int st = to_word(r, v);
    Py_DECREF(r);
    return st;
}

static int out_of_range(void)
{
    PyObject *name = PyUnicode_FromString("a size");
    if (name) {
        fail_arg(name, "is out of range");
        Py_DECREF(name);
    }
    return -1;
}

static int operand(PyObject *op, V *v, V *device)
{
    const Py_ssize_t parts = PyTuple_GET_SIZE(op);
    if (parts != 5 && parts != 7) {
        PyErr_SetString(PyExc_TypeError, "an operand is (name, tensor, kind, rows, cols) or (.., rows, cols, ld, whole)");
        return -1;
    }
    PyObject *name = PyTuple_GET_ITEM(op, 0), *t = PyTuple_GET_ITEM(op, 1);
    if (t == Py_None) {
        *v = 0;
        return 0;
    }
    if (PyLong_Check(t)) return to_word(t, v);
    if (!g_tensor || !PyObject_TypeCheck(t, (PyTypeObject *)g_tensor))
        return fail_arg(name, "is neither a tensor of the current CUDA device nor a device address");
    V on = -1, numel = 0, size[4] = {0, 0, 0, 0};        /* rows, cols, ld, whole */
    if (ask(t, s_get_device, &on)) return -1;
    if (on >= 0 && *device < 0) {
        PyObject *r = PyObject_CallNoArgs(g_get_device);
        if (!r) return -1;
        const int st = to_word(r, device);
        Py_DECREF(r);
        if (st) return -1;
    }
    if (on < 0 || on != *device)
        return fail_arg(name, "is neither a tensor of the current CUDA device nor a device address");
    const long kind = PyLong_AsLong(PyTuple_GET_ITEM(op, 2));
    if (kind == -1 && PyErr_Occurred()) return -1;
    PyObject *dtype = PyObject_GetAttr(t, s_dtype);
    if (!dtype) return -1;
    int known = 0;
    if (kind >= 0 && kind < MAX_KINDS && g_kinds[kind])
        for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(g_kinds[kind]); ++i)
            known |= PyTuple_GET_ITEM(g_kinds[kind], i) == dtype;
    Py_DECREF(dtype);
    if (!known) return fail_arg(name, "has another type than the call names");
    for (Py_ssize_t i = 0; i < parts - 3; ++i) {
        if (to_word(PyTuple_GET_ITEM(op, 3 + i), &size[i])) return -1;
        if (size[i] < INT_MIN || size[i] > INT_MAX) return out_of_range();
    }
    PyObject *dense = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!dense) return -1;
    const int is_dense = dense == Py_True;
    Py_DECREF(dense);
    if (ask(t, s_numel, &numel)) return -1;
    const V rows = size[0], cols = size[1], ld = size[2], whole = size[3];
    if (parts == 5) {
        if (!is_dense) return fail_arg(name, "has gaps between its elements, which the call takes as neighbours");
        if (rows > 0 && cols > 0 && numel < rows * cols)
            return fail_arg(name, "holds fewer elements than the call reads or writes");
    } else if (rows > 0 && cols > 0 && ld >= cols) {     /* else the library refuses the sizes */
        int plain = is_dense && numel == rows * ld && whole <= ld;
        if (!plain && is_dense && numel >= (rows - 1) * ld + whole) {
            PyObject *shape = PyObject_GetAttr(t, s_shape);
            if (!shape) return -1;
            const Py_ssize_t n = PyTuple_Check(shape) ? PyTuple_GET_SIZE(shape) : 0;
            V last = 0;
            const int st = n > 0 ? to_word(PyTuple_GET_ITEM(shape, n - 1), &last) : 0;
            Py_DECREF(shape);
            if (st) return -1;
            plain = n == 1 || last == ld;                /* a flat buffer, or rows of ld elements */
        }
        if (!plain) {
            PyObject *r = PyObject_CallFunction(g_layout, "OOLLLL", name, t, (long long)rows, (long long)cols,
                                                (long long)ld, (long long)whole);
            if (!r) return -1;
            Py_DECREF(r);
        }
    }
    return ask(t, s_data_ptr, v);
}

static PyObject *call(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    (void)self;
    const long which = n > 0 ? PyLong_AsLong(args[0]) : -1;
    if (which < 0 || which >= (long)(sizeof g_calls / sizeof g_calls[0]) ||
        n - 1 != (Py_ssize_t)strlen(g_calls[which].sig) || n - 1 > MAX_ARGS) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "call(index, arguments of that call)");
        return NULL;
    }
    V v[MAX_ARGS], device = -1;
    for (Py_ssize_t i = 0; i < n - 1; ++i) {
        PyObject *a = args[i + 1];
        if (a == Py_None) v[i] = 0;
        else if (PyTuple_CheckExact(a)) {
            if (operand(a, &v[i], &device)) return NULL;
        } else {
            PyObject *w = PyNumber_Index(a);     /* numpy's whole numbers, too */
            if (!w) return NULL;
            const int st = to_word(w, &v[i]);
            Py_DECREF(w);
            if (st) return NULL;
            if (g_calls[which].sig[i] == 'i' && (v[i] < INT_MIN || v[i] > INT_MAX)) {
                out_of_range();
                return NULL;
            }
        }
    }
    hfq_status st;
    Py_BEGIN_ALLOW_THREADS                       /* a launch waits where a stream's queue is full */
    st = g_calls[which].fn(v);
    Py_END_ALLOW_THREADS
    if (st != HFQ_OK) {
        PyObject *e = Py_BuildValue("(is)", (int)st, hfq_last_error());
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
        return NULL;
    }
    Py_RETURN_NONE;
}

/* setup(error, check of a matrix' layout, torch.Tensor or None, current device's call, {kind: (dtypes)}) */
static PyObject *setup(PyObject *self, PyObject *args)
{
    (void)self;
    PyObject *error, *layout, *tensor, *get_device, *kinds;
    if (!PyArg_ParseTuple(args, "OOOOO!", &error, &layout, &tensor, &get_device, &PyDict_Type, &kinds)) return NULL;
    if (tensor != Py_None && !PyType_Check(tensor)) {
        PyErr_SetString(PyExc_TypeError, "setup: a tensor type or None");
        return NULL;
    }
    Py_XSETREF(g_error, Py_NewRef(error));
    Py_XSETREF(g_layout, Py_NewRef(layout));
    Py_XSETREF(g_tensor, tensor == Py_None ? NULL : Py_NewRef(tensor));
    Py_XSETREF(g_get_device, Py_NewRef(get_device));
    PyObject *k, *d;
    Py_ssize_t pos = 0;
    while (PyDict_Next(kinds, &pos, &k, &d)) {
        const long i = PyLong_AsLong(k);
        if (i < 0 || i >= MAX_KINDS || !PyTuple_Check(d)) {
            PyErr_SetString(PyExc_ValueError, "setup: a kind");
            return NULL;
        }
        Py_XSETREF(g_kinds[i], Py_NewRef(d));
    }
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"call", (PyCFunction)(void (*)(void))call, METH_FASTCALL, "call(index, arguments): a checked call of the library"},
    {"setup", setup, METH_VARARGS, "setup(error, layout, tensor, get_device, kinds)"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__bind(void)
{
    s_dtype = PyUnicode_InternFromString("dtype");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_numel = PyUnicode_InternFromString("numel");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_shape = PyUnicode_InternFromString("shape");
    if (!s_shape || !s_dtype || !s_get_device || !s_is_contiguous || !s_numel || !s_data_ptr) return NULL;
    return PyModule_Create(&module);
}
