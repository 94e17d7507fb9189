/* Calls of the paged-cache functions from Python without ctypes.

   These calls take ten pointers and more and are made several times per layer
   and token, where the host's time counts: ctypes and the address of every
   tensor in Python come to about 3 us of a call, this module's arguments to
   about 1 us (2 us are the launch).  It marshals arguments and nothing else:
   tensors by their data_ptr(), None as a null pointer, integers as addresses,
   the parameter structs by their buffers, each of the class that types() was
   given for it (two of them are of one size).  The functions' own addresses
   come from the loaded library. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "fadkv.h"

static PyObject* s_data_ptr;
enum { PAGE, QK, ROPE, PAGED, TYPES };
static PyTypeObject* s_types[TYPES];

/* types(PageParams, QkParams, Rope, PagedParams): the structs' classes. */
static PyObject* types(PyObject* self, PyObject* const* args, Py_ssize_t n)
{
    (void)self;
    for (Py_ssize_t i = 0; i < n; ++i)
        if (n != TYPES || !PyType_Check(args[i])) n = -1;
    if (n != TYPES) {
        PyErr_SetString(PyExc_TypeError, "four classes wanted");
        return NULL;
    }
    for (int i = 0; i < TYPES; ++i) {
        Py_INCREF(args[i]);
        Py_XDECREF((PyObject*)s_types[i]);
        s_types[i] = (PyTypeObject*)args[i];
    }
    Py_RETURN_NONE;
}

/* Address of a tensor, an integer or None; 0 on success. */
static int address(PyObject* o, void** out)
{
    if (o == Py_None) {
        *out = NULL;
        return 0;
    }
    if (PyLong_Check(o)) {
        *out = PyLong_AsVoidPtr(o);
        return PyErr_Occurred() ? -1 : 0;
    }
    PyObject* r = PyObject_CallMethodNoArgs(o, s_data_ptr);
    if (!r) return -1;
    *out = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return PyErr_Occurred() ? -1 : 0;
}

/* The bytes of a struct of the expected class and size; null for None. */
static int structure(PyObject* o, int type, size_t size, const void** out)
{
    Py_buffer b;
    if (o == Py_None) {
        *out = NULL;
        return 0;
    }
    if (!s_types[type] || !PyObject_TypeCheck(o, s_types[type])) {
        PyErr_SetString(PyExc_TypeError, "wrong parameter struct");
        return -1;
    }
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) return -1;
    *out = b.buf;
    const int ok = (size_t)b.len == size;
    PyBuffer_Release(&b);       /* the caller's reference keeps the struct */
    if (!ok) PyErr_SetString(PyExc_TypeError, "wrong parameter struct");
    return ok ? 0 : -1;
}

static int pointers(PyObject* const* args, Py_ssize_t n, void** out)
{
    for (Py_ssize_t i = 0; i < n; ++i)
        if (address(args[i], &out[i]) != 0) return -1;
    return 0;
}

static int arity(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return 0;
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
    return -1;
}

/* (function, params, 11 arrays, stream) */
static PyObject* page_plan(PyObject* self, PyObject* const* args, Py_ssize_t n)
{
    void *f, *p[12];
    const void* params;
    (void)self;
    if (arity(n, 14) || address(args[0], &f) || structure(args[1], PAGE, sizeof(fadkv_page_params), &params) ||
        pointers(args + 2, 12, p))
        return NULL;
    __typeof__(&fadkv_page_plan) call = (__typeof__(&fadkv_page_plan))f;
    fadkv_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call(params, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11]);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* (function, params, rope, 11 arrays, stream) */
static PyObject* qk_norm_rope(PyObject* self, PyObject* const* args, Py_ssize_t n)
{
    void *f, *p[12];
    const void *params, *rope;
    (void)self;
    if (arity(n, 15) || address(args[0], &f) || structure(args[1], QK, sizeof(fadkv_qk_params), &params) ||
        structure(args[2], ROPE, sizeof(fadkv_rope), &rope) || pointers(args + 3, 12, p))
        return NULL;
    __typeof__(&fadkv_qk_norm_rope) call = (__typeof__(&fadkv_qk_norm_rope))f;
    fadkv_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call(params, rope, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11]);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* (function, params, 8 arrays, workspace, bytes, stream) */
static PyObject* paged_attend(PyObject* self, PyObject* const* args, Py_ssize_t n)
{
    void *f, *p[9], *st;
    const void* params;
    (void)self;
    if (arity(n, 13) || address(args[0], &f) || structure(args[1], PAGED, sizeof(fadkv_paged_params), &params) ||
        pointers(args + 2, 9, p) || address(args[12], &st))
        return NULL;
    const size_t bytes = PyLong_AsSize_t(args[11]);
    if (PyErr_Occurred()) return NULL;
    __typeof__(&fadkv_paged_attend_planned) call = (__typeof__(&fadkv_paged_attend_planned))f;
    fadkv_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call(params, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], bytes, st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* (function, params, 9 arrays, workspace, bytes, stream) */
static PyObject* paged_prefill(PyObject* self, PyObject* const* args, Py_ssize_t n)
{
    void *f, *p[10], *st;
    const void* params;
    (void)self;
    if (arity(n, 14) || address(args[0], &f) || structure(args[1], PAGED, sizeof(fadkv_paged_params), &params) ||
        pointers(args + 2, 10, p) || address(args[13], &st))
        return NULL;
    const size_t bytes = PyLong_AsSize_t(args[12]);
    if (PyErr_Occurred()) return NULL;
    __typeof__(&fadkv_paged_prefill_planned) call = (__typeof__(&fadkv_paged_prefill_planned))f;
    fadkv_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call(params, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], bytes, st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyMethodDef methods[] = {
    {"types", (PyCFunction)(void (*)(void))types, METH_FASTCALL, NULL},
    {"page_plan", (PyCFunction)(void (*)(void))page_plan, METH_FASTCALL, NULL},
    {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, NULL},
    {"paged_attend", (PyCFunction)(void (*)(void))paged_attend, METH_FASTCALL, NULL},
    {"paged_prefill", (PyCFunction)(void (*)(void))paged_prefill, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fadkv_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fadkv_calls(void)
{
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    return s_data_ptr ? PyModule_Create(&module) : NULL;
}
