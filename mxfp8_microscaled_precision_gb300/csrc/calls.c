/*
 * calls.c -- the calls of libmxq that run in every decoding step (mxq.h, operators
 * around the experts' products) as a CPython extension module.  It marshals arguments
 * only: every argument is an integer (an address, a size, an enum) or None for a null
 * pointer, or a float; every function returns the call's status.  A foreign call
 * of 13 to 18 arguments through ctypes costs 2 to 3 us on the GB300's host, twice
 * the launch itself needs; this one costs a tenth of that.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "mxq.h"

#define MOST 20

/* args[0 .. n) as integers in v (None: 0), where floats is a mask of the positions that hold floats, in f. */
static int take(const char* name, PyObject* const* args, Py_ssize_t given, int n, unsigned floats, long long* v,
                float* f) {
    if (given != n) {
        PyErr_Format(PyExc_TypeError, "%s takes %d arguments, not %zd", name, n, given);
        return 0;
    }
    for (int i = 0; i < n; ++i) {
        if ((floats >> i) & 1u) {
            const double d = PyFloat_AsDouble(args[i]);
            if (d == -1.0 && PyErr_Occurred()) return 0;
            f[i] = (float)d;
        } else if (args[i] == Py_None) {
            v[i] = 0;
        } else {
            v[i] = PyLong_AsLongLong(args[i]);
            if (v[i] == -1 && PyErr_Occurred()) return 0;
        }
    }
    return 1;
}

#define PTR(i) ((void*)(intptr_t)v[i])
#define STREAM(i) ((mxq_stream_t)(intptr_t)v[i])
/* An enum or int32 out of its range must not come out valid: the library refuses INT32_MIN. */
#define INT(i) (v[i] < INT32_MIN || v[i] > INT32_MAX ? INT32_MIN : (int32_t)v[i])

#define CALL(name, n, floats, expression)                                                      \
    static PyObject* py_##name(PyObject* self, PyObject* const* args, Py_ssize_t given) {      \
        long long v[MOST];                                                                     \
        float f[MOST];                                                                         \
        (void)self, (void)f;                                                                   \
        if (!take(#name, args, given, n, floats, v, f)) return NULL;                           \
        return PyLong_FromLong((long)(expression));                                            \
    }

CALL(route, 17, 1u << 13,
     mxq_route(PTR(0), INT(1), v[2], INT(3), v[4], PTR(5), PTR(6), INT(7), INT(8), INT(9), INT(10), INT(11), INT(12),
               f[13], PTR(14), PTR(15), STREAM(16)))
CALL(route_backward, 14, 1u << 10,
     mxq_route_backward(PTR(0), PTR(1), PTR(2), INT(3), v[4], INT(5), v[6], INT(7), INT(8), INT(9), f[10], PTR(11),
                        v[12], STREAM(13)))
CALL(moe_plan, 7, 0, mxq_moe_plan(PTR(0), v[1], INT(2), INT(3), PTR(4), PTR(5), STREAM(6)))
CALL(moe_dispatch, 10, 0,
     mxq_moe_dispatch(PTR(0), INT(1), v[2], INT(3), v[4], v[5], PTR(6), PTR(7), v[8], STREAM(9)))
CALL(moe_combine, 11, 0,
     mxq_moe_combine(PTR(0), INT(1), v[2], INT(3), v[4], v[5], PTR(6), PTR(7), PTR(8), v[9], STREAM(10)))
CALL(moe_combine_backward, 14, 0,
     mxq_moe_combine_backward(PTR(0), PTR(1), INT(2), v[3], INT(4), v[5], v[6], v[7], PTR(8), PTR(9), PTR(10), v[11],
                              PTR(12), STREAM(13)))
CALL(layer_norm, 14, 1u << 8,
     mxq_layer_norm(PTR(0), INT(1), v[2], v[3], v[4], PTR(5), PTR(6), INT(7), f[8], PTR(9), v[10], PTR(11), PTR(12),
                    STREAM(13)))
CALL(layer_norm_backward, 18, 0,
     mxq_layer_norm_backward(PTR(0), PTR(1), INT(2), v[3], v[4], v[5], v[6], PTR(7), INT(8), PTR(9), PTR(10), PTR(11),
                             v[12], PTR(13), PTR(14), PTR(15), v[16] < 0 ? 0 : (size_t)v[16], STREAM(17)))
CALL(layer_norm_backward_workspace_size, 2, 0, mxq_layer_norm_backward_workspace_size(v[0], v[1]))
CALL(grad_norm_workspace_size, 1, 0, mxq_grad_norm_workspace_size(INT(0)))

static PyObject *s_dtype, *s_is_cuda, *s_is_contiguous, *s_numel, *s_data_ptr;

/* t.name() as an integer; -1 with an error set otherwise. */
static long long method_int(PyObject* t, PyObject* name) {
    PyObject* r = PyObject_CallMethodNoArgs(t, name);
    if (r == NULL) return -1;
    const long long v = PyLong_AsLongLong(r);
    Py_DECREF(r);
    return v;
}

/* 1 if t is a contiguous CUDA tensor of dtype bf16 or f32 (its code in *code), 0 if not, -1 on an error. */
static int plain_tensor(PyObject* t, PyObject* bf16, PyObject* f32, int* code) {
    PyObject* r = PyObject_GetAttr(t, s_dtype);
    if (r == NULL) return -1;
    *code = r == bf16 ? MXQ_BF16 : MXQ_F32;
    const int known = r == bf16 || r == f32;
    Py_DECREF(r);
    if (!known) return 0;
    r = PyObject_GetAttr(t, s_is_cuda);
    if (r == NULL) return -1;
    const int cuda = r == Py_True;
    Py_DECREF(r);
    if (!cuda) return 0;
    r = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (r == NULL) return -1;
    const int yes = r == Py_True;
    Py_DECREF(r);
    return yes;
}

/*
 * grad_descs(grads, outs, torch.bfloat16, torch.float32): the mxq_grad_desc array of two
 * lists of tensors (outs may be grads itself) as a bytes object.  ValueError for a tensor that the
 * calls cannot take or an output unlike its gradient.
 */
static PyObject* grad_descs(PyObject* self, PyObject* const* args, Py_ssize_t given) {
    (void)self;
    if (given != 4 || !PyList_Check(args[0]) || !PyList_Check(args[1])) {
        PyErr_SetString(PyExc_TypeError, "grad_descs takes two lists and two dtypes");
        return NULL;
    }
    const Py_ssize_t n = PyList_GET_SIZE(args[0]);
    if (PyList_GET_SIZE(args[1]) != n) {
        PyErr_SetString(PyExc_ValueError, "out must have a tensor for every gradient");
        return NULL;
    }
    PyObject* bytes = PyBytes_FromStringAndSize(NULL, (n > 0 ? n : 1) * (Py_ssize_t)sizeof(mxq_grad_desc));
    if (bytes == NULL) return NULL;
    mxq_grad_desc* d = (mxq_grad_desc*)PyBytes_AS_STRING(bytes);
    for (Py_ssize_t i = 0; i < n; ++i) {
        /* the lists are the caller's own copies; a method of a tensor cannot shorten them */
        PyObject *g = PyList_GET_ITEM(args[0], i), *o = PyList_GET_ITEM(args[1], i);
        int code = 0, out_code = 0;
        int ok = plain_tensor(g, args[2], args[3], &code);
        if (ok == 0) PyErr_SetString(PyExc_ValueError, "gradients must be contiguous bfloat16 or float32 CUDA tensors");
        if (ok <= 0) goto fail;
        d[i].numel = method_int(g, s_numel);
        if (d[i].numel == -1 && PyErr_Occurred()) goto fail;
        d[i].grad = (const void*)(intptr_t)method_int(g, s_data_ptr);
        if (PyErr_Occurred()) goto fail;
        d[i].out = (void*)d[i].grad;
        d[i].dtype = code == MXQ_F32 ? MXQ_F32 : MXQ_BF16;
        if (o == g) continue;
        ok = plain_tensor(o, args[2], args[3], &out_code);
        if (ok < 0) goto fail;
        const long long size = method_int(o, s_numel);
        if (size == -1 && PyErr_Occurred()) goto fail;
        if (ok == 0 || out_code != code || size != d[i].numel) {
            PyErr_SetString(PyExc_ValueError, "every output must be a contiguous tensor like its gradient");
            goto fail;
        }
        d[i].out = (void*)(intptr_t)method_int(o, s_data_ptr);
        if (PyErr_Occurred()) goto fail;
    }
    return bytes;
fail:
    Py_DECREF(bytes);
    return NULL;
}

/* The descriptors at args[0] (the bytes of grad_descs). */
static const mxq_grad_desc* descs_of(PyObject* o, long long count) {
    if (!PyBytes_Check(o) || count < 0 || PyBytes_GET_SIZE(o) < count * (long long)sizeof(mxq_grad_desc)) {
        PyErr_SetString(PyExc_TypeError, "the descriptors of grad_descs are wanted");
        return NULL;
    }
    return (const mxq_grad_desc*)PyBytes_AS_STRING(o);
}

/* (descs, count, norm, workspace, workspace bytes, stream) */
static PyObject* py_grad_norm(PyObject* self, PyObject* const* args, Py_ssize_t given) {
    long long v[MOST];
    float f[MOST];
    (void)self;
    if (given < 1 || !take("grad_norm", args + 1, given - 1, 5, 0, v, f)) return NULL;
    const mxq_grad_desc* d = descs_of(args[0], v[0]);
    if (d == NULL) return NULL;
    return PyLong_FromLong((long)mxq_grad_norm(d, INT(0), PTR(1), PTR(2), v[3] < 0 ? 0 : (size_t)v[3], STREAM(4)));
}

/* (descs, count, max_norm, eps, norm, workspace, workspace bytes, stream) */
static PyObject* py_clip_grad_norm(PyObject* self, PyObject* const* args, Py_ssize_t given) {
    long long v[MOST];
    float f[MOST];
    (void)self;
    if (given < 1 || !take("clip_grad_norm", args + 1, given - 1, 7, (1u << 1) | (1u << 2), v, f)) return NULL;
    const mxq_grad_desc* d = descs_of(args[0], v[0]);
    if (d == NULL) return NULL;
    return PyLong_FromLong(
        (long)mxq_clip_grad_norm(d, INT(0), f[1], f[2], PTR(3), PTR(4), v[5] < 0 ? 0 : (size_t)v[5], STREAM(6)));
}

#define ENTRY(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}

static PyMethodDef methods[] = {
    ENTRY(route), ENTRY(route_backward), ENTRY(moe_plan), ENTRY(moe_dispatch), ENTRY(moe_combine),
    ENTRY(moe_combine_backward), ENTRY(layer_norm), ENTRY(layer_norm_backward),
    ENTRY(layer_norm_backward_workspace_size), ENTRY(grad_norm), ENTRY(clip_grad_norm),
    ENTRY(grad_norm_workspace_size), {"grad_descs", (PyCFunction)(void (*)(void))grad_descs, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mxqcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__mxqcall(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_is_cuda = PyUnicode_InternFromString("is_cuda");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_numel = PyUnicode_InternFromString("numel");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    if (!s_dtype || !s_is_cuda || !s_is_contiguous || !s_numel || !s_data_ptr) return NULL;
    return PyModule_Create(&module);
}
