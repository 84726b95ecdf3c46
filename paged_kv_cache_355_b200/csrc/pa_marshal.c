/* pa_marshal.c -- the argument marshalling of the calls that are shorter on
 * the device than a Python call's own cost: a CPython extension module, linked
 * with libpa.so, that takes a call's arguments as Python objects, tests every
 * tensor (on the call's device, of the expected element type, contiguous) and
 * calls the C entry point.  Nothing else: shapes are compared, and errors
 * worded, by the Python function of the same name.
 *
 *   call(entry, device, dtype, args) -> status
 *     entry   number of the entry point (its place in ENTRIES)
 *     device  the CUDA device index every tensor has to be on
 *     dtype   the torch dtype that stands for 'K' in the signature, or None
 *     args    tuple, one object a letter of the signature
 *   returns the pa_status of the entry point, or -1 - i where args[i] is
 *   refused.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>
#include <stdint.h>

#include "pa.h"

typedef union {
    void* p;
    int64_t l;
    int i;
    float f;
} slot;

/* Signature letters.  Tensors (a pointer): K of the call's dtype, i int32,
 * l int64, f float32, o any type, r of the call's dtype with its own strides.
 * k, j, m: like K, i, l, or None.  Scalars: I int, L int64, F float, P an
 * address.  */
static int call_rope(const slot* v) {
    return pa_rope_and_cache(v[0].p, v[1].p, v[2].p, v[3].l, v[4].l, v[5].l, v[6].p, v[7].p, v[8].p, v[9].p, v[10].p,
                             v[11].i, v[12].p, v[13].p, v[14].l, v[15].i, v[16].i, v[17].p, v[18].p, v[19].f, v[20].l,
                             v[21].i, v[22].i, v[23].i, v[24].i, v[25].l, v[26].i, v[27].p);
}
static int call_rope_decode(const slot* v) {
    return pa_rope_and_cache_decode(v[0].p, v[1].p, v[2].p, v[3].l, v[4].l, v[5].l, v[6].p, v[7].p, v[8].p, v[9].p,
                                    v[10].i, v[11].p, v[12].p, v[13].i, v[14].p, v[15].p, v[16].l, v[17].i, v[18].i,
                                    v[19].p, v[20].p, v[21].f, v[22].i, v[23].i, v[24].i, v[25].i, v[26].i, v[27].l,
                                    v[28].i, v[29].p, v[30].p);
}
static int call_bounds(const slot* v) {
    return pa_update_key_bounds(v[0].p, v[1].p, v[2].p, v[3].i, v[4].p, v[5].p, v[6].i, v[7].i, v[8].i, v[9].i, v[10].i,
                                v[11].l, v[12].i, v[13].p);
}
static int call_scores(const slot* v) {
    return pa_block_scores(v[0].p, v[1].p, v[2].p, v[3].i, v[4].p, v[5].p, v[6].i, v[7].i, v[8].p, v[9].l, v[10].l,
                           v[11].i, v[12].i, v[13].i, v[14].i, v[15].l, v[16].i, v[17].p);
}
static int call_select(const slot* v) {
    return pa_select_blocks(v[0].p, v[1].l, v[2].p, v[3].i, v[4].i, v[5].p, v[6].i, v[7].i, v[8].i, v[9].l, v[10].i,
                            v[11].p);
}
static int call_sparse(const slot* v) {
    return pa_paged_attention_decode_sparse(v[0].p, v[1].p, v[2].p, v[3].p, v[4].i, v[5].p, v[6].p, v[7].p, v[8].i,
                                            v[9].f, v[10].i, v[11].p, v[12].i, v[13].l, v[14].i, v[15].i, v[16].i,
                                            v[17].i, v[18].l, v[19].i, v[20].p);
}

static const struct {
    const char* name;
    const char* signature;
    int (*call)(const slot*);
} entries[] = {
    {"pa_rope_and_cache", "rrrLLLKKKliIjfLIIkkFLIIIILIP", call_rope},
    {"pa_rope_and_cache_decode", "rrrLLLKKKiIijIjfLIIkkFIIIIILImP", call_rope_decode},
    {"pa_update_key_bounds", "KKiIijIIIIILIP", call_bounds},
    {"pa_block_scores", "KKiIjiIIfLLIIIILIP", call_scores},
    {"pa_select_blocks", "fLiIIiIIILIP", call_select},
    {"pa_paged_attention_decode_sparse", "KKKiIjiiIFIoILIIIILIP", call_sparse},
};
enum { kEntries = sizeof(entries) / sizeof(entries[0]), kMostArgs = 32 };

/* the names of the tensor's methods and the dtypes, held for good */
static PyObject *s_get_device, *s_dtype, *s_is_contiguous, *s_data_ptr;
static PyObject *d_int32, *d_int64, *d_float32;

/* The address of a tensor that passes; 0 (no Python error) where it does not. */
static int tensor_address(PyObject* t, long device, PyObject* dtype, int contiguous, slot* out) {
    PyObject* x = PyObject_CallMethodNoArgs(t, s_get_device);
    if (!x) goto refused;
    const long at = PyLong_AsLong(x);
    Py_DECREF(x);
    if (at != device || device < 0) goto refused;
    if (dtype) {
        x = PyObject_GetAttr(t, s_dtype);
        if (!x) goto refused;
        const int same = x == dtype;
        Py_DECREF(x);
        if (!same) goto refused;
    }
    if (contiguous) {
        x = PyObject_CallMethodNoArgs(t, s_is_contiguous);
        if (!x) goto refused;
        const int yes = x == Py_True;
        Py_DECREF(x);
        if (!yes) goto refused;
    }
    x = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!x) goto refused;
    out->p = PyLong_AsVoidPtr(x);
    Py_DECREF(x);
    if (PyErr_Occurred()) goto refused;
    return 1;
refused:
    PyErr_Clear();
    return 0;
}

/* 1: done, 0: refused, -1: a Python error is set. */
static int read_argument(char letter, PyObject* a, long device, PyObject* dtype, slot* out) {
    long long value;
    int over = 0;
    out->l = 0;
    switch (letter) {
        case 'k':
        case 'j':
        case 'm':
            if (a == Py_None) return 1;
            return tensor_address(a, device, letter == 'k' ? dtype : letter == 'j' ? d_int32 : d_int64, 1, out);
        case 'K': return tensor_address(a, device, dtype, 1, out);
        case 'r': return tensor_address(a, device, dtype, 0, out);
        case 'i': return tensor_address(a, device, d_int32, 1, out);
        case 'l': return tensor_address(a, device, d_int64, 1, out);
        case 'f': return tensor_address(a, device, d_float32, 1, out);
        case 'o': return tensor_address(a, device, NULL, 1, out);
        case 'F': {
            const double x = PyFloat_AsDouble(a);
            if (x == -1.0 && PyErr_Occurred()) return -1;
            out->f = (float)x;
            return 1;
        }
        case 'P':
            out->p = PyLong_AsVoidPtr(a);
            return PyErr_Occurred() ? -1 : 1;
        default: break;
    }
    value = PyLong_AsLongLongAndOverflow(a, &over); /* takes what has __index__ */
    if (value == -1 && !over && PyErr_Occurred()) return -1;
    if (over || (letter == 'I' && (value > INT_MAX || value < INT_MIN))) {
        PyErr_SetString(PyExc_OverflowError, "an integer argument is out of range");
        return -1;
    }
    if (letter == 'I')
        out->i = (int)value;
    else
        out->l = value;
    return 1;
}

static PyObject* marshal_call(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 4 || !PyTuple_Check(a[3])) {
        PyErr_SetString(PyExc_TypeError, "call(entry, device, dtype, args)");
        return NULL;
    }
    const long entry = PyLong_AsLong(a[0]), device = PyLong_AsLong(a[1]);
    if (PyErr_Occurred()) return NULL;
    if (entry < 0 || entry >= kEntries) {
        PyErr_SetString(PyExc_ValueError, "no such entry point");
        return NULL;
    }
    const char* signature = entries[entry].signature;
    PyObject* dtype = a[2] == Py_None ? NULL : a[2];
    slot v[kMostArgs];
    Py_ssize_t i = 0;
    for (; signature[i]; ++i) {
        if (i >= PyTuple_GET_SIZE(a[3])) break;
        const int ok = read_argument(signature[i], PyTuple_GET_ITEM(a[3], i), device, dtype, &v[i]);
        if (ok < 0) return NULL;
        if (!ok) return PyLong_FromLong(-1 - (long)i);
    }
    if (signature[i] || i != PyTuple_GET_SIZE(a[3])) {
        PyErr_Format(PyExc_TypeError, "%s: wrong number of arguments", entries[entry].name);
        return NULL;
    }
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = entries[entry].call(v);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

/* init(int32, int64, float32): the dtype objects; returns (name, signature) of each entry */
static PyObject* marshal_init(PyObject* self, PyObject* args) {
    (void)self;
    PyObject *x, *y, *z;
    if (!PyArg_ParseTuple(args, "OOO", &x, &y, &z)) return NULL;
    Py_INCREF(x);
    Py_INCREF(y);
    Py_INCREF(z);
    d_int32 = x;
    d_int64 = y;
    d_float32 = z;
    PyObject* list = PyTuple_New(kEntries);
    for (int e = 0; list && e < kEntries; ++e) {
        PyObject* item = Py_BuildValue("(ss)", entries[e].name, entries[e].signature);
        if (!item) {
            Py_CLEAR(list);
            break;
        }
        PyTuple_SET_ITEM(list, e, item);
    }
    return list;
}

static PyMethodDef methods[] = {
    {"call", (PyCFunction)(void (*)(void))marshal_call, METH_FASTCALL, "call(entry, device, dtype, args) -> status"},
    {"init", marshal_init, METH_VARARGS, "init(int32, int64, float32) -> ((name, signature), ...)"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
    s_get_device = PyUnicode_InternFromString("get_device");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    if (!s_get_device || !s_dtype || !s_is_contiguous || !s_data_ptr) return NULL;
    return PyModule_Create(&module);
}
