/*
 * The operators' C entry points as functions of the Python interpreter: numbers,
 * None (a null pointer) and bytes in, the status out.  A call takes 0.3 us where
 * ctypes takes 1.9 to convert the same 18 arguments, as long as the launch itself.
 * bind() gives the addresses in the loaded libkvc.so.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/kvc.h"

enum { ATTEND, EVICT, STORE, DEQUANTIZE, ROTATE, ENTRIES };
static void* entry_of[ENTRIES];

static int count_is(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return 1;
  PyErr_Format(PyExc_TypeError, "%zd arguments, %zd are needed", got, want);
  return 0;
}

/* A pointer: a number, None or the first of some bytes. */
static void* pointer(PyObject* x) {
  if (x == Py_None) return NULL;
  if (PyBytes_Check(x)) return PyBytes_AS_STRING(x);
  return PyLong_AsVoidPtr(x);
}

static int64_t whole(PyObject* x) { return PyLong_AsLongLong(x); }

#define P(at) void* const p##at = pointer(a[at])
#define I(at) const int64_t i##at = whole(a[at])
#define N(at) const int32_t n##at = (int32_t)whole(a[at])
#define F(at) const float f##at = (float)PyFloat_AsDouble(a[at])
#define CALL(type, which, ...)                               \
  kvc_status status;                                         \
  if (PyErr_Occurred()) return NULL;                         \
  if (entry_of[which] == NULL) {                             \
    PyErr_SetString(PyExc_RuntimeError, "not bound");        \
    return NULL;                                             \
  }                                                          \
  Py_BEGIN_ALLOW_THREADS                                     \
  status = ((__typeof__(&type))entry_of[which])(__VA_ARGS__); \
  Py_END_ALLOW_THREADS                                       \
  return PyLong_FromLong(status)

static PyObject* attend(PyObject* self, PyObject* const* a, Py_ssize_t count) {
  if (!count_is(count, 25)) return NULL;
  P(0); I(1); I(2); I(3); N(4); P(5); N(6); I(7); P(8); I(9); I(10); P(11); F(12); P(13); P(14); P(15);
  P(16); I(17); P(18); I(19); I(20); P(21); I(22); N(23); P(24);
  CALL(kvc_attend_format, ATTEND, p0, i1, i2, i3, n4, p5, n6, i7, p8, i9, i10, p11, f12, p13, p14, p15, p16, i17,
       p18, i19, i20, p21, (size_t)i22, (uint32_t)n23, p24);
}

static PyObject* evict(PyObject* self, PyObject* const* a, Py_ssize_t count) {
  if (!count_is(count, 24)) return NULL;
  P(0); N(1); I(2); P(3); I(4); I(5); I(6); P(7); P(8); I(9); I(10); P(11); I(12); I(13); I(14); P(15);
  P(16); P(17); I(18); P(19); I(20); P(21); I(22); P(23);
  CALL(kvc_evict_format, EVICT, p0, n1, i2, p3, i4, i5, i6, p7, p8, i9, i10, p11, i12, i13, i14, p15, p16, p17, i18,
       p19, i20, p21, (size_t)i22, p23);
}

static PyObject* store(PyObject* self, PyObject* const* a, Py_ssize_t count) {
  if (!count_is(count, 16)) return NULL;
  P(0); N(1); I(2); I(3); P(4); N(5); I(6); P(7); P(8); I(9); I(10); N(11); P(12); P(13); I(14); P(15);
  CALL(kvc_store, STORE, p0, n1, i2, i3, p4, n5, i6, p7, p8, i9, i10, n11, p12, p13, i14, p15);
}

static PyObject* dequantize(PyObject* self, PyObject* const* a, Py_ssize_t count) {
  if (!count_is(count, 8)) return NULL;
  P(0); N(1); I(2); P(3); I(4); P(5); N(6); P(7);
  CALL(kvc_dequantize_format, DEQUANTIZE, p0, n1, i2, p3, i4, p5, n6, p7);
}

static PyObject* rotate(PyObject* self, PyObject* const* a, Py_ssize_t count) {
  if (!count_is(count, 18)) return NULL;
  P(0); N(1); I(2); I(3); I(4); N(5); P(6); I(7); I(8); N(9); P(10); P(11); I(12); N(13); P(14); I(15); I(16); P(17);
  CALL(kvc_rotate, ROTATE, p0, n1, i2, i3, i4, n5, p6, i7, i8, n9, p10, p11, i12, n13, p14, i15, i16, p17);
}

static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t count) {
  if (!count_is(count, ENTRIES)) return NULL;
  void* found[ENTRIES];
  for (int i = 0; i < ENTRIES; ++i) found[i] = pointer(a[i]);
  if (PyErr_Occurred()) return NULL;
  for (int i = 0; i < ENTRIES; ++i) entry_of[i] = found[i];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, NULL},
    {"kvc_attend_format", (PyCFunction)(void (*)(void))attend, METH_FASTCALL, NULL},
    {"kvc_evict_format", (PyCFunction)(void (*)(void))evict, METH_FASTCALL, NULL},
    {"kvc_store", (PyCFunction)(void (*)(void))store, METH_FASTCALL, NULL},
    {"kvc_dequantize_format", (PyCFunction)(void (*)(void))dequantize, METH_FASTCALL, NULL},
    {"kvc_rotate", (PyCFunction)(void (*)(void))rotate, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvc_call", NULL, -1, methods};

PyMODINIT_FUNC PyInit__kvc_call(void) { return PyModule_Create(&module); }
