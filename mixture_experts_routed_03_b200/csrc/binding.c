/*
 * binding.c -- a CPython extension with one function, for calls that are
 * shorter than their marshalling: call(address, *args) calls the C function
 * at `address` with its arguments as machine words and returns its int.  An
 * argument is None (NULL), an int, or an object with data_ptr() (a tensor).
 * The interpreter lock is released during the call, as ctypes does.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#define MAX_ARGS 12

typedef uintptr_t W;

static PyObject* name_data_ptr;

static int word(PyObject* o, W* w) {
  if (o == Py_None) {
    *w = 0;
    return 0;
  }
  if (PyLong_Check(o)) {
    *w = (W)PyLong_AsUnsignedLongLongMask(o);
    return PyErr_Occurred() ? -1 : 0;
  }
  PyObject* p = PyObject_CallMethodNoArgs(o, name_data_ptr);
  if (!p) return -1;
  *w = (W)PyLong_AsUnsignedLongLongMask(p);
  Py_DECREF(p);
  return PyErr_Occurred() ? -1 : 0;
}

static PyObject* call(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  (void)self;
  W a[MAX_ARGS + 1] = {0};
  if (n < 2 || n > MAX_ARGS + 1) {
    PyErr_Format(PyExc_TypeError, "call() takes an address and 1 to %d arguments", MAX_ARGS);
    return NULL;
  }
  for (Py_ssize_t i = 0; i < n; ++i)
    if (word(args[i], &a[i])) return NULL;
  int r = 0;
  Py_BEGIN_ALLOW_THREADS
  switch (n - 1) {
    case 6: r = ((int (*)(W, W, W, W, W, W))a[0])(a[1], a[2], a[3], a[4], a[5], a[6]); break;
    case 9: r = ((int (*)(W, W, W, W, W, W, W, W, W))a[0])(a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9]); break;
    case 10:
      r = ((int (*)(W, W, W, W, W, W, W, W, W, W))a[0])(a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10]);
      break;
    default: r = -1;
  }
  Py_END_ALLOW_THREADS
  if (r == -1) {
    PyErr_SetString(PyExc_TypeError, "call() makes calls of 6, 9 or 10 arguments");
    return NULL;
  }
  return PyLong_FromLong(r);
}

static PyMethodDef methods[] = {{"call", (PyCFunction)(void (*)(void))call, METH_FASTCALL, "call(address, *args) -> int"},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  name_data_ptr = PyUnicode_InternFromString("data_ptr");
  return name_data_ptr ? PyModule_Create(&module) : NULL;
}
