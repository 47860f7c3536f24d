// The checks of the tree calls' tensors, for CPython: type, shape, device and contiguity of up to twenty tensors a call
// cost more than the call itself when the interpreter runs them (14 of 18 us of csa_commit_tree).  No torch header: the
// attributes and methods are the tensors' public ones, looked up by name.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

static PyObject *s_dtype, *s_shape, *s_get_device, *s_is_contiguous, *s_data_ptr;

// Address of tensor t as a new int object, or NULL (no exception set) when it is not what the spec says.
static PyObject* address(PyObject* t, PyObject* dtype, PyObject* shape, long dev) {
  PyObject* v = PyObject_GetAttr(t, s_dtype);
  if (!v) goto fail;
  int ok = v == dtype;
  Py_DECREF(v);
  if (!ok) return NULL;
  v = PyObject_GetAttr(t, s_shape);
  if (!v) goto fail;
  ok = PyTuple_Check(v) && PyTuple_Check(shape) && PyTuple_GET_SIZE(v) == PyTuple_GET_SIZE(shape);
  for (Py_ssize_t i = 0; ok && i < PyTuple_GET_SIZE(v); ++i) {
    const long long a = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i)), b = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    ok = a == b && !PyErr_Occurred();
  }
  Py_DECREF(v);
  if (!ok) goto fail;
  v = PyObject_CallMethodNoArgs(t, s_get_device);
  if (!v) goto fail;
  ok = PyLong_AsLong(v) == dev && !PyErr_Occurred();
  Py_DECREF(v);
  if (!ok) goto fail;
  v = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (!v) goto fail;
  ok = v == Py_True;
  Py_DECREF(v);
  if (!ok) return NULL;
  v = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (v) return v;
fail:
  PyErr_Clear();
  return NULL;
}

// addresses(device, *specs), spec (name, tensor, dtype, shape): the list of the tensors' addresses, or the first spec
// that its tensor does not meet.
static PyObject* addresses(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  (void)self;
  if (n < 1) {
    PyErr_SetString(PyExc_TypeError, "addresses(device, *specs)");
    return NULL;
  }
  const long dev = PyLong_AsLong(args[0]);
  if (dev == -1 && PyErr_Occurred()) return NULL;
  PyObject* out = PyList_New(n - 1);
  if (!out) return NULL;
  for (Py_ssize_t i = 1; i < n; ++i) {
    PyObject* spec = args[i];
    if (!PyTuple_Check(spec) || PyTuple_GET_SIZE(spec) != 4) {
      PyErr_SetString(PyExc_TypeError, "a spec is (name, tensor, dtype, shape)");
      Py_DECREF(out);
      return NULL;
    }
    PyObject* p = address(PyTuple_GET_ITEM(spec, 1), PyTuple_GET_ITEM(spec, 2), PyTuple_GET_ITEM(spec, 3), dev);
    if (!p) {
      Py_DECREF(out);
      Py_INCREF(spec);
      return spec;
    }
    PyList_SET_ITEM(out, i - 1, p);
  }
  return out;
}

static PyMethodDef methods[] = {
    {"addresses", (PyCFunction)(void (*)(void))addresses, METH_FASTCALL, "addresses(device, *specs)"},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "csa_checks", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_csa_checks(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  if (!s_dtype || !s_shape || !s_get_device || !s_is_contiguous || !s_data_ptr) return NULL;
  return PyModule_Create(&module);
}
