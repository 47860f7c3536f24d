// The checks of the tree calls' tensors, for CPython: type, shape, device and contiguity of up to twenty tensors a call
// cost more than the call itself when the interpreter runs them (14 of 18 us of csa_commit_tree).  No torch header: the
// attributes and methods are the tensors' public ones, looked up by name (what needs torch's headers is in tensors.cpp).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

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

// ---------------------------------------------------------------- whole calls
// add_norm, append_pages and attend_pages as they are made step after step: every tensor given, contiguous, as the layer
// wants it.  Each looks at its tensors, and makes the library's call (at `fn`) if all are so: its status.  Anything else, a
// tensor to allocate, a stride, a wrong type, is None: the binding's own code then does or refuses it.  (Run by the
// interpreter, the checks of one small call cost 7 to 9 us; here 2 to 3 by the tensors' attributes, 0.4 with tensors.cpp;
// the launches 2 to 4.)
static PyObject *t_f32, *t_u8, *t_i32, *f_raw_stream, *f_device, *s_cuda_stream;

static PyObject* setup(PyObject* self, PyObject* args) {
  (void)self;
  PyObject* v[5];
  if (!PyArg_ParseTuple(args, "OOOOO", &v[0], &v[1], &v[2], &v[3], &v[4])) return NULL;
  PyObject** to[5] = {&t_f32, &t_u8, &t_i32, &f_raw_stream, &f_device};
  for (int i = 0; i < 5; ++i) {
    Py_INCREF(v[i]);
    Py_XSETREF(*to[i], v[i]);
  }
  Py_RETURN_NONE;
}

enum { kMaxDims = 8 };
typedef struct {
  int n;
  long long d[kMaxDims];
} Shape;

static int call_long(PyObject* t, PyObject* name, long long* out) {
  PyObject* v = PyObject_CallMethodNoArgs(t, name);
  if (!v) return 0;
  *out = PyLong_AsLongLong(v);
  Py_DECREF(v);
  return !PyErr_Occurred();
}

// tensors.cpp: the same by the tensor itself, -1 where only its attributes can tell
static int (*tensor)(PyObject*, PyObject*, int, int*, long long*, long long*, void**);

static PyObject* tensors(PyObject* self, PyObject* address) {
  (void)self;
  void* p = PyLong_AsVoidPtr(address);
  if (PyErr_Occurred()) return NULL;
  memcpy(&tensor, &p, sizeof(p));
  Py_RETURN_NONE;
}

// type, device, contiguity and address of t, its shape into s
static int look(PyObject* t, PyObject* dtype, Shape* s, long long* dev, void** p) {
  if (t == Py_None) return 0;
  if (tensor) {
    const int r = tensor(t, dtype, kMaxDims, &s->n, s->d, dev, p);
    if (r >= 0) return r;
  }
  PyObject* v = PyObject_GetAttr(t, s_dtype);
  if (!v) return 0;
  int ok = v == dtype;
  Py_DECREF(v);
  if (!ok) return 0;
  v = PyObject_GetAttr(t, s_shape);
  if (!v) return 0;
  ok = PyTuple_Check(v) && PyTuple_GET_SIZE(v) <= kMaxDims;
  if (ok) {
    s->n = (int)PyTuple_GET_SIZE(v);
    for (int i = 0; i < s->n; ++i) s->d[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
    ok = !PyErr_Occurred();
  }
  Py_DECREF(v);
  if (!ok || !call_long(t, s_get_device, dev) || *dev < 0) return 0;
  v = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (!v) return 0;
  ok = v == Py_True;
  Py_DECREF(v);
  long long a;
  if (!ok || !call_long(t, s_data_ptr, &a)) return 0;
  *p = (void*)(uintptr_t)a;
  return 1;
}
// the same of a tensor whose shape and device are known
static int as(PyObject* t, PyObject* dtype, long long dev, void** p, int n, const long long* dims) {
  Shape s;
  long long at;
  if (!look(t, dtype, &s, &at, p) || at != dev || s.n != n) return 0;
  for (int i = 0; i < n; ++i)
    if (s.d[i] != dims[i]) return 0;
  return 1;
}
#define AS(t, dtype, p, ...) \
  as(t, dtype, dev, p, (int)(sizeof((long long[]){__VA_ARGS__}) / sizeof(long long)), (const long long[]){__VA_ARGS__})

// the stream's handle; the call's device has to be the current one
static int stream_of(PyObject* stream, long long dev, void** raw) {
  PyObject* v = PyObject_CallNoArgs(f_device);
  if (!v) return 0;
  int ok = PyLong_AsLongLong(v) == dev;
  Py_DECREF(v);
  if (!ok) return 0;
  if (stream == Py_None) {
    PyObject* d = PyLong_FromLongLong(dev);
    v = d ? PyObject_CallOneArg(f_raw_stream, d) : NULL;
    Py_XDECREF(d);
  } else {
    v = PyObject_GetAttr(stream, s_cuda_stream);
  }
  if (!v) return 0;
  *raw = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(v);
  Py_DECREF(v);
  return !PyErr_Occurred();
}
static PyObject* not_plain(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}
static void* address_arg(PyObject* o) { return (void*)(uintptr_t)PyLong_AsUnsignedLongLong(o); }

// add_norm(fn, layer, dtype, x, residual, weight, group, out, residual_out, codes, scales, stream)
static PyObject* add_norm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 12 || !t_f32 || !PyBytes_Check(a[1])) return not_plain();
  Shape s;
  long long dev, group = 0;
  void *x, *r = NULL, *w = NULL, *out = NULL, *res = NULL, *codes = NULL, *scales = NULL, *raw;
  PyObject* dt = a[2];
  if (!look(a[3], dt, &s, &dev, &x) || s.n < 1 || s.d[s.n - 1] < 1) return not_plain();
  const long long X = s.d[s.n - 1];
  long long N = 1;
  for (int i = 0; i + 1 < s.n; ++i) N *= s.d[i];
  if (a[4] != Py_None ? !as(a[4], dt, dev, &r, s.n, s.d) : (a[8] != Py_None && a[8] != Py_False)) return not_plain();
  if (a[5] != Py_None && !AS(a[5], t_f32, &w, X)) return not_plain();
  if (a[7] != Py_False && !as(a[7], dt, dev, &out, s.n, s.d)) return not_plain();
  if (a[4] != Py_None && a[8] != Py_False && !as(a[8], dt, dev, &res, s.n, s.d)) return not_plain();
  if (a[6] != Py_None) {
    group = PyLong_AsLongLong(a[6]);
    if (PyErr_Occurred() || group < 1 || X % group || !as(a[9], t_u8, dev, &codes, s.n, s.d)) return not_plain();
    s.d[s.n - 1] = X / group;
    if (!as(a[10], t_f32, dev, &scales, s.n, s.d)) return not_plain();
  } else if (a[9] != Py_None || a[10] != Py_None) {
    return not_plain();
  }
  if (X > 16384 || !stream_of(a[11], dev, &raw)) return not_plain();
  int (*fn)(const void*, const void*, long long, const void*, long long, const void*, long long, int, void*, void*, void*,
            void*, int, void*) = (int (*)(const void*, const void*, long long, const void*, long long, const void*,
                                          long long, int, void*, void*, void*, void*, int, void*))address_arg(a[0]);
  int code;
  Py_BEGIN_ALLOW_THREADS
  code = fn(PyBytes_AS_STRING(a[1]), x, 0, r, 0, w, N, (int)X, out, res, codes, scales, (int)group, raw);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(code);
}

// csa_pages
typedef struct {
  void *codes, *scales;
  int n, rows;
} Pool;
static int pool_of(PyObject* codes, PyObject* scales, long long dev, long long D, Pool* p) {
  Shape s;
  long long at;
  if (!look(codes, t_u8, &s, &at, &p->codes) || at != dev || s.n != 3 || s.d[2] != D) return 0;
  if (s.d[0] > 1 << 30 || s.d[1] > 1 << 30 || !AS(scales, t_f32, &p->scales, s.d[0], s.d[1])) return 0;
  p->n = (int)s.d[0];
  p->rows = (int)s.d[1];
  return 1;
}
static int table_of(PyObject* t, long long dev, long long B, void** p, int* width) {
  Shape s;
  long long at;
  if (!look(t, t_i32, &s, &at, p) || at != dev || s.n != 2 || s.d[0] != B || s.d[1] > 1 << 30) return 0;
  *width = (int)s.d[1];
  return 1;
}

// append_pages(fn, layer, dtype, D, R/2, rows, codes, scales, table, pos, n_new, weight, norm, inv_freq, err, stream)
static PyObject* append_pages(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 16 || !t_f32 || !PyBytes_Check(a[1])) return not_plain();
  const long long D = PyLong_AsLongLong(a[3]), half = PyLong_AsLongLong(a[4]);
  Shape s, e;
  long long dev, at;
  Pool pool;
  int width;
  void *rows, *table, *pos, *fresh = NULL, *w = NULL, *frq = NULL, *err, *raw;
  if (!look(a[5], a[2], &s, &dev, &rows) || s.n != 3 || s.d[2] != D || s.d[0] > 1 << 24 || s.d[1] > 1 << 24 ||
      s.d[0] * s.d[1] > 1 << 24)
    return not_plain();
  const int norm = PyObject_IsTrue(a[12]);
  if (norm < 0 || !pool_of(a[6], a[7], dev, D, &pool) || !table_of(a[8], dev, s.d[0], &table, &width) ||
      !AS(a[9], t_i32, &pos, s.d[0]))
    return not_plain();
  if ((a[10] != Py_None && !AS(a[10], t_i32, &fresh, s.d[0])) || (a[11] != Py_None && (!norm || !AS(a[11], t_f32, &w, D))) ||
      (a[13] != Py_None && !AS(a[13], t_f32, &frq, half)))
    return not_plain();
  if (!look(a[14], t_i32, &e, &at, &err) || at != dev || e.n != 1 || e.d[0] < 1 || !stream_of(a[15], dev, &raw))
    return not_plain();
  int (*fn)(const void*, const void*, const void*, long long, long long, int, int, const void*, int, const void*,
            const void*, const void*, int, const void*, void*, void*) =
      (int (*)(const void*, const void*, const void*, long long, long long, int, int, const void*, int, const void*,
               const void*, const void*, int, const void*, void*, void*))address_arg(a[0]);
  int code;
  Py_BEGIN_ALLOW_THREADS
  code = fn(PyBytes_AS_STRING(a[1]), &pool, rows, 0, 0, (int)s.d[0], (int)s.d[1], table, width, pos, fresh, w, norm, frq,
            err, raw);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(code);
}

// attend_pages(fn, layer, dtype, H, D, R/2, topk, q, codes, scales, sink, pos, out, token_table, first, row_table, n_rows,
//              sel, n_sel, n_new, inv_freq, ws, err, stream)
static PyObject* attend_pages(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 24 || !t_f32 || !PyBytes_Check(a[1])) return not_plain();
  const long long H = PyLong_AsLongLong(a[3]), D = PyLong_AsLongLong(a[4]), half = PyLong_AsLongLong(a[5]),
                  topk = PyLong_AsLongLong(a[6]);
  Shape s, e;
  long long dev, at, bytes;
  Pool pool;
  int tw = 0, rw = 0;
  void *q, *out, *pos, *sink = NULL, *tok = NULL, *row = NULL, *nr = NULL, *sel = NULL, *ns = NULL, *fresh = NULL,
       *frq = NULL, *ws, *err, *raw;
  if (!look(a[7], a[2], &s, &dev, &q) || s.n != 4 || s.d[2] != H || s.d[3] != D) return not_plain();
  const long long B = s.d[0], T = s.d[1], first = PyLong_AsLongLong(a[14]);
  if (PyErr_Occurred() || B > 1 << 16 || T > 1 << 16 || B * T > 1 << 16 || first < 0 || first > 0x7fffffff) return not_plain();
  if (!pool_of(a[8], a[9], dev, D, &pool) || !AS(a[11], t_i32, &pos, B) || !AS(a[12], a[2], &out, B, T, H, D))
    return not_plain();
  if ((a[10] != Py_None && !AS(a[10], t_f32, &sink, H)) || (a[13] != Py_None && !table_of(a[13], dev, B, &tok, &tw)))
    return not_plain();
  if (a[15] != Py_None) {
    if (!table_of(a[15], dev, B, &row, &rw) || !AS(a[16], t_i32, &nr, B)) return not_plain();
  } else if (a[16] != Py_None || a[17] != Py_None || a[18] != Py_None || a[13] == Py_None) {
    return not_plain();
  }
  if (a[17] != Py_None ? !AS(a[17], t_i32, &sel, B, T, topk) || !AS(a[18], t_i32, &ns, B, T) : a[18] != Py_None)
    return not_plain();
  if ((a[19] != Py_None && !AS(a[19], t_i32, &fresh, B)) || (a[20] != Py_None && !AS(a[20], t_f32, &frq, half)))
    return not_plain();
  if (!look(a[21], t_u8, &e, &at, &ws) || at != dev || e.n != 1) return not_plain();
  bytes = e.d[0];
  if (!look(a[22], t_i32, &e, &at, &err) || at != dev || e.n != 1 || e.d[0] < 1 || !stream_of(a[23], dev, &raw))
    return not_plain();
  int (*fn)(const void*, const void*, const void*, int, int, const void*, const void*, const void*, const void*, int, int,
            const void*, int, const void*, const void*, const void*, const void*, void*, void*, size_t, void*, void*) =
      (int (*)(const void*, const void*, const void*, int, int, const void*, const void*, const void*, const void*, int,
               int, const void*, int, const void*, const void*, const void*, const void*, void*, void*, size_t, void*,
               void*))address_arg(a[0]);
  int code;
  Py_BEGIN_ALLOW_THREADS
  code = fn(PyBytes_AS_STRING(a[1]), &pool, q, (int)B, (int)T, sink, pos, fresh, tok, tw, (int)first, row, rw, nr, sel, ns,
            frq, out, ws, (size_t)bytes, err, raw);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(code);
}

static PyMethodDef methods[] = {
    {"addresses", (PyCFunction)(void (*)(void))addresses, METH_FASTCALL, "addresses(device, *specs)"},
    {"setup", setup, METH_VARARGS, "setup(float32, uint8, int32, raw stream of a device, current device)"},
    {"tensors", tensors, METH_O, "tensors(address of csa_tensor, or 0)"},
    {"add_norm", (PyCFunction)(void (*)(void))add_norm, METH_FASTCALL, "csa_add_norm on plain tensors"},
    {"append_pages", (PyCFunction)(void (*)(void))append_pages, METH_FASTCALL, "csa_append_pages on plain tensors"},
    {"attend_pages", (PyCFunction)(void (*)(void))attend_pages, METH_FASTCALL, "csa_attend_pages on plain tensors"},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "csa_checks", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_csa_checks(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (!s_cuda_stream || !s_dtype || !s_shape || !s_get_device || !s_is_contiguous || !s_data_ptr) return NULL;
  return PyModule_Create(&module);
}
