/* marshal.c -- the binding's inner steps as a CPython module: look at a tensor's layout, call a
 * function of the C ABI. A single token's kernels take a few microseconds, and the same steps in
 * Python and ctypes took longer than they do. Nothing here knows torch: tensors are asked through
 * their attributes (shape, dtype, stride(), get_device(), data_ptr(), is_contiguous()). */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

static PyObject *s_shape, *s_dtype, *s_stride, *s_get_device, *s_data_ptr, *s_is_contiguous;

/* t.name() as an integer; -1 with an exception set on failure. */
static long long ask(PyObject *t, PyObject *name) {
  PyObject *v = PyObject_CallMethodNoArgs(t, name);
  if (!v) return -1;
  const long long x = PyLong_AsLongLong(v);
  Py_DECREF(v);
  return x;
}

static long long item(PyObject *tuple, Py_ssize_t i) { return PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i)); }

/* Whether t has this dtype on this device: 1, 0, or -1 with an exception. */
static int placed(PyObject *t, PyObject *device, PyObject *dtype) {
  PyObject *d = PyObject_GetAttr(t, s_dtype);
  if (!d) return -1;
  Py_DECREF(d); /* dtypes live as long as torch */
  if (d != dtype) return 0;
  const long long at = ask(t, s_get_device);
  if (PyErr_Occurred()) return -1;
  return at == PyLong_AsLongLong(device);
}

/* rows(t, rows, width, device, dtype) -> (address, row stride in elements) of a [rows, width] view with
 * contiguous rows, or of [rows, heads, D] with contiguous heads; None if t is no such view. */
static PyObject *m_rows(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (n != 5) return PyErr_Format(PyExc_TypeError, "rows takes 5 arguments");
  PyObject *t = a[0], *shape = NULL, *st = NULL, *out = NULL;
  const long long rows = PyLong_AsLongLong(a[1]), width = PyLong_AsLongLong(a[2]);
  if (PyErr_Occurred()) return NULL;
  const int ok = placed(t, a[3], a[4]);
  if (ok < 0) return NULL;
  if (!ok) Py_RETURN_NONE;
  if (!(shape = PyObject_GetAttr(t, s_shape)) || !(st = PyObject_CallMethodNoArgs(t, s_stride))) goto end;
  if (PyTuple_Check(shape) && PyTuple_Check(st)) {
    const Py_ssize_t dim = PyTuple_GET_SIZE(shape);
    long long inner = -1;
    int flat = 0;
    if (dim == 2 && PyTuple_GET_SIZE(st) == 2) {
      inner = item(shape, 1);
      flat = item(st, 1) == 1 || inner == 1;
    } else if (dim == 3 && PyTuple_GET_SIZE(st) == 3) {
      const long long heads = item(shape, 1), d = item(shape, 2);
      inner = heads * d;
      flat = (item(st, 2) == 1 || d == 1) && (heads == 1 || item(st, 1) == d);
    }
    if (!PyErr_Occurred() && inner == width && item(shape, 0) == rows && (flat || rows == 0)) {
      /* (without a second row there is no stride to speak of) */
      const long long rs = rows > 1 ? item(st, 0) : width, p = PyErr_Occurred() ? -1 : ask(t, s_data_ptr);
      if (!PyErr_Occurred()) out = Py_BuildValue("(LL)", p, rs);
      goto end;
    }
  }
  if (!PyErr_Occurred()) {
    out = Py_None;
    Py_INCREF(out);
  }
end:
  Py_XDECREF(shape);
  Py_XDECREF(st);
  return out;
}

/* array(t, shape, device, dtype) -> address of a contiguous tensor of that shape; None if t is none. */
static PyObject *m_array(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (n != 4) return PyErr_Format(PyExc_TypeError, "array takes 4 arguments");
  int ok = placed(a[0], a[2], a[3]);
  if (ok > 0) {
    PyObject *shape = PyObject_GetAttr(a[0], s_shape);
    if (!shape) return NULL;
    ok = PyObject_RichCompareBool(shape, a[1], Py_EQ);
    Py_DECREF(shape);
  }
  if (ok > 0) {
    PyObject *c = PyObject_CallMethodNoArgs(a[0], s_is_contiguous);
    if (!c) return NULL;
    ok = PyObject_IsTrue(c);
    Py_DECREF(c);
  }
  if (ok < 0) return NULL;
  if (!ok) Py_RETURN_NONE;
  return PyObject_CallMethodNoArgs(a[0], s_data_ptr);
}

/* call(function's address, problem, *arguments) -> status. Every argument behind the problem is an
 * integer of at most 64 bits or an address (None: 0), so one prototype with as many integer arguments
 * as the longest function has serves them all (the callee takes those that it declares). */
enum { MOST = 28 };
typedef int (*abi_fn)(const void *, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                      int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                      int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t);
static PyObject *m_call(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (n < 2 || n - 2 > MOST) return PyErr_Format(PyExc_TypeError, "call: %zd arguments", n);
  int64_t v[MOST] = {0};
  for (Py_ssize_t i = 2; i < n; ++i) {
    if (a[i] == Py_None) continue;
    v[i - 2] = PyLong_AsLongLong(a[i]);
    if (v[i - 2] == -1 && PyErr_Occurred()) return NULL;
  }
  const abi_fn f = (abi_fn)(uintptr_t)PyLong_AsUnsignedLongLong(a[0]);
  if (PyErr_Occurred()) return NULL;
  Py_buffer p;
  if (PyObject_GetBuffer(a[1], &p, PyBUF_SIMPLE)) return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = f(p.buf, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8], v[9], v[10], v[11], v[12], v[13], v[14], v[15],
         v[16], v[17], v[18], v[19], v[20], v[21], v[22], v[23], v[24], v[25], v[26], v[27]);
  Py_END_ALLOW_THREADS
  PyBuffer_Release(&p);
  return PyLong_FromLong(st);
}

/* size(function's address, problem) -> bytes. */
static PyObject *m_size(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (n != 2) return PyErr_Format(PyExc_TypeError, "size takes 2 arguments");
  size_t (*f)(const void *) = (size_t (*)(const void *))(uintptr_t)PyLong_AsUnsignedLongLong(a[0]);
  if (PyErr_Occurred()) return NULL;
  Py_buffer p;
  if (PyObject_GetBuffer(a[1], &p, PyBUF_SIMPLE)) return NULL;
  const size_t bytes = f(p.buf);
  PyBuffer_Release(&p);
  return PyLong_FromSize_t(bytes);
}

static PyMethodDef methods[] = {{"rows", (PyCFunction)(void (*)(void))m_rows, METH_FASTCALL, "layout of a row view"},
                                {"array", (PyCFunction)(void (*)(void))m_array, METH_FASTCALL, "address of an array"},
                                {"call", (PyCFunction)(void (*)(void))m_call, METH_FASTCALL, "call a function of the C ABI"},
                                {"size", (PyCFunction)(void (*)(void))m_size, METH_FASTCALL, "call a size query of the C ABI"},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "inner steps of the binding", -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
  if (!(s_shape = PyUnicode_InternFromString("shape")) || !(s_dtype = PyUnicode_InternFromString("dtype")) ||
      !(s_stride = PyUnicode_InternFromString("stride")) || !(s_get_device = PyUnicode_InternFromString("get_device")) ||
      !(s_data_ptr = PyUnicode_InternFromString("data_ptr")) || !(s_is_contiguous = PyUnicode_InternFromString("is_contiguous")))
    return NULL;
  return PyModule_Create(&module);
}
