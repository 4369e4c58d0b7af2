// The checks of tensor arguments that cache.py makes of every call, as a Python extension: asked through
// Python's attributes one by one they took a third of a small call (an append of nine tensors 8.8 us on the
// host, with these 5.4).  What a function does not accept it hands to the check in Python, which says what is
// wrong with it (`otherwise`).
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool is_type(const at::Tensor& t, PyObject* dtype) {
  return THPDtype_Check(dtype) && reinterpret_cast<THPDtype*>(dtype)->scalar_type == t.scalar_type();
}

PyObject* address(const at::Tensor& t) { return PyLong_FromVoidPtr(t.data_ptr()); }

// A size or device index; None: -1, any.  False and an exception where it is not a whole number.
bool number(PyObject* o, int64_t* v) {
  *v = o == Py_None ? -1 : PyLong_AsLongLong(o);
  return !(*v == -1 && PyErr_Occurred());
}

enum { VEC, MAT, TABLE, VIEW, CHECKS };
PyObject* in_python[CHECKS];  // the same checks in Python

// What `f` gives for a tensor; otherwise what the check in Python does.
template <typename F>
PyObject* ask(int check, PyObject* const* a, Py_ssize_t nargs, F f) {
  try {
    const at::Tensor* t = tensor(a[0]);
    PyObject* r = t ? f(*t) : nullptr;
    if (r || PyErr_Occurred()) return r;
  } catch (const std::exception&) {  // (a tensor without sizes or an address)
  }
  if (!in_python[check]) {
    PyErr_SetString(PyExc_RuntimeError, "otherwise() was not called");
    return nullptr;
  }
  return PyObject_Vectorcall(in_python[check], a, nargs, nullptr);
}

bool arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return n == want;
}

// vec(t, name, dtype, n, device): the address of a contiguous vector of n elements
PyObject* vec(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  int64_t n, device;
  if (!arguments(nargs, 5) || !number(a[3], &n) || !number(a[4], &device)) return nullptr;
  return ask(VEC, a, nargs, [&](const at::Tensor& t) -> PyObject* {
    if (!is_type(t, a[2]) || t.get_device() != device || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
      return nullptr;
    return address(t);
  });
}

// mat(t, name, dtypes, rows, cols, device): (address, row stride) of a matrix with contiguous rows; None: any
PyObject* mat(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  int64_t rows, cols, device;
  if (!arguments(nargs, 6) || !number(a[3], &rows) || !number(a[4], &cols) || !number(a[5], &device)) return nullptr;
  if (!PyTuple_Check(a[2])) {
    PyErr_SetString(PyExc_TypeError, "dtypes are a tuple");
    return nullptr;
  }
  return ask(MAT, a, nargs, [&](const at::Tensor& t) -> PyObject* {
    bool known = false;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(a[2]); ++i) known |= is_type(t, PyTuple_GET_ITEM(a[2], i));
    if (!known || t.get_device() != device || t.dim() != 2) return nullptr;
    const int64_t r = t.size(0), c = t.size(1), stride = t.stride(0);
    if ((rows >= 0 && r != rows) || (cols >= 0 && c != cols) || (c > 1 && t.stride(1) != 1) || (r > 1 && stride < c))
      return nullptr;
    return Py_BuildValue("(NL)", address(t), (long long)(r > 1 ? stride : c));
  });
}

// table(t, name, rows, device): the address of a contiguous int32 matrix; None: any rows
PyObject* table(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  int64_t rows, device;
  if (!arguments(nargs, 4) || !number(a[2], &rows) || !number(a[3], &device)) return nullptr;
  return ask(TABLE, a, nargs, [&](const at::Tensor& t) -> PyObject* {
    if (t.scalar_type() != at::kInt || t.get_device() != device || t.dim() != 2 || (rows >= 0 && t.size(0) != rows) ||
        !t.is_contiguous())
      return nullptr;
    return address(t);
  });
}

// pages(t, name, block_size, record, device): (address, strides of pages and records, pages) of a cache
PyObject* pages(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  int64_t block, record, device;
  if (!arguments(nargs, 5) || !number(a[2], &block) || !number(a[3], &record) || !number(a[4], &device)) return nullptr;
  return ask(VIEW, a, nargs, [&](const at::Tensor& t) -> PyObject* {
    if (t.scalar_type() != at::kByte || t.get_device() != device || t.dim() != 3 || t.size(1) != block ||
        t.size(2) < record || t.stride(2) != 1)
      return nullptr;
    return Py_BuildValue("(NLLL)", address(t), (long long)t.stride(0), (long long)t.stride(1), (long long)t.size(0));
  });
}

// otherwise(vec, mat, table, pages): the checks in Python
PyObject* otherwise(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (!arguments(nargs, CHECKS)) return nullptr;
  for (int i = 0; i < CHECKS; ++i) {
    Py_INCREF(a[i]);
    PyObject* old = in_python[i];
    in_python[i] = a[i];
    Py_XDECREF(old);
  }
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"vec", (PyCFunction)(void (*)())vec, METH_FASTCALL, nullptr},
                         {"mat", (PyCFunction)(void (*)())mat, METH_FASTCALL, nullptr},
                         {"table", (PyCFunction)(void (*)())table, METH_FASTCALL, nullptr},
                         {"pages", (PyCFunction)(void (*)())pages, METH_FASTCALL, nullptr},
                         {"otherwise", (PyCFunction)(void (*)())otherwise, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__args() {
  PyObject* m = PyModule_Create(&module);
  // the version that it is for; what cache.py expects of it
  if (m && (PyModule_AddStringConstant(m, "TORCH", ARGS_TORCH) || PyModule_AddIntConstant(m, "INTERFACE", 2))) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
