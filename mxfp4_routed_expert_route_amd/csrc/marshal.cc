// Argument checks of the Python binding, natively: the pointer of a tensor that has the expected
// type, shape, GPU and contiguity.  Ten such checks in Python cost as much host time as the
// launches of a small call (0.45 us each, here 0.1).  What is wrong with an argument is said by
// the Python function given to set_refuse, which raises.
#include <exception>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject* refuse = nullptr;

// arg(tensor, dtypes, shape, device, name) -> address
PyObject* arg(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  if (n == 5 && THPVariable_Check(a[0]) && PyTuple_Check(a[1]) && PyTuple_Check(a[2])) {
    const at::Tensor& t = THPVariable_Unpack(a[0]);
    const long dev = PyLong_AsLong(a[3]);
    if (dev == -1 && PyErr_Occurred()) return nullptr;
    bool ok = dev >= 0 && t.layout() == at::kStrided && t.is_cuda() && t.get_device() == dev && t.is_contiguous();
    const Py_ssize_t dims = PyTuple_GET_SIZE(a[2]);
    ok = ok && t.dim() == dims;
    for (Py_ssize_t i = 0; ok && i < dims; ++i) {
      const long long d = PyLong_AsLongLong(PyTuple_GET_ITEM(a[2], i));
      if (d == -1 && PyErr_Occurred()) return nullptr;
      ok = t.size(i) == d;
    }
    bool type = false;
    for (Py_ssize_t i = 0; ok && !type && i < PyTuple_GET_SIZE(a[1]); ++i) {
      PyObject* d = PyTuple_GET_ITEM(a[1], i);
      type = THPDtype_Check(d) && reinterpret_cast<THPDtype*>(d)->scalar_type == t.scalar_type();
    }
    if (ok && type) return PyLong_FromVoidPtr(t.data_ptr());
  }
  if (refuse == nullptr) {
    PyErr_SetString(PyExc_ValueError, "unsuitable argument");
    return nullptr;
  }
  return PyObject_Vectorcall(refuse, a, static_cast<size_t>(n), nullptr);
} catch (const std::exception& e) {   // a tensor without storage, for one
  PyErr_SetString(PyExc_ValueError, e.what());
  return nullptr;
}

PyObject* set_refuse(PyObject*, PyObject* fn) {
  Py_XINCREF(fn);
  Py_XDECREF(refuse);
  refuse = fn;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"arg", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(arg)), METH_FASTCALL, nullptr},
    {"set_refuse", set_refuse, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
