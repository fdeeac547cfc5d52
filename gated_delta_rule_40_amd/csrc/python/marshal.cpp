// marshal.cpp -- the binding's tensor checks as a CPython extension.
//
// Every call of the library checks each tensor it is given (shape, dtype,
// device, contiguity) and takes its address.  In Python that is 0.4 us a
// tensor, which for a single-token call of ten tensors is as long as the launch;
// here it is 0.1 us.  What does not fit goes back to a Python function, which
// says what is wrong.
#include <Python.h>

#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject* refuse = nullptr;  // called with the arguments that did not fit; raises

// Whether t is a dense tensor of exactly this shape, dtype and device.
bool fits(PyObject* t, PyObject* shape, PyObject* dtype, PyObject* device) {
  if (!THPVariable_Check(t) || !PyTuple_Check(shape) || !THPDtype_Check(dtype) ||
      !THPDevice_Check(device))
    return false;
  const at::Tensor& x = THPVariable_Unpack(t);
  if (x.layout() != at::kStrided ||
      x.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type ||
      x.device() != reinterpret_cast<THPDevice*>(device)->device)
    return false;
  const auto sizes = x.sizes();
  const Py_ssize_t n = PyTuple_GET_SIZE(shape);
  if (static_cast<Py_ssize_t>(sizes.size()) != n) return false;
  for (Py_ssize_t i = 0; i < n; ++i) {
    const long long s = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    if (s == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
    if (s != sizes[i]) return false;
  }
  return x.is_contiguous();
}

PyObject* address(PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "expected (tensor, name, shape, dtype, device)");
    return nullptr;
  }
  try {
    if (fits(a[0], a[2], a[3], a[4]))
      return PyLong_FromUnsignedLongLong(
          reinterpret_cast<unsigned long long>(THPVariable_Unpack(a[0]).data_ptr()));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  if (!refuse) {
    PyErr_SetString(PyExc_ValueError, "tensor does not fit the call");
    return nullptr;
  }
  PyObject* r = PyObject_CallFunctionObjArgs(refuse, a[0], a[1], a[2], a[3], a[4], nullptr);
  if (r) {  // it has to raise
    Py_DECREF(r);
    PyErr_SetString(PyExc_ValueError, "tensor does not fit the call");
  }
  return nullptr;
}

// ptr(tensor, name, shape, dtype, device) -> address
PyObject* ptr(PyObject*, PyObject* const* a, Py_ssize_t n) { return address(a, n); }

// The same, None for None.
PyObject* opt(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n > 0 && a[0] == Py_None) Py_RETURN_NONE;
  return address(a, n);
}

PyObject* on_refusal(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(refuse, f);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"ptr", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(ptr)), METH_FASTCALL,
     "Address of a dense tensor of exactly this shape, dtype and device."},
    {"opt", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(opt)), METH_FASTCALL,
     "ptr, or None for None."},
    {"on_refusal", on_refusal, METH_O, "Sets the function that raises for what does not fit."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
