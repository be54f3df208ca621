// Argument check of the binding: whether a torch tensor is contiguous, of a
// dtype and shape and on a device, and its data pointer.  A call of a small
// operator checks five to eight tensors; from Python each takes 0.45 us of the
// 6 us that the call takes the host, from here 0.1.
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

namespace {

// pointer(tensor, dtype, shape, device index) -> address, or None where the tensor differs
PyObject* pointer(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4 || !THPVariable_Check(args[0]) || !THPDtype_Check(args[1]) || !PyTuple_Check(args[2])) {
    PyErr_SetString(PyExc_TypeError, "expected (tensor, dtype, tuple, device index)");
    return nullptr;
  }
  const long dev = PyLong_AsLong(args[3]);
  if (dev == -1 && PyErr_Occurred()) return nullptr;
  const Py_ssize_t dims = PyTuple_GET_SIZE(args[2]);
  try {
    const at::Tensor& t = THPVariable_Unpack(args[0]);
    bool same = t.scalar_type() == reinterpret_cast<THPDtype*>(args[1])->scalar_type && t.layout() == at::kStrided && t.is_cuda() &&
                t.get_device() == dev && t.dim() == dims && t.is_contiguous();
    for (Py_ssize_t i = 0; same && i < dims; ++i) {
      const long long s = PyLong_AsLongLong(PyTuple_GET_ITEM(args[2], i));
      if (s == -1 && PyErr_Occurred()) return nullptr;
      same = t.size(i) == s;
    }
    if (!same) Py_RETURN_NONE;
    return PyLong_FromVoidPtr(t.data_ptr());
  } catch (const std::exception& e) {  // a tensor without storage
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {{"pointer", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(pointer)), METH_FASTCALL,
                          "pointer(tensor, dtype, shape, device index) -> address, or None where the tensor differs"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__args() { return PyModule_Create(&module); }
