// Argument checks of the Python binding's row operators in one native call: each takes
// about ten tensors, and asking every one of them from Python for its device, type, shape,
// layout and address costs as much as launching the kernel. Nothing here touches the GPU.
//
// dense(device, tensor, dtype, shape, tensor, dtype, shape, ...) returns the tensors'
// addresses (None for None), or the number of the first that is not a dense tensor of that
// type and shape on that device. matrix(device, tensor, dtype, shape) returns (address,
// elements from row to row) of a two-dimensional one whose rows may be spaced, or None if
// it is not one. The caller words the error.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

namespace {

constexpr long long kEmpty = 256;  // address of a tensor without elements: nothing of it is accessed

bool same(const at::Tensor& t, long dev, PyObject* dtype, PyObject* shape) {
  if (!t.is_cuda() || t.get_device() != dev) return false;
  if (!THPDtype_Check(dtype) || t.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type) return false;
  if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != t.dim()) return false;
  for (int64_t i = 0; i < t.dim(); ++i)
    if (PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i)) != t.size(i)) return false;
  return true;
}

PyObject* address(const at::Tensor& t) {
  const auto p = t.numel() ? reinterpret_cast<uintptr_t>(t.const_data_ptr()) : (uintptr_t)kEmpty;
  return PyLong_FromUnsignedLongLong((unsigned long long)p);
}

PyObject* dense(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n < 1 || (n - 1) % 3) {
    PyErr_SetString(PyExc_TypeError, "dense(device, tensor, dtype, shape, ...)");
    return nullptr;
  }
  const long dev = PyLong_AsLong(args[0]);
  if (PyErr_Occurred()) return nullptr;
  const Py_ssize_t m = (n - 1) / 3;
  THPObjectPtr out(PyTuple_New(m));
  if (!out) return nullptr;
  for (Py_ssize_t i = 0; i < m; ++i) {
    PyObject* o = args[1 + 3 * i];
    PyObject* p = nullptr;
    if (o == Py_None) {
      Py_INCREF(Py_None);
      p = Py_None;
    } else if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (same(t, dev, args[2 + 3 * i], args[3 + 3 * i]) && t.is_contiguous()) p = address(t);
    }
    if (!p) return PyErr_Occurred() ? nullptr : PyLong_FromSsize_t(i);
    PyTuple_SET_ITEM(out.get(), i, p);
  }
  return out.release();
  END_HANDLE_TH_ERRORS
}

PyObject* matrix(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "matrix(device, tensor, dtype, shape)");
    return nullptr;
  }
  const long dev = PyLong_AsLong(args[0]);
  if (PyErr_Occurred()) return nullptr;
  if (!THPVariable_Check(args[1])) Py_RETURN_NONE;
  const at::Tensor& t = THPVariable_Unpack(args[1]);
  if (t.dim() != 2 || !same(t, dev, args[2], args[3])) {
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  }
  const int64_t cols = t.size(1), ld = t.size(0) > 1 ? t.stride(0) : cols;
  if ((cols > 1 && t.stride(1) != 1) || ld < cols) Py_RETURN_NONE;
  PyObject* p = address(t);
  return p ? Py_BuildValue("NL", p, (long long)ld) : nullptr;
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"dense", (PyCFunction)(void (*)(void))dense, METH_FASTCALL, "addresses of dense tensors, or the first wrong one"},
    {"matrix", (PyCFunction)(void (*)(void))matrix, METH_FASTCALL, "address and row spacing of a matrix, or None"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
