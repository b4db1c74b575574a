// tensor.cpp — the softmax layers' calls' checks of a tensor argument, as one
// step for the interpreter (module _tensor).  A token's worth of such calls is
// bound by the host: asked of torch attribute by attribute, a tensor costs 0.3
// us (a strided one 0.5) of the 8 to 10 us that a call took; here 0.07.  Each
// function returns None for whatever it does not pass: the binding then asks
// again in words.
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

namespace {

// address of a contiguous tensor of this type, size and device: (tensor, dtype, numel, device index)
PyObject* address(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4 || !THPVariable_Check(a[0]) || !THPDtype_Check(a[1])) Py_RETURN_NONE;
  const long long want = PyLong_AsLongLong(a[2]), index = PyLong_AsLongLong(a[3]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  try {
    const at::Tensor& t = THPVariable_Unpack(a[0]);
    if (t.defined() && t.is_cuda() && t.get_device() == index && t.numel() == want && t.is_contiguous() &&
        t.scalar_type() == reinterpret_cast<THPDtype*>(a[1])->scalar_type)
      return PyLong_FromUnsignedLongLong((unsigned long long)t.data_ptr());
  } catch (...) {
  }
  Py_RETURN_NONE;
}

// (address, elements between tokens) of a tensor [tokens][heads][d] whose heads are contiguous
// within a token: (tensor, tokens, heads, d, device index), any of the last four None for "any"
PyObject* rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5 || !THPVariable_Check(a[0])) Py_RETURN_NONE;
  long long want[4];
  for (int i = 0; i < 4; i++) {
    want[i] = a[1 + i] == Py_None ? -1 : PyLong_AsLongLong(a[1 + i]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    if (a[1 + i] != Py_None && want[i] < 0) Py_RETURN_NONE;
  }
  try {
    const at::Tensor& t = THPVariable_Unpack(a[0]);
    if (!t.defined() || !t.is_cuda() || t.dim() != 3 || (want[3] >= 0 && t.get_device() != want[3])) Py_RETURN_NONE;
    const auto size = t.sizes(), step = t.strides();
    for (int i = 0; i < 3; i++)
      if (want[i] >= 0 && size[i] != want[i]) Py_RETURN_NONE;
    const long long row = size[1] * size[2];
    if (step[2] != 1 || (size[1] > 1 && step[1] != size[2])) Py_RETURN_NONE;
    return Py_BuildValue("(KL)", (unsigned long long)t.data_ptr(), size[0] > 1 ? (long long)step[0] : row);
  } catch (...) {
  }
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"address", (PyCFunction)(void (*)(void))address, METH_FASTCALL, "address(tensor, dtype, numel, index)"},
    {"rows", (PyCFunction)(void (*)(void))rows, METH_FASTCALL, "rows(tensor, tokens, heads, d, index)"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor", "checks of tensor arguments", -1, methods};

}  // namespace

// (nothing of torch is called here: the binding compares the version first)
PyMODINIT_FUNC PyInit__tensor(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
