// The binding's argument check: a tensor's address if it is contiguous, of the wanted type
// and shape, and on the wanted GPU.  Ten of them per call took 0.45 us each through the
// interpreter (a call's launch takes 2.5); here each takes a tenth of that.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

bool same_shape(const at::Tensor& t, PyObject* shape) {
  const Py_ssize_t n = PyTuple_GET_SIZE(shape);
  if (t.dim() != n) return false;
  for (Py_ssize_t i = 0; i < n; ++i) {
    const long long v = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    if (v == -1 && PyErr_Occurred()) return false;
    if (t.size(i) != v) return false;
  }
  return true;
}

// What is wrong with t, as a ValueError.
PyObject* misfit(PyObject* t, PyObject* name, PyObject* dtype, PyObject* shape, long device) {
  if (PyErr_Occurred()) return nullptr;
  PyObject* have[4] = {PyObject_GetAttrString(t, "dtype"), PyObject_GetAttrString(t, "shape"),
                       PyObject_GetAttrString(t, "device"),
                       PyObject_CallMethod(t, "is_contiguous", nullptr)};
  PyObject* size = have[1] ? PySequence_Tuple(have[1]) : nullptr;
  if (have[0] && size && have[2] && have[3])
    PyErr_Format(PyExc_ValueError,
                 "%U must be a contiguous %S tensor of shape %S on cuda:%ld, got %S %S on %S%s", name,
                 dtype, shape, device, have[0], size, have[2],
                 PyObject_IsTrue(have[3]) == 1 ? "" : ", not contiguous");
  Py_XDECREF(size);
  for (PyObject* x : have) Py_XDECREF(x);
  return nullptr;
}

// tensor(t, name, dtype, shape, device, optional=True)
PyObject* tensor(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n < 5 || n > 6 || !PyUnicode_Check(a[1]) || !THPDtype_Check(a[2]) || !PyTuple_Check(a[3]) ||
      !PyLong_Check(a[4])) {
    PyErr_SetString(PyExc_TypeError, "tensor(t, name, dtype, shape, device, optional=True)");
    return nullptr;
  }
  if (a[0] == Py_None) {
    if (n < 6 || PyObject_IsTrue(a[5]) == 1) Py_RETURN_NONE;
    return PyErr_Format(PyExc_ValueError, "%U is required", a[1]);
  }
  if (!THPVariable_Check(a[0]))
    return PyErr_Format(PyExc_ValueError, "%U must be a tensor", a[1]);
  const long device = PyLong_AsLong(a[4]);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  try {
    const at::Tensor& t = THPVariable_Unpack(a[0]);
    if (t.scalar_type() == reinterpret_cast<THPDtype*>(a[2])->scalar_type &&
        same_shape(t, a[3]) && t.get_device() == device && t.is_contiguous())
      return PyLong_FromVoidPtr(t.data_ptr());
  } catch (const std::exception& e) {   // a tensor without storage, for one
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  return misfit(a[0], a[1], a[2], a[3], device);
}

PyMethodDef methods[] = {
    {"tensor", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tensor)), METH_FASTCALL,
     "Pointer of a contiguous tensor of this type and shape on this GPU (or None)."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

// Whether these are the PyTorch and the Python that the module was built for: in others the
// objects above need not look the same.
bool built_for_this() {
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
  PyObject* here = version ? PyUnicode_FromFormat("PyTorch %S, %s", version, PyImport_GetMagicTag())
                           : nullptr;
  const bool same = here && PyUnicode_CompareWithASCIIString(here, RKV_BUILT_FOR) == 0;
  if (here && !same)
    PyErr_Format(PyExc_ImportError, "it was built for %s, this is %U", RKV_BUILT_FOR, here);
  Py_XDECREF(here);
  Py_XDECREF(version);
  Py_XDECREF(torch);
  return same;
}

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return built_for_this() ? PyModule_Create(&module) : nullptr; }
