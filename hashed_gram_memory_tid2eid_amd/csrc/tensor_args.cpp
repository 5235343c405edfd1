// tensor_args.cpp -- the checks of a tensor argument and its address in one native call, for the
// Python binding.  A serving call has up to 13 tensors; checked in Python they cost 0.27 us each
// and more than the launch (plan of 256 rows: 8.4 us a call, 6.0 with this).  Built as
// the extension module _tensor_args against the installed torch; the library itself stays a
// plain C ABI without it.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <c10/core/impl/VirtualGuardImpl.h>

#include <exception>
#include <string>

namespace {

// The tensor behind a Python object, or null with an exception set.
const at::Tensor* tensor_of(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) {
    PyErr_Format(PyExc_TypeError, "%s must be a device tensor", name);
    return nullptr;
  }
  return &t;
}

bool right_place(const at::Tensor& t, const char* name, long dev) {
  if (t.get_device() == dev) return true;
  PyErr_Format(PyExc_ValueError, "%s is on device %ld, the call on device %ld", name, (long)t.get_device(), dev);
  return false;
}

bool right_type(const at::Tensor& t, const char* name, PyObject* dtype) {
  if (!THPDtype_Check(dtype)) {
    PyErr_SetString(PyExc_TypeError, "a dtype is wanted");
    return false;
  }
  const at::ScalarType want = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
  if (t.scalar_type() == want) return true;
  PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(want), c10::toString(t.scalar_type()));
  return false;
}

// No exception leaves a call.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a tensor argument could not be read");
  }
  return nullptr;
}

bool wants(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, got);
  return false;
}

// device(t, name): the device of a call, which must be the current one.
PyObject* device(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!wants(n, 2)) return nullptr;
    const char* name = PyUnicode_AsUTF8(a[1]);
    const at::Tensor* t = name ? tensor_of(a[0], name) : nullptr;
    if (!t) return nullptr;
    const long dev = t->get_device(), now = c10::impl::getDeviceGuardImpl(c10::DeviceType::CUDA)->getDevice().index();
    if (dev != now) {
      PyErr_Format(PyExc_ValueError, "%s is on device %ld, the current device is %ld", name, dev, now);
      return nullptr;
    }
    return PyLong_FromLong(dev);
  });
}

// address(t, name, dtype, least, dev): address of a contiguous tensor of this type with at least
// so many elements on that device; None for None.
PyObject* address(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!wants(n, 5)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;
    const char* name = PyUnicode_AsUTF8(a[1]);
    const at::Tensor* t = name ? tensor_of(a[0], name) : nullptr;
    if (!t || !right_type(*t, name, a[2])) return nullptr;
    const long long least = PyLong_AsLongLong(a[3]);
    const long dev = PyLong_AsLong(a[4]);
    if (PyErr_Occurred() || !right_place(*t, name, dev)) return nullptr;
    if (t->numel() < least) {
      PyErr_Format(PyExc_ValueError, "%s too small: %lld elements, %lld needed", name, (long long)t->numel(), least);
      return nullptr;
    }
    if (!t->is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
      return nullptr;
    }
    return PyLong_FromVoidPtr(t->data_ptr());
  });
}

// matrix(t, name, dtype or None, dev): (address, rows, columns, leading dimension) of a matrix
// whose rows are contiguous and do not overlap.  Rows and columns fit the library's 32-bit
// arguments: ctypes would cut them down without a word.
PyObject* matrix(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!wants(n, 4)) return nullptr;
    const char* name = PyUnicode_AsUTF8(a[1]);
    const at::Tensor* t = name ? tensor_of(a[0], name) : nullptr;
    if (!t || (a[2] != Py_None && !right_type(*t, name, a[2]))) return nullptr;
    const long dev = PyLong_AsLong(a[3]);
    if (PyErr_Occurred() || !right_place(*t, name, dev)) return nullptr;
    if (t->dim() != 2) {
      PyErr_Format(PyExc_ValueError, "%s must be a matrix", name);
      return nullptr;
    }
    const int64_t rows = t->size(0), cols = t->size(1);
    if (rows >> 31 != 0 || cols >> 31 != 0) {
      PyErr_Format(PyExc_ValueError, "%s must have fewer than 2^31 rows and columns, got %lld x %lld", name, (long long)rows,
                   (long long)cols);
      return nullptr;
    }
    if (cols > 1 && t->stride(1) != 1) {
      PyErr_Format(PyExc_ValueError, "%s must have contiguous rows", name);
      return nullptr;
    }
    const int64_t ld = rows <= 1 ? cols : t->stride(0);
    if (ld < cols) {
      PyErr_Format(PyExc_ValueError, "%s must not have overlapping rows", name);
      return nullptr;
    }
    return Py_BuildValue("(NLLL)", PyLong_FromVoidPtr(t->data_ptr()), (long long)rows, (long long)cols, (long long)ld);
  });
}

PyMethodDef methods[] = {
    {"device", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(device)), METH_FASTCALL, nullptr},
    {"address", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(address)), METH_FASTCALL, nullptr},
    {"matrix", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(matrix)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", "Checked addresses of tensor arguments.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// TENSOR_ARGS_TORCH is the torch it was built for, with which alone it is used; TENSOR_ARGS_ID a hash of
// everything it was built from and for.
PyMODINIT_FUNC PyInit__tensor_args() {
  PyObject* m = PyModule_Create(&module);
  if (m && (PyModule_AddStringConstant(m, "torch_version", TENSOR_ARGS_TORCH) != 0 ||
            PyModule_AddStringConstant(m, "build_id", TENSOR_ARGS_ID) != 0)) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
