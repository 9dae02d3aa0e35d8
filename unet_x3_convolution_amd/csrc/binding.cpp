// Python calls of the operators around and in a block, by their C signatures.
//
// These take up to 37 arguments and enqueue kernels of a few microseconds: through
// ctypes, with an address asked of each tensor in Python, a call took 5.5 us of the
// host's time, more than the kernel; here 1.2.  An argument is converted by the
// parameter's type: pointers from None, whole numbers or what has a data_ptr() (torch
// tensors), numbers with a check of their range.  The interpreter's lock is released
// during the call, as ctypes does.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>
#include <tuple>
#include <type_traits>
#include <utility>

#include "../../include/oidn_mi355x.h"

namespace {

PyObject* g_data_ptr;      // the interned method name

bool to_address(PyObject* o, void*& out) {
  if (o == Py_None) {
    out = nullptr;
    return true;
  }
  PyObject* n = o;
  if (PyLong_Check(o)) Py_INCREF(n);
  else if (!(n = PyObject_CallMethodNoArgs(o, g_data_ptr))) return false;
  out = PyLong_AsVoidPtr(n);
  Py_DECREF(n);
  return !PyErr_Occurred();
}

template <typename T>
bool convert(PyObject* o, T& out) {
  if constexpr (std::is_pointer_v<T>) {
    void* p;
    if (!to_address(o, p)) return false;
    out = static_cast<T>(p);
    return true;
  } else if constexpr (std::is_floating_point_v<T>) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) return false;
    out = static_cast<T>(v);
    if (std::isfinite(out) || !std::isfinite(v)) return true;
    PyErr_Format(PyExc_OverflowError, "%R does not fit the parameter", o);
    return false;
  } else if constexpr (std::is_same_v<T, size_t>) {
    out = PyLong_AsSize_t(o);
    return !PyErr_Occurred();
  } else {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return false;
    out = static_cast<T>(v);
    if (static_cast<long>(out) == v) return true;
    PyErr_Format(PyExc_OverflowError, "%ld does not fit the parameter", v);
    return false;
  }
}

template <auto F>
struct Call;
template <typename... A, int (*F)(A...)>
struct Call<F> {
  template <size_t... I>
  static bool convert_all(std::tuple<A...>& to, PyObject* const* args, std::index_sequence<I...>) {
    return (convert(args[I], std::get<I>(to)) && ...);
  }
  static PyObject* run(PyObject*, PyObject* const* args, Py_ssize_t count) {
    if (count != static_cast<Py_ssize_t>(sizeof...(A)))
      return PyErr_Format(PyExc_TypeError, "%zd arguments given, %zu taken", count, sizeof...(A));
    std::tuple<A...> values;
    if (!convert_all(values, args, std::index_sequence_for<A...>{})) return nullptr;
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = std::apply(F, values);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
  }
};

template <auto F>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&Call<F>::run)), METH_FASTCALL, nullptr};
}
#define OIDN_METHOD(name) method<name>(#name)
PyMethodDef g_methods[] = {
    OIDN_METHOD(oidn_fp8_pack),
    OIDN_METHOD(oidn_fp8_unpack),
    OIDN_METHOD(oidn_linear_fp8),
    OIDN_METHOD(oidn_linear_fp8_backward),
    OIDN_METHOD(oidn_norm),
    OIDN_METHOD(oidn_norm_backward),
    OIDN_METHOD(oidn_norm_residual),
    OIDN_METHOD(oidn_norm_residual_backward),
    OIDN_METHOD(oidn_dropout),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  return g_data_ptr ? PyModule_Create(&g_module) : nullptr;
}
