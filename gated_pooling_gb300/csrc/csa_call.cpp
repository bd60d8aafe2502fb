// csa_call.cpp -- the entry points that enqueue work, called from Python: the library's own functions behind
// positional arguments, and nothing else. A tensor stands for its data pointer (its data_ptr()), an int for
// itself or for an address, None for NULL; what comes back is the status.
//
// ctypes takes 0.1 us an argument and its Python side as much again for a pointer: 6 us for the 27 arguments of a
// step, more than the GPU works on a small one. So it takes 1. Where this module is not built for a Python, the package
// goes through ctypes.
#include <Python.h>

#include <cstdint>
#include <limits>
#include <tuple>
#include <type_traits>
#include <utility>

#include "csa_compressor.h"

namespace {

PyObject* g_data_ptr;  // "data_ptr"

// One argument as the C function takes it; false with a Python error set where it cannot be one.
template <typename T>
bool convert(PyObject* o, T& v) {
  if constexpr (std::is_pointer_v<T>) {
    if (o == Py_None) {
      v = nullptr;
      return true;
    }
    PyObject* address = PyLong_Check(o) ? Py_NewRef(o) : PyObject_CallMethodNoArgs(o, g_data_ptr);
    if (address == nullptr) return false;
    const unsigned long long a = PyLong_AsUnsignedLongLong(address);
    Py_DECREF(address);
    v = reinterpret_cast<T>(static_cast<uintptr_t>(a));
  } else if constexpr (std::is_floating_point_v<T>) {
    v = static_cast<T>(PyFloat_AsDouble(o));
  } else {
    static_assert(std::is_integral_v<T>, "a pointer or a number");
    if constexpr (std::is_unsigned_v<T>) {
      v = static_cast<T>(PyLong_AsUnsignedLongLong(o));
    } else {
      const long long a = PyLong_AsLongLong(o);
      if (a < std::numeric_limits<T>::min() || a > std::numeric_limits<T>::max()) {
        PyErr_Format(PyExc_OverflowError, "%lld is out of an argument's range", a);
        return false;
      }
      v = static_cast<T>(a);
    }
  }
  return PyErr_Occurred() == nullptr;
}

template <typename... A, size_t... I>
PyObject* call(csa_status_t (*f)(A...), PyObject* const* args, Py_ssize_t n, std::index_sequence<I...>) {
  if (n != static_cast<Py_ssize_t>(sizeof...(A)))
    return PyErr_Format(PyExc_TypeError, "%zd arguments instead of %zu", n, sizeof...(A));
  std::tuple<A...> v;
  if (!(convert(args[I], std::get<I>(v)) && ...)) return nullptr;
  csa_status_t status;
  Py_BEGIN_ALLOW_THREADS status = f(std::get<I>(v)...);
  Py_END_ALLOW_THREADS return PyLong_FromLong(status);
}
template <typename... A>
PyObject* call(csa_status_t (*f)(A...), PyObject* const* args, Py_ssize_t n) {
  return call(f, args, n, std::index_sequence_for<A...>{});
}

#define CSA_CALL(name) \
  PyObject* py_##name(PyObject*, PyObject* const* args, Py_ssize_t n) { return call(name, args, n); }
#define CSA_CALLS(X)                                                                                       \
  X(csa_compressor_fwd) X(csa_compressor_bwd) X(csa_compressor_bwd_noalloc) X(csa_compressor_step)          \
  X(csa_compressor_map_blocks) X(csa_kpool_fwd) X(csa_norm_rope_fwd) X(csa_norm_rope_bwd) X(csa_cache_write) \
  X(csa_cache_append) X(csa_cache_read) X(csa_cache_attn) X(csa_cache_attn_prefix)
CSA_CALLS(CSA_CALL)

#define CSA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr},
PyMethodDef g_methods[] = {CSA_CALLS(CSA_METHOD){nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_csa_call", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__csa_call() {
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  return g_data_ptr == nullptr ? nullptr : PyModule_Create(&g_module);
}
