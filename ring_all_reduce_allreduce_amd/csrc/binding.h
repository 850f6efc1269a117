// binding.h -- what the sources of the Python extension _ops_binding share:
// errors, arguments as tensors and numbers, checks, allocation on the current
// stream, results.
#pragma once

#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/ringsim_ops.h"

namespace ringsim_binding {

extern PyObject* g_ringsim_error;  // RingsimError of the package
extern PyObject* g_memory_error;   // torch.OutOfMemoryError

// An error that is already set in the interpreter, and errors to be set.
struct PythonError {};
struct WrongType : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct WrongValue : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Refused {
  int code;
  const char* what;
};

// Runs one call and turns what it throws into a Python exception.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const PythonError&) {
  } catch (const WrongType& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const WrongValue& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Refused& r) {
    PyObject* e = g_ringsim_error ? PyObject_CallFunction(g_ringsim_error, "is", r.code, r.what) : nullptr;
    if (e) {
      PyErr_SetObject(g_ringsim_error, e);
      Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
      PyErr_SetString(PyExc_RuntimeError, r.what);
    }
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_memory_error ? g_memory_error : PyExc_MemoryError, e.what_without_backtrace());
  } catch (const std::bad_alloc&) {
    PyErr_NoMemory();
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

inline void check(ringsim_result_t code, const char* what) {
  if (code != RINGSIM_SUCCESS) throw Refused{(int)code, what};
}

inline std::string shape_text(at::IntArrayRef s) {
  std::ostringstream o;
  o << s;
  return o.str();
}

// The tensor an argument holds; null for None.
inline const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw WrongType(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
inline const at::Tensor& required(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) throw WrongType(std::string(name) + " must be a tensor");
  return *t;
}

// A conversion's error: of a number that is too large a wrong value, else its own.
[[noreturn]] inline void conversion_error() {
  if (!PyErr_ExceptionMatches(PyExc_OverflowError)) throw PythonError{};
  PyErr_Clear();
  throw WrongValue("a number is out of range");
}
inline double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) conversion_error();
  return v;
}
inline long whole(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) conversion_error();
  return v;
}

inline int type_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return RINGSIM_FLOAT32;
    case at::kBFloat16: return RINGSIM_BFLOAT16;
    case at::kHalf: return RINGSIM_FLOAT16;
    default: return -1;
  }
}

inline void check_strided(const at::Tensor& t, const char* name) {
  if (t.layout() != at::kStrided) throw WrongValue(std::string(name) + " must be a strided tensor");
}
inline void check_device(const at::Tensor& t, int device, const char* name) {
  check_strided(t, name);
  if (!t.is_cuda() || t.get_device() != device)
    throw WrongValue(std::string(name) + " must be a tensor on the current device");
}

// The allocation at::empty ends in, without its way through the dispatcher
// (0.45 us against 0.7).
inline at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int device) {
  return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)device), std::nullopt);
}

// -1 on a host without a GPU, which no tensor is on.
inline int current_device() { return c10::hip::device_count() > 0 ? (int)c10::hip::current_device() : -1; }
inline ringsim_stream_t current_stream(int device) {
  return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
}

inline PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
inline PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

// The argument itself if there was one, else the new tensor, else None.
inline PyObject* result(PyObject* given, const at::Tensor& made) {
  if (given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  return made.defined() ? wrap(made) : none();
}

inline PyObject* pack(std::initializer_list<PyObject*> parts) {
  PyObject* t = PyTuple_New((Py_ssize_t)parts.size());
  Py_ssize_t i = 0;
  bool ok = t != nullptr;
  for (PyObject* p : parts) {
    ok = ok && p;
    if (t)
      PyTuple_SET_ITEM(t, i++, p);  // takes the reference, null included
    else
      Py_XDECREF(p);
  }
  if (!ok) {
    Py_XDECREF(t);
    throw PythonError{};
  }
  return t;
}

inline void want_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) throw WrongType("expected " + std::to_string(want) + " arguments");
}

inline void* data(const at::Tensor& t) { return t.data_ptr(); }

// Lets other Python threads run while a call allocates and launches, both of
// which can wait for the driver. What stands in its scope must not touch
// Python objects, and what was read from them must be held: by the caller's
// arguments, or by a list's own references.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* const state_;
};

// Says that the memory of an argument has been written, so that autograd
// notices where it had been saved. Tensors of inference mode have no version.
inline void written(PyObject* given) {
  if (given == Py_None) return;
  const at::Tensor& t = THPVariable_Unpack(given);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

inline PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

}  // namespace ringsim_binding
