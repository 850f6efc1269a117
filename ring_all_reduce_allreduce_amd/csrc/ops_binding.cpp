// ops_binding.cpp -- the Python extension module _ops_binding: checks torch
// tensors, allocates results and workspaces on the current stream, and calls
// the C ABI of include/ringsim_ops.h.
//
// Compiled, not ctypes like the collectives' binding, because it is the host
// that bounds small calls: marshalling in Python took 12-18 us a call and
// 0.4 us for every tensor of a list (here 12 to 16 ns), where the kernels of
// one token take about 4 us. operators.py holds the functions users call; arguments arrive here by
// position.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/ringsim_ops.h"

namespace {

PyObject* g_ringsim_error = nullptr;  // RingsimError of the package
PyObject* g_memory_error = nullptr;   // torch.OutOfMemoryError

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

void check(ringsim_result_t code, const char* what) {
  if (code != RINGSIM_SUCCESS) throw Refused{(int)code, what};
}

std::string shape_text(at::IntArrayRef s) {
  std::ostringstream o;
  o << s;
  return o.str();
}

// The tensor an argument holds; null for None.
const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw WrongType(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& required(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) throw WrongType(std::string(name) + " must be a tensor");
  return *t;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}
long whole(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}

int type_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return RINGSIM_FLOAT32;
    case at::kBFloat16: return RINGSIM_BFLOAT16;
    case at::kHalf: return RINGSIM_FLOAT16;
    default: return -1;
  }
}

void check_strided(const at::Tensor& t, const char* name) {
  if (t.layout() != at::kStrided) throw WrongValue(std::string(name) + " must be a strided tensor");
}
void check_device(const at::Tensor& t, int device, const char* name) {
  check_strided(t, name);
  if (!t.is_cuda() || t.get_device() != device)
    throw WrongValue(std::string(name) + " must be a tensor on the current device");
}

// The allocation at::empty ends in, without its way through the dispatcher
// (0.45 us against 0.7).
at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int device) {
  return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)device), std::nullopt);
}

// -1 on a host without a GPU, which no tensor is on.
int current_device() { return c10::hip::device_count() > 0 ? (int)c10::hip::current_device() : -1; }
ringsim_stream_t current_stream(int device) {
  return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
}

// The leading dimensions of a shape that count: those of size 1 take no part
// in where a row lies, and their strides may be anything. The last of them is
// the inner one; those before it are taken together as the outer one.
struct Leading {
  c10::SmallVector<int, 8> dims;  // from the inner one outwards
  bool no_rows = false;

  explicit Leading(at::IntArrayRef shape) {
    for (int i = (int)shape.size() - 2; i >= 0; --i) {
      if (shape[i] != 1) dims.push_back(i);
      no_rows = no_rows || shape[i] == 0;
    }
  }
};

// {outer, inner} strides of a tensor whose rows are its last dimension: up to
// two leading dimensions of any strides, or more whose outer ones follow one
// another in memory without gaps.
void rows(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, int device,
          int64_t stride[2]) {
  if (t.scalar_type() != type)
    throw WrongType(std::string(name) + " must have dtype " + c10::toString(type) + ", not " +
                    c10::toString(t.scalar_type()));
  check_strided(t, name);
  if (t.sizes() != shape)
    throw WrongValue(std::string(name) + " must have shape " + shape_text(shape) + ", not " + shape_text(t.sizes()));
  const auto st = t.strides();
  if (shape.back() > 1 && st.back() != 1)
    throw WrongValue(std::string("the last dimension of ") + name + " must be contiguous");
  const Leading lead(shape);
  const auto& d = lead.dims;
  stride[0] = stride[1] = 0;
  if (!lead.no_rows) {
    for (size_t k = 2; k < d.size(); ++k)
      if (st[d[k]] != st[d[k - 1]] * shape[d[k - 1]])
        throw WrongValue(std::string("the leading dimensions of ") + name + " must be contiguous among themselves");
    if (d.size() == 1) stride[0] = st[d[0]];
    if (d.size() > 1) {
      stride[0] = st[d[1]];
      stride[1] = st[d[0]];
    }
  }
  check_device(t, device, name);
}

// [outer, inner, cols] of a shape, as rows() takes its strides.
void row_counts(at::IntArrayRef shape, int64_t* outer, int64_t* inner, int64_t* cols) {
  const Leading lead(shape);
  *cols = shape.back();
  *outer = *inner = 1;
  for (size_t k = 0; k < lead.dims.size(); ++k)
    *(k == 0 && lead.dims.size() > 1 ? inner : outer) *= shape[lead.dims[k]];
}

// Types of the normed tensor and of the weight, and the weight's shape.
void norm_types(const at::Tensor& x, const at::Tensor* w, const char* name, int device, int* code, int* wcode) {
  *code = *wcode = type_code(x.scalar_type());
  if (*code < 0) throw WrongType(std::string("unsupported dtype ") + c10::toString(x.scalar_type()) + " of " + name);
  if (x.dim() == 0) throw WrongValue(std::string(name) + " needs at least one dimension");
  if (!w) return;
  *wcode = type_code(w->scalar_type());
  if (*wcode != *code && *wcode != RINGSIM_FLOAT32)
    throw WrongType(std::string("weight must have dtype ") + c10::toString(x.scalar_type()) + " or Float, not " +
                    c10::toString(w->scalar_type()));
  if (w->dim() != 1 || w->size(0) != x.size(-1))
    throw WrongValue("weight must have shape [" + std::to_string(x.size(-1)) + "], not " + shape_text(w->sizes()));
  if (!w->is_contiguous()) throw WrongValue("weight must be contiguous");
  check_device(*w, device, "weight");
}

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

// The argument itself if there was one, else the new tensor, else None.
PyObject* result(PyObject* given, const at::Tensor& made) {
  if (given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  return made.defined() ? wrap(made) : none();
}

PyObject* pack(std::initializer_list<PyObject*> parts) {
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

void want_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) throw WrongType("expected " + std::to_string(want) + " arguments");
}

void* data(const at::Tensor& t) { return t.data_ptr(); }

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
void written(PyObject* given) {
  if (given == Py_None) return;
  const at::Tensor& t = THPVariable_Unpack(given);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// rms_norm(x, weight, residual, eps, quant, group, out, residual_out, scales)
PyObject* rms_norm(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded([&] {
    want_args(nargs, 9);
    const at::Tensor& x = required(args[0], "x");
    const at::Tensor* w = tensor(args[1], "weight");
    const at::Tensor* res = tensor(args[2], "residual");
    const bool quant = whole(args[4]) != 0;
    const int64_t group = whole(args[5]);
    const at::Tensor *out = tensor(args[6], "out"), *res_out = tensor(args[7], "residual_out"),
                     *scales = tensor(args[8], "scales");
    const int device = current_device();
    ringsim_rms_norm_t a{};
    a.eps = (float)number(args[3]);
    norm_types(x, w, "x", device, &a.dtype, &a.weight_dtype);
    a.out_dtype = quant ? (int)RINGSIM_FLOAT8_E4M3 : a.dtype;
    if (group != 0 && !(quant && (group == 32 || group == 64 || group == 128)))
      throw WrongValue("unsupported group " + std::to_string(group));
    if (!res && res_out) throw WrongValue("residual_out needs a residual");
    if (!quant && scales) throw WrongValue("scales come with an output in 8 bits");
    const auto shape = x.sizes();
    const auto type = x.scalar_type(), out_type = quant ? at::kFloat8_e4m3fn : type;
    rows(x, "x", shape, type, device, a.x_stride);
    if (res) rows(*res, "residual", shape, type, device, a.residual_stride);
    if (out) rows(*out, "out", shape, out_type, device, a.out_stride);
    if (res_out) rows(*res_out, "residual_out", shape, type, device, a.residual_out_stride);
    c10::SmallVector<int64_t, 5> scale_shape(shape.begin(), shape.end());
    scale_shape.back() = group ? (shape.back() + group - 1) / group : 1;
    if (scales) {
      if (scales->scalar_type() != at::kFloat || scales->sizes() != at::IntArrayRef(scale_shape) ||
          !scales->is_contiguous())
        throw WrongValue("scales must be contiguous float32 of shape " + shape_text(scale_shape));
      check_device(*scales, device, "scales");
    }
    row_counts(shape, &a.outer, &a.inner, &a.cols);
    a.group = (int)group;
    at::Tensor made_out, made_res, made_scales;
    {
      const Unlocked unlocked;
      if (!out) {
        made_out = empty(shape, out_type, device);
        rows(made_out, "out", shape, out_type, device, a.out_stride);
        out = &made_out;
      }
      if (res && !res_out) {
        made_res = empty(shape, type, device);
        rows(made_res, "residual_out", shape, type, device, a.residual_out_stride);
        res_out = &made_res;
      }
      if (quant && !scales) {
        made_scales = empty(scale_shape, at::kFloat, device);
        scales = &made_scales;
      }
      a.x = data(x);
      a.residual = res ? data(*res) : nullptr;
      a.weight = w ? data(*w) : nullptr;
      a.out = data(*out);
      a.residual_out = res ? data(*res_out) : nullptr;
      a.scales = quant ? static_cast<float*>(data(*scales)) : nullptr;
      check(ringsim_rms_norm(&a, current_stream(device)), "ringsim_rms_norm");
    }
    for (int i = 6; i < 9; ++i) written(args[i]);
    return pack({result(args[6], made_out), result(args[7], made_res), result(args[8], made_scales)});
  });
}

// rms_norm_backward(grad_out, h, weight, grad_residual, eps, grad_in, grad_weight, need_grad_weight)
PyObject* rms_norm_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded([&] {
    want_args(nargs, 8);
    const at::Tensor &dy = required(args[0], "grad_out"), &h = required(args[1], "h");
    const at::Tensor *w = tensor(args[2], "weight"), *res = tensor(args[3], "grad_residual"),
                     *dx = tensor(args[5], "grad_in"), *dw = tensor(args[6], "grad_weight");
    const int device = current_device();
    ringsim_rms_norm_backward_t a{};
    a.eps = (float)number(args[4]);
    const int need = PyObject_IsTrue(args[7]);
    if (need < 0) throw PythonError{};
    norm_types(h, w, "h", device, &a.dtype, &a.weight_dtype);
    if (!w && dw) throw WrongValue("grad_weight needs a weight");
    const auto shape = h.sizes();
    const auto type = h.scalar_type();
    rows(h, "h", shape, type, device, a.h_stride);
    rows(dy, "grad_out", shape, type, device, a.grad_out_stride);
    if (res) rows(*res, "grad_residual", shape, type, device, a.grad_residual_stride);
    if (dw) {
      if (dw->scalar_type() != w->scalar_type() || dw->sizes() != w->sizes() || !dw->is_contiguous())
        throw WrongValue("grad_weight must be contiguous, of the weight's shape and dtype");
      check_device(*dw, device, "grad_weight");
    }
    if (dx) rows(*dx, "grad_in", shape, type, device, a.grad_in_stride);
    row_counts(shape, &a.outer, &a.inner, &a.cols);
    at::Tensor made_dx, made_dw, workspace;
    {
      const Unlocked unlocked;
      if (!dx) {
        made_dx = empty(shape, type, device);
        rows(made_dx, "grad_in", shape, type, device, a.grad_in_stride);
        dx = &made_dx;
      }
      if (w && (need || dw)) {
        if (!dw) {
          made_dw = empty(w->sizes(), w->scalar_type(), device);
          dw = &made_dw;
        }
        check(ringsim_rms_norm_backward_workspace(a.outer * a.inner, a.cols, a.dtype, &a.workspace_bytes),
              "ringsim_rms_norm_backward_workspace");
        if (a.workspace_bytes) {
          workspace = empty({(int64_t)a.workspace_bytes}, at::kByte, device);
          a.workspace = data(workspace);
        }
        a.grad_weight = data(*dw);
      }
      a.grad_out = data(dy);
      a.h = data(h);
      a.weight = w ? data(*w) : nullptr;
      a.grad_residual = res ? data(*res) : nullptr;
      a.grad_in = data(*dx);
      check(ringsim_rms_norm_backward(&a, current_stream(device)), "ringsim_rms_norm_backward");
    }
    for (int i = 5; i < 7; ++i) written(args[i]);
    return pack({result(args[5], made_dx), result(args[6], made_dw)});
  });
}

// A list of gradients as the C ABI takes it. Its tensors are held by a tuple of
// its own, since other threads may change the caller's list during the call.
struct GradList {
  PyObject* seq = nullptr;
  std::vector<void*> ptrs;
  std::vector<int64_t> counts;
  std::vector<int> types;

  GradList(PyObject* o, const char* name, int device) {
    seq = PySequence_Tuple(o);
    if (!seq) throw PythonError{};
    try {
      const Py_ssize_t n = PyTuple_GET_SIZE(seq);
      ptrs.reserve(n);
      counts.reserve(n);
      types.reserve(n);
      for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor& t = required(PyTuple_GET_ITEM(seq, i), name);
        const int code = type_code(t.scalar_type());
        if (code < 0) throw WrongType(std::string("unsupported dtype ") + c10::toString(t.scalar_type()) + " in " + name);
        check_device(t, device, name);
        if (!t.is_contiguous()) throw WrongValue(std::string(name) + " must be contiguous");
        ptrs.push_back(data(t));
        counts.push_back(t.numel());
        types.push_back(code);
      }
      if (n > INT32_MAX) throw WrongValue("too many tensors");
    } catch (...) {
      Py_DECREF(seq);
      throw;
    }
  }
  ~GradList() { Py_XDECREF(seq); }
  GradList(const GradList&) = delete;
  GradList& operator=(const GradList&) = delete;
  int size() const { return (int)ptrs.size(); }
  void all_written() const {
    for (int i = 0; i < size(); ++i) written(PyTuple_GET_ITEM(seq, i));
  }
};

// The outputs' addresses, which have to match the gradients.
const GradList* match(const GradList* outs, const GradList& grads) {
  if (outs && (outs->counts != grads.counts || outs->types != grads.types))
    throw WrongValue("outs must match grads in number, sizes and dtypes");
  return outs;
}

// The norm an argument holds; null for None.
const at::Tensor* norm_arg(PyObject* o, int device) {
  const at::Tensor* t = tensor(o, "norm");
  if (!t) return nullptr;
  if (t->scalar_type() != at::kFloat || t->numel() != 1) throw WrongValue("norm must be one float32");
  check_device(*t, device, "norm");
  return t;
}

// What a call that forms a norm writes: the norm, and a workspace if its list
// needs one.
struct NormMemory {
  at::Tensor made, workspace;
  float* norm;
  size_t bytes = 0;

  NormMemory(const GradList& g, const at::Tensor* given, int device) {
    if (!given) made = empty({}, at::kFloat, device);
    norm = static_cast<float*>(data(given ? *given : made));
    check(ringsim_grad_norm_workspace(g.size(), g.counts.data(), g.types.data(), &bytes), "ringsim_grad_norm_workspace");
    if (bytes) workspace = empty({(int64_t)bytes}, at::kByte, device);
  }
  void* space() const { return workspace.defined() ? data(workspace) : nullptr; }
};

// grad_norm(grads, scale, norm)
PyObject* grad_norm(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded([&] {
    want_args(nargs, 3);
    const int device = current_device();
    const float scale = (float)number(args[1]);
    const GradList g(args[0], "grads", device);
    const at::Tensor* norm = norm_arg(args[2], device);
    std::optional<NormMemory> m;
    {
      const Unlocked unlocked;
      m.emplace(g, norm, device);
      check(ringsim_grad_norm(g.size(), g.ptrs.data(), g.counts.data(), g.types.data(), scale, m->norm, m->space(),
                              m->bytes, current_stream(device)),
            "ringsim_grad_norm");
    }
    written(args[2]);
    return result(args[2], m->made);
  });
}

// scale_grads(grads, norm, max_norm, outs, scale, eps)
PyObject* scale_grads(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded([&] {
    want_args(nargs, 6);
    const int device = current_device();
    const float max_norm = (float)number(args[2]), scale = (float)number(args[4]), eps = (float)number(args[5]);
    const GradList g(args[0], "grads", device);
    required(args[1], "norm");
    const at::Tensor* norm = norm_arg(args[1], device);
    std::optional<GradList> outs;
    if (args[3] != Py_None) outs.emplace(args[3], "outs", device);
    const GradList* o = match(outs ? &*outs : nullptr, g);
    {
      const Unlocked unlocked;
      check(ringsim_scale_grads(g.size(), g.ptrs.data(), o ? o->ptrs.data() : nullptr, g.counts.data(), g.types.data(),
                                scale, static_cast<const float*>(data(*norm)), max_norm, eps, current_stream(device)),
            "ringsim_scale_grads");
    }
    (o ? o : &g)->all_written();
    return none();
  });
}

// clip_grads(grads, max_norm, outs, scale, eps, norm)
PyObject* clip_grads(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded([&] {
    want_args(nargs, 6);
    const int device = current_device();
    const float max_norm = (float)number(args[1]), scale = (float)number(args[3]), eps = (float)number(args[4]);
    const GradList g(args[0], "grads", device);
    std::optional<GradList> outs;
    if (args[2] != Py_None) outs.emplace(args[2], "outs", device);
    const GradList* o = match(outs ? &*outs : nullptr, g);
    const at::Tensor* norm = norm_arg(args[5], device);
    std::optional<NormMemory> m;
    {
      const Unlocked unlocked;
      m.emplace(g, norm, device);
      check(ringsim_clip_grads(g.size(), g.ptrs.data(), o ? o->ptrs.data() : nullptr, g.counts.data(), g.types.data(),
                               scale, max_norm, eps, m->norm, m->space(), m->bytes, current_stream(device)),
            "ringsim_clip_grads");
    }
    (o ? o : &g)->all_written();
    written(args[5]);
    return result(args[5], m->made);
  });
}

// set_errors(RingsimError, torch.OutOfMemoryError)
PyObject* set_errors(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded([&] {
    want_args(nargs, 2);
    Py_INCREF(args[0]);
    Py_XSETREF(g_ringsim_error, args[0]);
    Py_INCREF(args[1]);
    Py_XSETREF(g_memory_error, args[1]);
    return none();
  });
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {
    {"rms_norm", fast(rms_norm), METH_FASTCALL, nullptr},
    {"rms_norm_backward", fast(rms_norm_backward), METH_FASTCALL, nullptr},
    {"grad_norm", fast(grad_norm), METH_FASTCALL, nullptr},
    {"scale_grads", fast(scale_grads), METH_FASTCALL, nullptr},
    {"clip_grads", fast(clip_grads), METH_FASTCALL, nullptr},
    {"set_errors", fast(set_errors), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ops_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops_binding() { return PyModule_Create(&g_module); }
