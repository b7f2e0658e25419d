// binding.h -- what the torch bindings share: checks of arguments, outputs, workspaces and the way out of
// C++ exceptions.
#pragma once

#include <Python.h>

#include <cstring>
#include <stdexcept>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime.h>
#include <torch/csrc/autograd/python_variable.h>

#include "logmel.h"

namespace lm_binding {

using at::Tensor;

struct GradError {};

// Another operation's refusal, as the ValueError that it becomes.
[[noreturn]] inline void refuse(const std::string &what) { throw std::invalid_argument(what); }

inline const Tensor *tensor_or_null(PyObject *o, const char *name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
  return &THPVariable_Unpack(o);
}

inline const Tensor &tensor(PyObject *o, const char *name) {
  const Tensor *t = tensor_or_null(o, name);
  if (!t || !t->is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  return *t;
}

// An optional or required tensor on device `dev`.
inline const Tensor *on(PyObject *o, const char *name, int dev) {
  const Tensor *t = tensor_or_null(o, name);
  if (!t) return nullptr;
  if (!t->is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t->get_device() != dev) refuse(std::string(name) + " must be on the same device as the other inputs");
  return t;
}

// Neither direction of differentiation passes through these operations.  (Tangents exist under
// no_grad, too.)
inline void no_grad(std::initializer_list<const Tensor *> ts) {
  const bool backward = c10::GradMode::is_enabled();
  for (const Tensor *t : ts)
    if (t && ((backward && t->requires_grad()) || t->_fw_grad(0).defined())) throw GradError{};
}

// What a user's tensor holds has changed: a graph that saved it finds out.
inline void written(const Tensor *t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

inline int half_code(at::ScalarType t) { return t == at::kHalf ? LM_F16 : t == at::kBFloat16 ? LM_BF16 : -1; }
inline int float_code(at::ScalarType t) { return t == at::kFloat ? LM_F32 : half_code(t); }
inline at::ScalarType type_of(int code) { return code == LM_F32 ? at::kFloat : code == LM_F16 ? at::kHalf : at::kBFloat16; }

inline Tensor make(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, dev)));
}

enum Op { kLinear, kAttend, kBeam, kReorder };

// Scratch of an operation on a stream, for callers that hold the interpreter's lock (binding.cpp).
Tensor workspace(Op op, int dev, cudaStream_t stream, size_t bytes);

inline PyObject *status(int rc) { return PyLong_FromLong(rc); }

// The stride of a tensor's rows when its leading dimensions are one.
inline int64_t row_stride(const Tensor &t, const char *name) {
  const auto sz = t.sizes(), st = t.strides();
  const int64_t d = t.dim();
  if (d == 1 || t.numel() == 0) return sz[d - 1];
  int64_t row = st[d - 2], n = sz[d - 2];
  for (int64_t i = d - 3; i >= 0; --i) {
    if (sz[i] == 1) continue;
    if (n == 1) {
      row = st[i];
    } else if (st[i] != row * n) {
      refuse(std::string(name) + "'s leading dimensions must be evenly spaced rows");
    }
    n *= sz[i];
  }
  return row;
}

// No C++ exception leaves the module.
template <PyObject *(*F)(PyObject *const *), int ARGS>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != ARGS) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", ARGS, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const std::invalid_argument &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const GradError &) {
    PyErr_SetString(PyExc_RuntimeError,
                    "log_mel_spectrogram_gb300 ops are inference-only: tensors must not require grad (use "
                    "torch.no_grad() or detach()) or carry a tangent");
  } catch (const std::exception &e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <PyObject *(*F)(PyObject *const *), int ARGS>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, ARGS>));
}

extern PyMethodDef kLayerMethods[];  // layers.cpp

// A weight in 4 bits as the Python module passes it: (packed, scale, n, k, group, dtype) (layers.cpp).
struct Weight4 {
  lm_weight4 c;
  Tensor packed, scale;
  int dev, code;
};
Weight4 weight4_of(PyObject *o);

}  // namespace lm_binding
