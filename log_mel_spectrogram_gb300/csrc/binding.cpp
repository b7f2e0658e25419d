// binding.cpp -- the torch side of linear, the key/value cache and the beam
// step: checks of arguments, outputs and workspaces, and the C call, without
// the interpreter in between (a decoding step makes dozens of these calls, and
// each takes a few microseconds on the GPU).
//
// The C ABI (include/logmel.h) does the work.  A status other than LM_OK is
// returned as an int, for the Python module to raise.
#include <Python.h>

#include <cstring>
#include <map>
#include <mutex>
#include <stdexcept>
#include <string>
#include <tuple>
#include <vector>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime.h>
#include <torch/csrc/autograd/python_variable.h>

#include "logmel.h"

namespace {

using at::Tensor;

struct GradError {};

// Another operation's refusal, as the ValueError that it becomes.
[[noreturn]] void refuse(const std::string &what) { throw std::invalid_argument(what); }

const Tensor *tensor_or_null(PyObject *o, const char *name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
  return &THPVariable_Unpack(o);
}

const Tensor &tensor(PyObject *o, const char *name) {
  const Tensor *t = tensor_or_null(o, name);
  if (!t || !t->is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  return *t;
}

// An optional or required tensor on device `dev`.
const Tensor *on(PyObject *o, const char *name, int dev) {
  const Tensor *t = tensor_or_null(o, name);
  if (!t) return nullptr;
  if (!t->is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t->get_device() != dev) refuse(std::string(name) + " must be on the same device as the other inputs");
  return t;
}

// Neither direction of differentiation passes through these operations.  (Tangents exist under
// no_grad, too.)
void no_grad(std::initializer_list<const Tensor *> ts) {
  const bool backward = c10::GradMode::is_enabled();
  for (const Tensor *t : ts)
    if (t && ((backward && t->requires_grad()) || t->_fw_grad(0).defined())) throw GradError{};
}

// What a user's tensor holds has changed: a graph that saved it finds out.
void written(const Tensor *t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

int half_code(at::ScalarType t) { return t == at::kHalf ? LM_F16 : t == at::kBFloat16 ? LM_BF16 : -1; }
int float_code(at::ScalarType t) { return t == at::kFloat ? LM_F32 : half_code(t); }
at::ScalarType type_of(int code) { return code == LM_F32 ? at::kFloat : code == LM_F16 ? at::kHalf : at::kBFloat16; }

Tensor make(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, dev)));
}

enum Op { kLinear, kAttend, kBeam, kReorder };

constexpr int64_t kLeastBytes = 1 << 16;  // of a workspace that is kept
constexpr size_t kMostKept = 128;         // workspaces; past that the one whose last use is longest ago goes

// A zeroed workspace.  An operation's kernels leave its counters at zero, so
// one per operation, device and stream serves every call on it; a call that a
// graph captures gets one of its own, cleared on each replay.  Streams go by
// their ids: a handle comes back after its stream is destroyed, whose work may
// still be under way.
//
// linear has no counters, and needs much where it copies an operand off 16-byte
// boundaries (128 MB for a weight of 50001 x 1023): what is more than the least is that call's
// alone, and nothing is cleared.
Tensor workspace(Op op, int dev, cudaStream_t stream, size_t bytes) {
  struct Kept {
    Tensor t;
    uint64_t used = 0;
  };
  using Key = std::tuple<int, int, unsigned long long>;
  static std::mutex mu;
  static auto *const all = new std::map<Key, Kept>;  // outlives the interpreter's end
  static uint64_t uses = 0;
  const auto options = at::TensorOptions().dtype(at::kByte).device(at::Device(at::kCUDA, dev));
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess) (void)cudaGetLastError();
  const bool captured = cs != cudaStreamCaptureStatusNone;
  if (op == kLinear && (captured || bytes > static_cast<size_t>(kLeastBytes)))
    return at::empty({static_cast<int64_t>(bytes)}, options);
  if (captured) return at::zeros({static_cast<int64_t>(bytes)}, options);
  unsigned long long id = 0;
  if (const cudaError_t e = cudaStreamGetId(stream, &id); e != cudaSuccess) {
    (void)cudaGetLastError();
    throw std::runtime_error(std::string("cudaStreamGetId: ") + cudaGetErrorString(e));
  }
  std::lock_guard<std::mutex> lk(mu);
  Kept &k = (*all)[std::make_tuple(static_cast<int>(op), dev, id)];
  k.used = ++uses;
  if (!k.t.defined() || static_cast<size_t>(k.t.numel()) < bytes) {
    int64_t size = kLeastBytes;
    while (static_cast<size_t>(size) < bytes) size *= 2;
    k.t = at::zeros({size}, options);
  }
  const Tensor t = k.t;
  if (all->size() > kMostKept) {
    auto oldest = all->begin();
    for (auto i = all->begin(); i != all->end(); ++i)
      if (i->second.used < oldest->second.used) oldest = i;
    all->erase(oldest);
  }
  return t;
}

PyObject *status(int rc) { return PyLong_FromLong(rc); }

// The stride of a tensor's rows when its leading dimensions are one.
int64_t row_stride(const Tensor &t, const char *name) {
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

// linear(x, weight, bias, activation, residual, scale, out, out_dtype or -1)
PyObject *linear(PyObject *const *a) {
  const Tensor &x = tensor(a[0], "x");
  if (x.dim() < 1) refuse("x must be a CUDA tensor [..., K]");
  const int dev = x.get_device();
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  const int code = half_code(x.scalar_type());
  if (code < 0) refuse("x must be float16 or bfloat16");
  const Tensor *w = on(a[1], "weight", dev), *bias = on(a[2], "bias", dev), *res = on(a[4], "residual", dev),
               *given = on(a[6], "out", dev);
  if (!w) refuse("weight must be a CUDA tensor");
  no_grad({&x, w, bias, res, given});
  const int64_t dims = x.dim(), k = x.size(-1);
  if (w->scalar_type() != x.scalar_type() || w->dim() != 2 || w->size(1) != k)
    refuse("weight must be [N, K] of x's dtype and last dimension");
  const int64_t n = w->size(0);
  if (k > 1 && (x.stride(-1) != 1 || w->stride(1) != 1))
    refuse("the last dimension of x and weight must be contiguous");
  lm_linear_args p = {};
  p.k = k;
  p.n = n;
  p.weight_row_stride = w->stride(0);
  p.dtype = code;
  p.activation = static_cast<int32_t>(PyLong_AsLong(a[3]));
  p.scale = static_cast<float>(PyFloat_AsDouble(a[5]));
  if (PyErr_Occurred()) return nullptr;
  const auto sz = x.sizes(), st = x.strides();
  if (dims == 1) {
    p.groups = p.rows = 1;
  } else {
    p.groups = 1;
    p.rows = sz[dims - 2];
    p.x_row_stride = st[dims - 2];
    // The dimensions in front of the rows: one stride.
    bool first = true;
    int64_t span = 0;
    for (int64_t i = dims - 3; i >= 0; --i) {
      if (sz[i] != 1 && x.numel() != 0) {
        if (first) {
          p.x_group_stride = st[i];
          first = false;
        } else if (st[i] != span) {
          refuse("x's leading dimensions must be evenly spaced");
        }
        span = st[i] * sz[i];
      }
      p.groups *= sz[i];
    }
  }
  if (bias) {
    p.bias_dtype = float_code(bias->scalar_type());
    if ((p.bias_dtype != LM_F32 && p.bias_dtype != code) || bias->dim() != 1 || bias->size(0) != n ||
        (n > 1 && bias->stride(0) != 1))
      refuse("bias must be [N], contiguous, of dtype float32 or x's");
    p.bias = bias->data_ptr();
  }
  c10::SmallVector<int64_t, 6> shape(sz.begin(), sz.end());
  shape[dims - 1] = n;
  int od = static_cast<int>(PyLong_AsLong(a[7]));
  Tensor out;
  if (given) {
    if (given->sizes() != at::IntArrayRef(shape)) refuse("out must have x's leading dimensions and N");
    const int gd = float_code(given->scalar_type());
    if (od >= 0 ? gd != od : gd != code && gd != LM_F32) refuse("out must be of x's dtype or float32");
    if (n > 1 && given->stride(-1) != 1) refuse("the last dimension of out must be contiguous");
    out = *given;
    od = gd;
    p.out_row_stride = row_stride(out, "out");
  } else {
    if (od < 0) od = code;
    if (od != code && od != LM_F32) refuse("out_dtype must be x's dtype or float32");
    out = make(shape, type_of(od), dev);
    p.out_row_stride = n;
  }
  p.out_dtype = od;
  if (res) {
    if (res->scalar_type() != x.scalar_type() || res->sizes() != at::IntArrayRef(shape))
      refuse("residual must have x's dtype and leading dimensions, and N");
    if (n > 1 && res->stride(-1) != 1) refuse("the last dimension of residual must be contiguous");
    p.residual = res->data_ptr();
    p.residual_row_stride = row_stride(*res, "residual");
  }
  p.x = x.data_ptr();
  p.weight = w->data_ptr();
  p.out = out.data_ptr();
  size_t need = 0;
  int rc = lm_linear_workspace_size(&p, &need);
  if (rc == LM_OK) {
    const cudaStream_t s = c10::cuda::getCurrentCUDAStream(dev).stream();
    const Tensor ws = workspace(kLinear, dev, s, need);
    rc = lm_linear(&p, ws.data_ptr(), static_cast<size_t>(ws.numel()), reinterpret_cast<lm_stream_t>(s));
  }
  if (rc != LM_OK) return status(rc);
  written(given);
  return THPVariable_Wrap(out);
}

// ---- the cache: args, device, dtype come first ----

struct Cache {
  lm_kv_cache c;
  int dev, code;
};

Cache cache_of(PyObject *const *a) {
  Cache k;
  if (!PyBytes_Check(a[0]) || PyBytes_GET_SIZE(a[0]) != static_cast<Py_ssize_t>(sizeof(lm_kv_cache)))
    refuse("not a cache");
  std::memcpy(&k.c, PyBytes_AS_STRING(a[0]), sizeof(k.c));
  k.dev = static_cast<int>(PyLong_AsLong(a[1]));
  k.code = static_cast<int>(PyLong_AsLong(a[2]));
  return k;
}

int layer_of(const Cache &k, PyObject *o) {
  const long layer = PyLong_AsLong(o);
  if (layer < 0 || layer >= k.c.layers) {
    PyErr_Clear();
    refuse("layer must be in 0 .. " + std::to_string(k.c.layers - 1));
  }
  return static_cast<int>(layer);
}

// [rows, tokens, heads, head_dim] and its strides.
const Tensor &tokens_of(const Cache &k, PyObject *o, const char *name, int64_t heads, int64_t *strides) {
  const Tensor &t = tensor(o, name);
  if (t.get_device() != k.dev) refuse(std::string(name) + " must be on the cache's device");
  if (half_code(t.scalar_type()) != k.code) refuse(std::string(name) + " must be of the cache's dtype");
  if (t.dim() != 4 || t.size(0) != k.c.rows || t.size(3) != k.c.head_dim || (heads >= 0 && t.size(2) != heads))
    refuse(std::string(name) + " must be [" + std::to_string(k.c.rows) + ", tokens, " +
           (heads >= 0 ? std::to_string(heads) : std::string("heads")) + ", " + std::to_string(k.c.head_dim) + "]");
  if (t.stride(3) != 1) refuse("the last dimension of " + std::string(name) + " must be contiguous");
  for (int i = 0; i < 3; ++i) strides[i] = t.stride(i);
  return t;
}

const int32_t *counts_of(const Cache &k, PyObject *o) {
  const Tensor *t = tensor_or_null(o, "counts");
  if (!t) return nullptr;
  if (!t->is_cuda() || t->scalar_type() != at::kInt || t->dim() != 1 || t->size(0) != k.c.rows ||
      !t->is_contiguous() || t->get_device() != k.dev)
    refuse("counts must be a contiguous int32 CUDA tensor [" + std::to_string(k.c.rows) + "] on the cache's device");
  return t->data_ptr<int32_t>();
}

// kv_append(args, device, dtype, layer, k, v, counts, values)
PyObject *kv_append(PyObject *const *a) {
  const Cache c = cache_of(a);
  const int layer = layer_of(c, a[3]);
  int64_t ks[3], vs[3];
  const Tensor &k = tokens_of(c, a[4], "k", c.c.heads, ks), &v = tokens_of(c, a[5], "v", c.c.heads, vs);
  no_grad({&k, &v});
  if (k.size(1) != v.size(1)) refuse("k and v must have as many tokens");
  const int32_t *const counts = counts_of(c, a[6]);
  const c10::cuda::OptionalCUDAGuard guard(k.device());
  const int64_t t = k.size(1);
  Tensor kv, vv;
  if (a[7] == Py_True) {
    const int64_t b = c.c.block, span = t ? ((t - 1 + b - 1) / b + 1) * b : 0;
    kv = make({c.c.rows, span, c.c.heads, c.c.head_dim}, type_of(c.code), c.dev);
    vv = make({c.c.rows, span, c.c.heads, c.c.head_dim}, type_of(c.code), c.dev);
  }
  const int rc = t > INT32_MAX ? static_cast<int>(LM_ERR_UNSUPPORTED)
                               : lm_kv_append(&c.c, layer, k.data_ptr(), v.data_ptr(), ks, vs, static_cast<int32_t>(t),
                                              counts, c.code, kv.defined() ? kv.data_ptr() : nullptr,
                                              vv.defined() ? vv.data_ptr() : nullptr,
                                              reinterpret_cast<lm_stream_t>(c10::cuda::getCurrentCUDAStream(c.dev).stream()));
  if (rc != LM_OK) return status(rc);
  if (!kv.defined()) Py_RETURN_NONE;
  return Py_BuildValue("(NN)", THPVariable_Wrap(kv), THPVariable_Wrap(vv));
}

// kv_attend(args, device, dtype, layer, q, counts, causal, scale or None, out)
PyObject *kv_attend(PyObject *const *a) {
  const Cache c = cache_of(a);
  const int layer = layer_of(c, a[3]);
  int64_t qs[3];
  const Tensor &q = tokens_of(c, a[4], "q", -1, qs);
  const int64_t t = q.size(1), hq = q.size(2);
  if (hq == 0 || hq % c.c.heads) refuse("q must have a multiple of " + std::to_string(c.c.heads) + " heads");
  if (t > INT32_MAX || hq > INT32_MAX) return status(LM_ERR_UNSUPPORTED);
  const int32_t *const counts = counts_of(c, a[5]);
  const int causal = PyObject_IsTrue(a[6]);
  double scale = 1.0 / std::sqrt(static_cast<double>(c.c.head_dim));
  if (a[7] != Py_None) scale = PyFloat_AsDouble(a[7]);
  if (PyErr_Occurred()) return nullptr;
  const c10::cuda::OptionalCUDAGuard guard(q.device());
  const Tensor *given = on(a[8], "out", c.dev);
  no_grad({&q, given});
  if (given && (given->scalar_type() != q.scalar_type() || given->sizes() != q.sizes() || !given->is_contiguous()))
    refuse("out must be contiguous, of q's dtype and shape");
  Tensor out = given ? *given : make(q.sizes(), q.scalar_type(), c.dev);
  size_t need = 0;
  int rc = lm_kv_attend_workspace_size(&c.c, static_cast<int32_t>(t), static_cast<int32_t>(hq), &need);
  if (rc == LM_OK) {
    const cudaStream_t s = c10::cuda::getCurrentCUDAStream(c.dev).stream();
    const Tensor ws = workspace(kAttend, c.dev, s, need);
    rc = lm_kv_attend(&c.c, layer, q.data_ptr(), qs, static_cast<int32_t>(t), static_cast<int32_t>(hq), counts,
                      causal ? static_cast<int32_t>(t) : 0, causal, static_cast<float>(scale), c.code, out.data_ptr(),
                      ws.data_ptr(), static_cast<size_t>(ws.numel()), reinterpret_cast<lm_stream_t>(s));
  }
  if (rc != LM_OK) return status(rc);
  written(given);
  return THPVariable_Wrap(out);
}

// kv_read(args, device, dtype, layer or -1, start, count)
PyObject *kv_read(PyObject *const *a) {
  const Cache c = cache_of(a);
  const long all = PyLong_AsLong(a[3]);
  const int layer = all == -1 ? -1 : layer_of(c, a[3]);
  const long long start = PyLong_AsLongLong(a[4]), count = PyLong_AsLongLong(a[5]);
  if (PyErr_Occurred()) return nullptr;
  if (start < 0 || count < 0) refuse("start and count must be >= 0");
  if (start > INT32_MAX || count > INT32_MAX) return status(LM_ERR_UNSUPPORTED);
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, c.dev));
  c10::SmallVector<int64_t, 5> shape;
  if (layer < 0) shape.push_back(c.c.layers);
  for (int64_t d : {static_cast<int64_t>(c.c.rows), static_cast<int64_t>(count), static_cast<int64_t>(c.c.heads),
                    static_cast<int64_t>(c.c.head_dim)})
    shape.push_back(d);
  Tensor k = make(shape, type_of(c.code), c.dev), v = make(shape, type_of(c.code), c.dev);
  const int rc = lm_kv_read(&c.c, layer, static_cast<int32_t>(start), static_cast<int32_t>(count), c.code,
                            k.data_ptr(), v.data_ptr(),
                            reinterpret_cast<lm_stream_t>(c10::cuda::getCurrentCUDAStream(c.dev).stream()));
  if (rc != LM_OK) return status(rc);
  return Py_BuildValue("(NN)", THPVariable_Wrap(k), THPVariable_Wrap(v));
}

// kv_reorder(args, device, dtype, parents)
PyObject *kv_reorder(PyObject *const *a) {
  const Cache c = cache_of(a);
  const Tensor &p = tensor(a[3], "parents");
  if (p.scalar_type() != at::kInt || p.dim() != 2 || p.numel() != c.c.rows || !p.is_contiguous() ||
      p.get_device() != c.dev)
    refuse("parents must be a contiguous [clips, beams] int32 CUDA tensor of " + std::to_string(c.c.rows) +
           " rows on the cache's device");
  const c10::cuda::OptionalCUDAGuard guard(p.device());
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(c.dev).stream();
  const Tensor ws = workspace(kReorder, c.dev, s, 16 + 4 * static_cast<size_t>(p.size(0)));
  const int rc = p.size(1) > INT32_MAX ? static_cast<int>(LM_ERR_UNSUPPORTED)
                 : c.c.rows == 0       ? static_cast<int>(LM_OK)
                                       : lm_kv_reorder(&c.c, p.data_ptr<int32_t>(), static_cast<int32_t>(p.size(1)),
                                                       ws.data_ptr(), static_cast<size_t>(ws.numel()),
                                                       reinterpret_cast<lm_stream_t>(s));
  if (rc != LM_OK) return status(rc);
  Py_RETURN_NONE;
}

// beam_step(logits, scores, finished, history, length, eos or None)
PyObject *beam_step(PyObject *const *a) {
  const Tensor &x = tensor(a[0], "logits");
  if (x.dim() != 3) refuse("logits must be a CUDA tensor [clips, beams, vocab]");
  const int dev = x.get_device();
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  lm_beam_args p = {};
  p.dtype = float_code(x.scalar_type());
  if (p.dtype < 0) refuse("logits must be float32, float16 or bfloat16");
  const Tensor &scores = tensor(a[1], "scores");
  no_grad({&x, &scores});
  const int64_t clips = x.size(0), beams = x.size(1), vocab = x.size(2);
  if ((vocab > 1 && x.stride(2) != 1) || (clips > 1 && beams > 1 && x.stride(0) != beams * x.stride(1)))
    refuse("logits must be evenly spaced rows of contiguous values");
  auto fits = [&](const Tensor &t, at::ScalarType type) {
    return t.is_cuda() && t.scalar_type() == type && t.dim() >= 2 && t.size(0) == clips && t.size(1) == beams &&
           t.is_contiguous() && t.get_device() == dev;
  };
  if (!fits(scores, at::kFloat) || scores.dim() != 2)
    refuse("scores must be a contiguous [clips, beams] float32 CUDA tensor on the logits' device");
  const Tensor *finished = tensor_or_null(a[2], "finished"), *history = tensor_or_null(a[3], "history");
  p.eos = -1;
  if (a[5] != Py_None) {
    p.eos = PyLong_AsLongLong(a[5]);
    if (PyErr_Occurred()) return nullptr;
    if (p.eos < 0 || p.eos >= vocab) refuse("eos must be a token of the vocabulary");
  }
  if (finished) {
    if (!fits(*finished, at::kBool) || finished->dim() != 2)
      refuse("finished must be a contiguous [clips, beams] bool CUDA tensor on the logits' device");
    if (p.eos < 0) refuse("finished beams need eos");
    p.finished = static_cast<const uint8_t *>(finished->data_ptr());
  }
  Tensor told;
  if (history) {
    if (!fits(*history, at::kInt) || history->dim() != 3)
      refuse("history must be a contiguous [clips, beams, width] int32 CUDA tensor on the logits' device");
    p.width = history->size(2);
    p.length = PyLong_AsLongLong(a[4]);
    if (PyErr_Occurred()) return nullptr;
    if (p.length < 0 || p.length >= p.width) refuse("length must be a place of the history");
    told = make(history->sizes(), at::kInt, dev);
    p.history = history->data_ptr<int32_t>();
    p.out_history = told.data_ptr<int32_t>();
  }
  if (beams > INT32_MAX) return status(LM_ERR_UNSUPPORTED);
  const Tensor next = make({clips, beams}, at::kFloat, dev), tokens = make({clips, beams}, at::kInt, dev),
               parents = make({clips, beams}, at::kInt, dev), ended = make({clips, beams}, at::kBool, dev);
  p.logits = x.data_ptr();
  p.scores = scores.data_ptr<float>();
  p.out_scores = next.data_ptr<float>();
  p.out_tokens = tokens.data_ptr<int32_t>();
  p.out_parents = parents.data_ptr<int32_t>();
  p.out_finished = static_cast<uint8_t *>(ended.data_ptr());
  p.clips = clips;
  p.vocab = vocab;
  p.row_stride = beams > 1 ? x.stride(1) : x.stride(0);
  p.beams = static_cast<int32_t>(beams);
  size_t need = 0;
  int rc = lm_beam_step_workspace_size(&p, &need);
  if (rc == LM_OK) {
    const cudaStream_t s = c10::cuda::getCurrentCUDAStream(dev).stream();
    const Tensor ws = workspace(kBeam, dev, s, need);
    rc = lm_beam_step(&p, ws.data_ptr(), static_cast<size_t>(ws.numel()), reinterpret_cast<lm_stream_t>(s));
  }
  if (rc != LM_OK) return status(rc);
  PyObject *last = Py_None;
  if (history) {
    last = THPVariable_Wrap(told);
  } else {
    Py_INCREF(last);
  }
  return Py_BuildValue("(NNNNN)", THPVariable_Wrap(next), THPVariable_Wrap(tokens), THPVariable_Wrap(parents),
                       THPVariable_Wrap(ended), last);
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

PyMethodDef kMethods[] = {
    {"linear", fast<linear, 8>(), METH_FASTCALL, nullptr},
    {"kv_append", fast<kv_append, 8>(), METH_FASTCALL, nullptr},
    {"kv_attend", fast<kv_attend, 9>(), METH_FASTCALL, nullptr},
    {"kv_read", fast<kv_read, 6>(), METH_FASTCALL, nullptr},
    {"kv_reorder", fast<kv_reorder, 4>(), METH_FASTCALL, nullptr},
    {"beam_step", fast<beam_step, 6>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_decode", "linear, the key/value cache and the beam step", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode(void) { return PyModule_Create(&kModule); }
