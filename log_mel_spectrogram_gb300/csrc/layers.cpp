// layers.cpp -- the torch side of layer_norm and gated_linear, with their gradients, and of weights in
// 4 bits: checks of arguments, outputs and workspaces, the autograd nodes, and the C call.
#include "binding.h"

#include <cmath>
#include <optional>
#include <unordered_set>
#include <vector>

#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/graph_task.h>
#include <torch/csrc/autograd/variable.h>

namespace lm_binding {

namespace {

using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

const char *status_name(int rc) {
  static const char *const names[] = {"LM_OK", "LM_ERR_INVALID_ARG", "LM_ERR_UNSUPPORTED", "LM_ERR_MISALIGNED",
                                      "LM_ERR_CUDA", "LM_ERR_OUT_OF_MEMORY", "LM_ERR_DEVICE_FAULT", "LM_ERR_WORKSPACE"};
  return rc >= 0 && rc < 8 ? names[rc] : "unknown status";
}

// A status of a call inside an autograd node, which becomes the module's LogmelError where it can (the
// forward pass) and a RuntimeError where it cannot (the backward pass runs on a thread of torch's).
struct StatusError : std::runtime_error {
  int rc;
  StatusError(const char *what, int rc_) : std::runtime_error(std::string(what) + ": " + status_name(rc_)), rc(rc_) {}
};

void ok(int rc, const char *what) {
  if (rc != LM_OK) throw StatusError(what, rc);
}

void no_tangents(std::initializer_list<const Tensor *> ts) {
  for (const Tensor *t : ts)
    if (t && t->defined() && t->_fw_grad(0).defined())
      throw std::runtime_error("log_mel_spectrogram_gb300: tensors must not carry a tangent (there is no forward-mode "
                               "derivative)");
}

bool wants_grad(std::initializer_list<const Tensor *> ts) {
  if (!c10::GradMode::is_enabled()) return false;
  for (const Tensor *t : ts)
    if (t && t->defined() && t->requires_grad()) return true;
  return false;
}

bool capturing(cudaStream_t s) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cs) != cudaSuccess) (void)cudaGetLastError();
  return cs != cudaStreamCaptureStatusNone;
}

// A node of a graph runs on the stream that it was made on, a leaf's on that of the first graph over it, and
// that one lives as long as such a graph does.  Where that is the default stream, a backward pass that is being captured
// would make that stream wait for the captured one, which ends the capture and with it the process.  It is refused
// while the forward pass is captured, for leaves among the inputs, and for what lies behind them when the gradients
// are taken.
bool on_default_stream(torch::autograd::Node &node) {
  const auto stream = node.stream();
  return stream && c10::cuda::CUDAStream(*stream).stream() == nullptr;
}

[[noreturn]] void refuse_capture() {
  throw std::runtime_error("log_mel_spectrogram_gb300: a graph of the default stream over the same leaf is alive; a "
                           "backward pass cannot be captured beside it (delete its outputs first, or run it on a "
                           "side stream)");
}

void no_eager_graph(std::initializer_list<const Tensor *> ts, int dev) {
  if (!capturing(c10::cuda::getCurrentCUDAStream(dev).stream())) return;
  for (const Tensor *t : ts) {
    if (!t || !t->defined() || !t->requires_grad() || t->grad_fn()) continue;
    const auto node = torch::autograd::impl::try_get_grad_accumulator(*t);
    if (node && on_default_stream(*node)) refuse_capture();
  }
}

// ... of the nodes that the pass will come to after this one.
void no_eager_nodes(int dev) {
  if (!capturing(c10::cuda::getCurrentCUDAStream(dev).stream())) return;
  const auto *const info = torch::autograd::get_current_graph_task_exec_info();  // (empty: all of them)
  const auto here = torch::autograd::get_current_node();
  std::vector<torch::autograd::Node *> todo;
  std::unordered_set<torch::autograd::Node *> seen;
  if (here) todo.push_back(here.get());
  while (!todo.empty()) {
    const torch::autograd::Node *const node = todo.back();
    todo.pop_back();
    for (const torch::autograd::Edge &e : node->next_edges()) {
      torch::autograd::Node *const next = e.function.get();
      if (!next || !seen.insert(next).second) continue;
      if (info && !info->empty()) {
        const auto at = info->find(next);
        if (at == info->end() || !at->second.should_execute()) continue;
      }
      if (on_default_stream(*next)) refuse_capture();
      todo.push_back(next);
    }
  }
}

void no_second_derivative() {
  if (c10::GradMode::is_enabled())
    throw std::runtime_error("log_mel_spectrogram_gb300: there are no second derivatives (create_graph must be False)");
}

lm_stream_t stream_of(int dev) {
  return reinterpret_cast<lm_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
}

// Scratch of one backward pass.  It runs on a thread of torch's engine, without the interpreter's lock, so another
// thread's calls on the stream fall between its launches: what workspace() keeps for the stream may be theirs.
Tensor own_scratch(int dev, size_t bytes) { return make({static_cast<int64_t>(bytes)}, at::kByte, dev); }

Tensor defined_or_none(const Tensor *t) { return t ? *t : Tensor(); }

// Optional inputs of an autograd node; an absent one has no edge, so a node counts its edges over those there are.
using Optional = std::optional<Tensor>;
Optional optional(const Tensor *t) { return t ? Optional(*t) : Optional(); }
Tensor defined_or_none(const Optional &t) { return t ? *t : Tensor(); }

PyObject *wrapped(Tensor t) { return THPVariable_Wrap(std::move(t)); }

// Evenly spaced rows with contiguous elements: as it is, or copied.
Tensor as_rows(const Tensor &t) {
  const auto sz = t.sizes(), st = t.strides();
  const int64_t d = t.dim();
  bool even = sz[d - 1] <= 1 || st[d - 1] == 1;
  int64_t row = -1, n = 1;
  for (int64_t i = d - 2; i >= 0 && even; --i) {
    if (sz[i] == 1) continue;
    if (row < 0) {
      row = st[i];
    } else if (st[i] != row * n) {
      even = false;
    }
    n *= sz[i];
  }
  return even || t.numel() == 0 ? t : t.contiguous();
}

int64_t rows_of(const Tensor &t) {
  int64_t n = 1;
  for (int64_t i = 0; i + 1 < t.dim(); ++i) n *= t.size(i);
  return n;
}

// ---- layer norm ----

const void *ptr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

void norm_forward(const Tensor &x, const Tensor &w, const Tensor &b, double eps, const Tensor &out, const Tensor &stats) {
  const int dev = x.get_device();
  const int code = float_code(x.scalar_type());
  lm_norm_args p = {};
  p.x = x.data_ptr();
  p.weight = ptr(w);
  p.bias = ptr(b);
  p.out = out.data_ptr();
  p.stats = stats.defined() ? stats.data_ptr<float>() : nullptr;
  p.rows = rows_of(x);
  p.width = x.size(-1);
  p.x_row_stride = row_stride(x, "x");
  p.out_row_stride = row_stride(out, "out");
  p.dtype = code;
  p.weight_dtype = w.defined() ? float_code(w.scalar_type()) : LM_F32;
  p.bias_dtype = b.defined() ? float_code(b.scalar_type()) : LM_F32;
  p.eps = static_cast<float>(eps);
  ok(lm_layer_norm(&p, stream_of(dev)), "lm_layer_norm");
}

struct NormFn : public torch::autograd::Function<NormFn> {
  static Tensor forward(AutogradContext *ctx, const Tensor &x, const Optional &weight, const Optional &bias, double eps) {
    const Tensor w = defined_or_none(weight), b = defined_or_none(bias);
    const int dev = x.get_device();
    const Tensor out = make(x.sizes(), x.scalar_type(), dev);
    const Tensor stats = make({3, rows_of(x)}, at::kFloat, dev);
    norm_forward(x, w, b, eps, out, stats);
    ctx->save_for_backward({x, w, stats});
    ctx->saved_data["bias"] = static_cast<int64_t>(b.defined() ? float_code(b.scalar_type()) : -1);
    return out;
  }

  static variable_list backward(AutogradContext *ctx, variable_list grads) {
    no_second_derivative();
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &x = saved[0], &w = saved[1], &stats = saved[2];
    const int64_t bias = ctx->saved_data["bias"].toInt();
    const int dev = x.get_device();
    const c10::cuda::OptionalCUDAGuard guard(x.device());
    no_eager_nodes(dev);
    const int64_t width = x.size(-1);
    const Tensor g = as_rows(grads[0]);
    Tensor dx, dw, db;
    lm_norm_backward_args p = {};
    size_t edge = 0;
    if (ctx->needs_input_grad(edge++)) dx = make(x.sizes(), x.scalar_type(), dev);
    if (w.defined() && ctx->needs_input_grad(edge++)) dw = make({width}, w.scalar_type(), dev);
    if (bias >= 0 && ctx->needs_input_grad(edge++)) db = make({width}, type_of(static_cast<int>(bias)), dev);
    p.x = x.data_ptr();
    p.weight = ptr(w);
    p.stats = stats.data_ptr<float>();
    p.grad = g.data_ptr();
    p.dx = dx.defined() ? dx.data_ptr() : nullptr;
    p.dweight = dw.defined() ? dw.data_ptr() : nullptr;
    p.dbias = db.defined() ? db.data_ptr() : nullptr;
    p.rows = rows_of(x);
    p.width = width;
    p.x_row_stride = row_stride(x, "x");
    p.grad_row_stride = row_stride(g, "grad");
    p.dtype = float_code(x.scalar_type());
    p.weight_dtype = w.defined() ? float_code(w.scalar_type()) : LM_F32;
    p.bias_dtype = bias >= 0 ? static_cast<int32_t>(bias) : static_cast<int32_t>(LM_F32);
    size_t need = 0;
    ok(lm_layer_norm_backward_workspace_size(&p, &need), "lm_layer_norm_backward");
    const cudaStream_t s = c10::cuda::getCurrentCUDAStream(dev).stream();
    const Tensor ws = own_scratch(dev, need);
    ok(lm_layer_norm_backward(&p, ws.data_ptr(), static_cast<size_t>(ws.numel()), reinterpret_cast<lm_stream_t>(s)),
       "lm_layer_norm_backward");
    return {dx, dw, db, Tensor()};
  }
};

// A parameter of a layer: [size], contiguous, f32 or x's type.
const Tensor *vector_of(PyObject *o, const char *name, const Tensor &x, int64_t size) {
  const Tensor *t = on(o, name, x.get_device());
  if (t && ((t->scalar_type() != at::kFloat && t->scalar_type() != x.scalar_type()) || t->dim() != 1 ||
            t->size(0) != size || (size > 1 && t->stride(0) != 1)))
    refuse(std::string(name) + " must be [" + std::to_string(size) + "], contiguous, of dtype float32 or x's");
  return t;
}

// layer_norm(x, weight, bias, eps, out)
PyObject *layer_norm(PyObject *const *a) {
  const Tensor &x = tensor(a[0], "x");
  if (x.dim() < 1) refuse("x must be a CUDA tensor [..., width]");
  const int dev = x.get_device();
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  if (float_code(x.scalar_type()) < 0) refuse("x must be float32, float16 or bfloat16");
  const int64_t width = x.size(-1);
  if (width > 1 && x.stride(-1) != 1) refuse("the last dimension of x must be contiguous");
  (void)row_stride(x, "x");
  const Tensor *w = vector_of(a[1], "weight", x, width), *b = vector_of(a[2], "bias", x, width);
  const double eps = PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred()) return nullptr;
  if (!(static_cast<float>(eps) >= 0)) refuse("eps must be >= 0");
  const Tensor *given = on(a[4], "out", dev);
  no_tangents({&x, w, b, given});
  const bool grad = wants_grad({&x, w, b, given});
  if (given) {
    if (grad) throw std::runtime_error("log_mel_spectrogram_gb300: out goes without gradients (use torch.no_grad())");
    if (given->scalar_type() != x.scalar_type() || given->sizes() != x.sizes())
      refuse("out must have x's dtype and shape");
    if (width > 1 && given->stride(-1) != 1) refuse("the last dimension of out must be contiguous");
  }
  try {
    if (grad) {
      no_eager_graph({&x, w, b}, dev);
      return wrapped(NormFn::apply(x, optional(w), optional(b), eps));
    }
    const Tensor out = given ? *given : make(x.sizes(), x.scalar_type(), dev);
    norm_forward(x, defined_or_none(w), defined_or_none(b), eps, out, Tensor());
    written(given);
    return wrapped(out);
  } catch (const StatusError &e) {
    return status(e.rc);
  }
}

// ---- the gated layer ----

lm_gated_args gated_args(const Tensor &x, const Tensor &wg, const Tensor &wu, const Tensor &bg, const Tensor &bu,
                         int64_t act) {
  lm_gated_args p = {};
  p.x = x.data_ptr();
  p.w_gate = wg.data_ptr();
  p.w_up = wu.data_ptr();
  p.b_gate = ptr(bg);
  p.b_up = ptr(bu);
  p.rows = rows_of(x);
  p.k = x.size(-1);
  p.n = wg.size(0);
  p.x_row_stride = row_stride(x, "x");
  p.gate_row_stride = wg.stride(0);
  p.up_row_stride = wu.stride(0);
  p.dtype = half_code(x.scalar_type());
  const Tensor &b = bg.defined() ? bg : bu;
  p.bias_dtype = b.defined() ? float_code(b.scalar_type()) : LM_F32;
  p.activation = static_cast<int32_t>(act);
  return p;
}

void gated_forward(const Tensor &x, const Tensor &wg, const Tensor &wu, const Tensor &bg, const Tensor &bu, int64_t act,
                   const Tensor &out) {
  const int dev = x.get_device();
  lm_gated_args p = gated_args(x, wg, wu, bg, bu, act);
  p.out = out.data_ptr();
  p.out_row_stride = row_stride(out, "out");
  size_t need = 0;
  ok(lm_gated_linear_workspace_size(&p, &need), "lm_gated_linear");
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream(dev).stream();
  const Tensor ws = workspace(kLinear, dev, s, need);
  ok(lm_gated_linear(&p, ws.data_ptr(), static_cast<size_t>(ws.numel()), reinterpret_cast<lm_stream_t>(s)),
     "lm_gated_linear");
}

at::DimVector out_shape(const Tensor &x, int64_t n) {
  at::DimVector shape(x.sizes().begin(), x.sizes().end());
  shape.back() = n;
  return shape;
}

struct GatedFn : public torch::autograd::Function<GatedFn> {
  static Tensor forward(AutogradContext *ctx, const Tensor &x, const Tensor &wg, const Tensor &wu,
                        const Optional &b_gate, const Optional &b_up, int64_t act) {
    const Tensor bg = defined_or_none(b_gate), bu = defined_or_none(b_up);
    const Tensor out = make(out_shape(x, wg.size(0)), x.scalar_type(), x.get_device());
    gated_forward(x, wg, wu, bg, bu, act, out);
    ctx->save_for_backward({x, wg, wu, bg, bu});
    ctx->saved_data["act"] = act;
    return out;
  }

  static variable_list backward(AutogradContext *ctx, variable_list grads) {
    no_second_derivative();
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &x = saved[0], &wg = saved[1], &wu = saved[2], &bg = saved[3], &bu = saved[4];
    const int dev = x.get_device();
    const c10::cuda::OptionalCUDAGuard guard(x.device());
    no_eager_nodes(dev);
    const Tensor g = as_rows(grads[0]);
    lm_gated_backward_args p = {};
    p.forward = gated_args(x, wg, wu, bg, bu, ctx->saved_data["act"].toInt());
    p.grad = g.data_ptr();
    p.grad_row_stride = row_stride(g, "grad");
    Tensor d[5];
    size_t edge = 0;
    void **const to[5] = {&p.dx, &p.dw_gate, &p.dw_up, &p.db_gate, &p.db_up};
    for (int i = 0; i < 5; ++i) {
      const Tensor &t = saved[static_cast<size_t>(i)];
      if (!t.defined() || !ctx->needs_input_grad(edge++)) continue;
      d[i] = make(t.sizes(), t.scalar_type(), dev);
      *to[i] = d[i].data_ptr();
    }
    size_t need = 0;
    ok(lm_gated_linear_backward_workspace_size(&p, &need), "lm_gated_linear_backward");
    const cudaStream_t s = c10::cuda::getCurrentCUDAStream(dev).stream();
    const Tensor ws = own_scratch(dev, need);
    ok(lm_gated_linear_backward(&p, ws.data_ptr(), static_cast<size_t>(ws.numel()), reinterpret_cast<lm_stream_t>(s)),
       "lm_gated_linear_backward");
    return {d[0], d[1], d[2], d[3], d[4], Tensor()};
  }
};

// gated_linear(x, w_gate, w_up, b_gate, b_up, activation, out)
PyObject *gated_linear(PyObject *const *a) {
  const Tensor &x = tensor(a[0], "x");
  if (x.dim() < 1) refuse("x must be a CUDA tensor [..., K]");
  const int dev = x.get_device();
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  if (half_code(x.scalar_type()) < 0) refuse("x must be float16 or bfloat16");
  const Tensor *wg = on(a[1], "w_gate", dev), *wu = on(a[2], "w_up", dev);
  if (!wg || !wu) refuse("w_gate and w_up must be CUDA tensors");
  const int64_t k = x.size(-1);
  for (const Tensor *w : {wg, wu})
    if (w->scalar_type() != x.scalar_type() || w->dim() != 2 || w->size(1) != k || w->size(0) != wg->size(0))
      refuse("w_gate and w_up must be [N, K] of x's dtype and last dimension");
  const int64_t n = wg->size(0);
  if (k > 1 && (x.stride(-1) != 1 || wg->stride(1) != 1 || wu->stride(1) != 1))
    refuse("the last dimension of x, w_gate and w_up must be contiguous");
  (void)row_stride(x, "x");
  const Tensor *bg = vector_of(a[3], "b_gate", x, n), *bu = vector_of(a[4], "b_up", x, n);
  if (bg && bu && bg->scalar_type() != bu->scalar_type()) refuse("b_gate and b_up must be of one dtype");
  const long act = PyLong_AsLong(a[5]);
  if (PyErr_Occurred()) return nullptr;
  const Tensor *given = on(a[6], "out", dev);
  no_tangents({&x, wg, wu, bg, bu, given});
  const bool grad = wants_grad({&x, wg, wu, bg, bu, given});
  if (given) {
    if (grad) throw std::runtime_error("log_mel_spectrogram_gb300: out goes without gradients (use torch.no_grad())");
    if (given->scalar_type() != x.scalar_type() || given->sizes() != at::IntArrayRef(out_shape(x, n)))
      refuse("out must have x's dtype and leading dimensions, and N");
    if (n > 1 && given->stride(-1) != 1) refuse("the last dimension of out must be contiguous");
  }
  try {
    if (grad) {
      no_eager_graph({&x, wg, wu, bg, bu}, dev);
      return wrapped(GatedFn::apply(x, *wg, *wu, optional(bg), optional(bu), static_cast<int64_t>(act)));
    }
    const Tensor out = given ? *given : make(out_shape(x, n), x.scalar_type(), dev);
    gated_forward(x, *wg, *wu, defined_or_none(bg), defined_or_none(bu), act, out);
    written(given);
    return wrapped(out);
  } catch (const StatusError &e) {
    return status(e.rc);
  }
}

// ---- weights in 4 bits ----

PyObject *new_weight4(int64_t n, int64_t k, int group, int dev, lm_weight4 *c, Tensor *packed, Tensor *scale) {
  *c = {};
  c->n = n;
  c->k = k;
  c->group = group;
  size_t pb = 0, sb = 0;
  if (const int rc = lm_weight4_size(c, &pb, &sb); rc != LM_OK) return status(rc);
  const int64_t blocks = (n + 127) / 128, ktiles = (k + 63) / 64, groups = (k + group - 1) / group;
  *packed = make({blocks, ktiles, 4096}, at::kByte, dev);
  *scale = make({blocks, groups, 128}, at::kFloat, dev);
  c->packed = packed->data_ptr();
  c->scale = scale->data_ptr<float>();
  return nullptr;
}

// weight4_pack(q, scale, group) -> (packed, scale)
PyObject *weight4_pack(PyObject *const *a) {
  const Tensor &q = tensor(a[0], "q");
  const int dev = q.get_device();
  const c10::cuda::OptionalCUDAGuard guard(q.device());
  const Tensor *s = on(a[1], "scale", dev);
  const int group = static_cast<int>(PyLong_AsLong(a[2]));
  if (PyErr_Occurred()) return nullptr;
  if (q.scalar_type() != at::kChar || q.dim() != 2 || !q.is_contiguous())
    refuse("q must be a contiguous int8 CUDA tensor [N, K]");
  const int64_t n = q.size(0), k = q.size(1), groups = (k + group - 1) / group;
  if (!s || s->scalar_type() != at::kFloat || s->dim() != 2 || s->size(0) != n || s->size(1) != groups ||
      !s->is_contiguous())
    refuse("scale must be a contiguous float32 CUDA tensor [N, " + std::to_string(groups) + "]");
  no_grad({s});
  lm_weight4 c;
  Tensor packed, scale;
  if (PyObject *const bad = new_weight4(n, k, group, dev, &c, &packed, &scale)) return bad;
  if (const int rc = lm_weight4_pack(&c, static_cast<const int8_t *>(q.data_ptr()), s->data_ptr<float>(), stream_of(dev));
      rc != LM_OK)
    return status(rc);
  return Py_BuildValue("(NN)", wrapped(packed), wrapped(scale));
}

// weight4_quantize(weight, group) -> (packed, scale)
PyObject *weight4_quantize(PyObject *const *a) {
  const Tensor &w = tensor(a[0], "weight");
  const int dev = w.get_device();
  const c10::cuda::OptionalCUDAGuard guard(w.device());
  const int group = static_cast<int>(PyLong_AsLong(a[1]));
  if (PyErr_Occurred()) return nullptr;
  const int code = float_code(w.scalar_type());
  if (code < 0 || w.dim() != 2 || (w.size(1) > 1 && w.stride(1) != 1))
    refuse("weight must be a CUDA tensor [N, K] of float32, float16 or bfloat16 with K contiguous");
  no_grad({&w});
  lm_weight4 c;
  Tensor packed, scale;
  if (PyObject *const bad = new_weight4(w.size(0), w.size(1), group, dev, &c, &packed, &scale)) return bad;
  if (const int rc = lm_weight4_quantize(&c, w.data_ptr(), w.stride(0), code, stream_of(dev)); rc != LM_OK)
    return status(rc);
  return Py_BuildValue("(NN)", wrapped(packed), wrapped(scale));
}

// weight4_values(weight, dtype)
PyObject *weight4_values(PyObject *const *a) {
  const Weight4 w = weight4_of(a[0]);
  const int code = static_cast<int>(PyLong_AsLong(a[1]));
  if (PyErr_Occurred()) return nullptr;
  no_grad({&w.scale});
  const c10::cuda::OptionalCUDAGuard guard(w.packed.device());
  const Tensor out = make({w.c.n, w.c.k}, type_of(code), w.dev);
  if (const int rc = lm_weight4_values(&w.c, out.data_ptr(), w.c.k, code, stream_of(w.dev)); rc != LM_OK)
    return status(rc);
  return wrapped(out);
}

}  // namespace

Weight4 weight4_of(PyObject *o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 6) refuse("not a weight in 4 bits");
  Weight4 w;
  w.packed = tensor(PyTuple_GET_ITEM(o, 0), "weight");
  w.scale = tensor(PyTuple_GET_ITEM(o, 1), "weight");
  w.c = {};
  w.c.n = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 2));
  w.c.k = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 3));
  w.c.group = static_cast<int32_t>(PyLong_AsLong(PyTuple_GET_ITEM(o, 4)));
  w.code = static_cast<int>(PyLong_AsLong(PyTuple_GET_ITEM(o, 5)));
  if (PyErr_Occurred()) {
    PyErr_Clear();
    refuse("not a weight in 4 bits");
  }
  w.dev = w.packed.get_device();
  size_t pb = 0, sb = 0;
  if (lm_weight4_size(&w.c, &pb, &sb) != LM_OK || w.scale.get_device() != w.dev || !w.packed.is_contiguous() ||
      !w.scale.is_contiguous() || w.packed.nbytes() != pb || w.scale.nbytes() != sb ||
      w.packed.scalar_type() != at::kByte || w.scale.scalar_type() != at::kFloat)
    refuse("the tensors of a weight in 4 bits are not those that pack or quantize_weight made");
  w.c.packed = w.packed.data_ptr();
  w.c.scale = w.scale.data_ptr<float>();
  return w;
}

PyMethodDef kLayerMethods[] = {
    {"layer_norm", fast<layer_norm, 5>(), METH_FASTCALL, nullptr},
    {"gated_linear", fast<gated_linear, 7>(), METH_FASTCALL, nullptr},
    {"weight4_pack", fast<weight4_pack, 3>(), METH_FASTCALL, nullptr},
    {"weight4_quantize", fast<weight4_quantize, 2>(), METH_FASTCALL, nullptr},
    {"weight4_values", fast<weight4_values, 2>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

}  // namespace lm_binding
