// norm.cu -- layer norm over the last dimension, forward and backward.
//
// Forward: mean, then the deviations d = x - mean from the rounded mean; their
// own mean puts right what rounding left off, so that
//   var = avg(d^2) - avg(d)^2,  n = (d - avg(d)) / sqrt(var + eps).
// Backward, with h = grad * weight:
//   dx = (h - avg(h) - n avg(h n)) / sqrt(var + eps),
//   dweight = sum over rows of grad n,  dbias = sum over rows of grad.
#include <climits>

#include "half.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace lm {
namespace {

constexpr int kThreads = 256;
constexpr int kMostChunks = 304;  // parts of the rows whose sums are joined at the end

struct NormParams {
  const void *x, *weight, *bias, *grad;
  void *out;              // y, or dx
  float *stats;           // [3][rows]
  float *partial;         // [chunks][2][width]
  int64_t rows, width, x_row, grad_row, out_row;
  int32_t weight_f32, bias_f32, chunks;
  float eps;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The sums of two values over the CTA, for every thread.
__device__ __forceinline__ float2 cta_sum2(float a, float b, float2 *scratch) {
  a = warp_sum(a);
  b = warp_sum(b);
  __syncthreads();
  if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = make_float2(a, b);
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
  for (int i = 0; i < kThreads / 32; ++i) {
    s.x += scratch[i].x;
    s.y += scratch[i].y;
  }
  return s;
}

template <typename T>
__device__ __forceinline__ float param_at(const void *p, int f32, int64_t i, float otherwise) {
  if (!p) return otherwise;
  return f32 ? static_cast<const float *>(p)[i] : to_f32(static_cast<const T *>(p)[i]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_rows(const NormParams p) {
  __shared__ float2 scratch[kThreads / 32];
  pdl_launch();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const T *const x = static_cast<const T *>(p.x) + row * p.x_row;
  T *const out = static_cast<T *>(p.out) + row * p.out_row;
  const float inv = 1.0f / static_cast<float>(p.width);
  float s = 0.0f, q = 0.0f;
  for (int64_t i = threadIdx.x; i < p.width; i += kThreads) s += to_f32(x[i]);
  const float mean = cta_sum2(s, 0.0f, scratch).x * inv;
  s = 0.0f;
  for (int64_t i = threadIdx.x; i < p.width; i += kThreads) {
    const float d = to_f32(x[i]) - mean;
    s += d;
    q += d * d;
  }
  const float2 t = cta_sum2(s, q, scratch);
  const float off = t.x * inv, var = t.y * inv - off * off;
  const float r = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + p.eps);
  if (p.stats && threadIdx.x == 0) {
    p.stats[row] = mean;
    p.stats[p.rows + row] = off;
    p.stats[2 * p.rows + row] = r;
  }
  for (int64_t i = threadIdx.x; i < p.width; i += kThreads) {
    const float n = ((to_f32(x[i]) - mean) - off) * r;
    out[i] = from_f32<T>(n * param_at<T>(p.weight, p.weight_f32, i, 1.0f) + param_at<T>(p.bias, p.bias_f32, i, 0.0f));
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_backward_rows(const NormParams p) {
  __shared__ float2 scratch[kThreads / 32];
  pdl_launch();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const T *const x = static_cast<const T *>(p.x) + row * p.x_row;
  const T *const g = static_cast<const T *>(p.grad) + row * p.grad_row;
  T *const out = static_cast<T *>(p.out) + row * p.out_row;
  const float mean = p.stats[row], off = p.stats[p.rows + row], r = p.stats[2 * p.rows + row];
  const float inv = 1.0f / static_cast<float>(p.width);
  float s = 0.0f, q = 0.0f;
  for (int64_t i = threadIdx.x; i < p.width; i += kThreads) {
    const float n = ((to_f32(x[i]) - mean) - off) * r;
    const float h = to_f32(g[i]) * param_at<T>(p.weight, p.weight_f32, i, 1.0f);
    s += h;
    q += h * n;
  }
  const float2 t = cta_sum2(s, q, scratch);
  for (int64_t i = threadIdx.x; i < p.width; i += kThreads) {
    const float n = ((to_f32(x[i]) - mean) - off) * r;
    const float h = to_f32(g[i]) * param_at<T>(p.weight, p.weight_f32, i, 1.0f);
    out[i] = from_f32<T>((h - t.x * inv - n * (t.y * inv)) * r);
  }
}

// Sums over a part of the rows (blockIdx.y) for a thread's column.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_backward_columns(const NormParams p) {
  pdl_launch();
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= p.width) return;
  const int64_t first = p.rows * blockIdx.y / p.chunks, end = p.rows * (blockIdx.y + 1) / p.chunks;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = first; row < end; ++row) {
    const float g = to_f32(static_cast<const T *>(p.grad)[row * p.grad_row + i]);
    const float d = to_f32(static_cast<const T *>(p.x)[row * p.x_row + i]) - p.stats[row];
    dw += g * ((d - p.stats[p.rows + row]) * p.stats[2 * p.rows + row]);
    db += g;
  }
  float *const to = p.partial + static_cast<int64_t>(blockIdx.y) * 2 * p.width + i;
  to[0] = dw;
  to[p.width] = db;
}

// Joins the parts in their order.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_join(const float *partial, int chunks, int64_t width, void *dweight,
                                                      int weight_f32, void *dbias, int bias_f32) {
  pdl_launch();
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= 2 * width) return;
  float s = 0.0f;
  for (int c = 0; c < chunks; ++c) s += partial[static_cast<int64_t>(c) * 2 * width + i];
  void *const to = i < width ? dweight : dbias;
  if (!to) return;
  const int64_t at = i < width ? i : i - width;
  if (i < width ? weight_f32 : bias_f32) {
    static_cast<float *>(to)[at] = s;
  } else {
    static_cast<T *>(to)[at] = from_f32<T>(s);
  }
}

int64_t size_of(int32_t dtype) { return dtype == LM_F32 ? 4 : 2; }
bool aligned(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(n) == 0; }
bool float_type(int32_t t) { return t == LM_F32 || t == LM_F16 || t == LM_BF16; }

lm_status check_sizes(int64_t rows, int64_t width, int64_t x_row, int64_t other_row, int32_t dtype, int32_t weight_dtype,
                      int32_t bias_dtype) {
  if (rows < 0 || width < 0 || x_row < 0 || other_row < 0) return LM_ERR_INVALID_ARG;
  if (!float_type(dtype) || (weight_dtype != LM_F32 && weight_dtype != dtype) ||
      (bias_dtype != LM_F32 && bias_dtype != dtype))
    return LM_ERR_UNSUPPORTED;
  const int64_t most = INT_MAX - 512;
  if (rows > most || width > most || (width > 0 && rows > (1ll << 60) / width) || x_row > (1ll << 38) ||
      other_row > (1ll << 38))
    return LM_ERR_UNSUPPORTED;
  return LM_OK;
}

template <typename T>
lm_status forward(const NormParams &p, cudaStream_t s) {
  return launch_dependent(norm_rows<T>, dim3(static_cast<unsigned>(p.rows)), kThreads, 0, s, 1, p);
}

int chunks_of(int64_t rows) { return rows < kMostChunks ? static_cast<int>(rows) : kMostChunks; }

template <typename T>
lm_status backward(NormParams p, void *dweight, void *dbias, cudaStream_t s) {
  if (p.out && p.rows > 0)
    if (lm_status st = launch_dependent(norm_backward_rows<T>, dim3(static_cast<unsigned>(p.rows)), kThreads, 0, s, 1, p);
        st != LM_OK)
      return st;
  if (!dweight && !dbias) return LM_OK;
  const unsigned across = static_cast<unsigned>((p.width + kThreads - 1) / kThreads);
  if (p.chunks > 0)
    if (lm_status st = launch_dependent(norm_backward_columns<T>, dim3(across, static_cast<unsigned>(p.chunks)), kThreads,
                                        0, s, 1, p);
        st != LM_OK)
      return st;
  return launch_dependent(norm_join<T>, dim3(static_cast<unsigned>((2 * p.width + kThreads - 1) / kThreads)), kThreads, 0,
                          s, 1, p.partial, p.chunks, p.width, dweight, p.weight_f32, dbias, p.bias_f32);
}

}  // namespace
}  // namespace lm

extern "C" lm_status lm_layer_norm(const lm_norm_args *a, lm_stream_t stream) {
  using namespace lm;
  if (!a) return LM_ERR_INVALID_ARG;
  if (lm_status st =
          check_sizes(a->rows, a->width, a->x_row_stride, a->out_row_stride, a->dtype, a->weight_dtype, a->bias_dtype);
      st != LM_OK)
    return st;
  if (!(a->eps >= 0.0f)) return LM_ERR_INVALID_ARG;
  if (a->rows == 0 || a->width == 0) return LM_OK;
  if (!a->x || !a->out) return LM_ERR_INVALID_ARG;
  const int64_t size = size_of(a->dtype), ws = size_of(a->weight_dtype), bs = size_of(a->bias_dtype);
  if (!aligned(a->x, size) || !aligned(a->out, size) || !aligned(a->weight, ws) || !aligned(a->bias, bs) ||
      !aligned(a->stats, 4))
    return LM_ERR_MISALIGNED;
  const ByteRows out{a->out, a->rows, a->out_row_stride * size, a->width * size};
  const ByteRows x{a->x, a->rows, a->x_row_stride * size, a->width * size};
  const bool same = a->out == a->x && (a->rows == 1 || a->out_row_stride == a->x_row_stride);
  if ((a->rows > 1 && a->out_row_stride < a->width) || (!same && rows_meet(out, x)) ||
      (a->weight && rows_meet(out, {a->weight, 1, 0, a->width * ws})) ||
      (a->bias && rows_meet(out, {a->bias, 1, 0, a->width * bs})))
    return LM_ERR_INVALID_ARG;
  if (a->stats) {
    const ByteRows stats{a->stats, 1, 0, a->rows * 12};
    if (rows_meet(stats, out) || rows_meet(stats, x) || (a->weight && rows_meet(stats, {a->weight, 1, 0, a->width * ws})) ||
        (a->bias && rows_meet(stats, {a->bias, 1, 0, a->width * bs})))
      return LM_ERR_INVALID_ARG;
  }
  NormParams p = {};
  p.x = a->x;
  p.weight = a->weight;
  p.bias = a->bias;
  p.out = a->out;
  p.stats = a->stats;
  p.rows = a->rows;
  p.width = a->width;
  p.x_row = a->x_row_stride;
  p.out_row = a->out_row_stride;
  p.weight_f32 = a->weight_dtype == LM_F32;
  p.bias_f32 = a->bias_dtype == LM_F32;
  p.eps = a->eps;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return a->dtype == LM_F32 ? forward<float>(p, s) : a->dtype == LM_F16 ? forward<__half>(p, s)
                                                                       : forward<__nv_bfloat16>(p, s);
}

extern "C" lm_status lm_layer_norm_backward_workspace_size(const lm_norm_backward_args *a, size_t *bytes) {
  using namespace lm;
  if (!a || !bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st =
          check_sizes(a->rows, a->width, a->x_row_stride, a->grad_row_stride, a->dtype, a->weight_dtype, a->bias_dtype);
      st != LM_OK)
    return st;
  *bytes = 256 + static_cast<size_t>(chunks_of(a->rows)) * 8 * static_cast<size_t>(a->width);
  return LM_OK;
}

extern "C" lm_status lm_layer_norm_backward(const lm_norm_backward_args *a, void *workspace, size_t workspace_bytes,
                                            lm_stream_t stream) {
  using namespace lm;
  size_t need = 0;
  if (lm_status st = lm_layer_norm_backward_workspace_size(a, &need); st != LM_OK) return st;
  if (a->width == 0 || (!a->dx && !a->dweight && !a->dbias)) return LM_OK;
  if (a->rows > 0 && (!a->x || !a->grad || !a->stats)) return LM_ERR_INVALID_ARG;
  const int64_t size = size_of(a->dtype), ws = size_of(a->weight_dtype), bs = size_of(a->bias_dtype);
  if (!aligned(a->x, size) || !aligned(a->grad, size) || !aligned(a->dx, size) || !aligned(a->weight, ws) ||
      !aligned(a->dweight, ws) || !aligned(a->dbias, bs) || !aligned(a->stats, 4) || !aligned(workspace, 16))
    return LM_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < need) return LM_ERR_WORKSPACE;
  const ByteRows in[] = {{a->x, a->rows, a->x_row_stride * size, a->width * size},
                         {a->grad, a->rows, a->grad_row_stride * size, a->width * size},
                         {a->weight, a->weight ? 1 : 0, 0, a->width * ws},
                         {a->stats, 1, 0, a->rows * 12}};
  const ByteRows outs[] = {{a->dx, a->dx ? 1 : 0, 0, a->rows * a->width * size},
                           {a->dweight, a->dweight ? 1 : 0, 0, a->width * ws},
                           {a->dbias, a->dbias ? 1 : 0, 0, a->width * bs}};
  for (int i = 0; i < 3; ++i) {
    for (const ByteRows &r : in)
      if (rows_meet(outs[i], r)) return LM_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (rows_meet(outs[i], outs[j])) return LM_ERR_INVALID_ARG;
  }
  NormParams p = {};
  p.x = a->x;
  p.weight = a->weight;
  p.grad = a->grad;
  p.out = a->dx;
  p.stats = const_cast<float *>(a->stats);
  p.partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + 256);
  p.rows = a->rows;
  p.width = a->width;
  p.x_row = a->x_row_stride;
  p.grad_row = a->grad_row_stride;
  p.out_row = a->width;
  p.weight_f32 = a->weight_dtype == LM_F32;
  p.bias_f32 = a->bias_dtype == LM_F32;
  p.chunks = chunks_of(a->rows);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return a->dtype == LM_F32   ? backward<float>(p, a->dweight, a->dbias, s)
         : a->dtype == LM_F16 ? backward<__half>(p, a->dweight, a->dbias, s)
                              : backward<__nv_bfloat16>(p, a->dweight, a->dbias, s);
}
