// linear4.cu -- weights of 4 bits with group scales: their layout, rounding and values, and
// y = residual + scale * act(x W^T + bias) with such a weight.
#include <climits>

#include "activate.cuh"
#include "half.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace lm {
namespace {

constexpr int kTileBytes = 512;  // 16 rows by 64 k

struct Weight {
  const uint32_t *packed;
  const float *scale;
  int64_t n, k;
  int32_t group, ktiles, groups;
};

__host__ __device__ inline int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The word of `packed` that holds row i, k j .. j + 7 (j a multiple of 8).
__device__ __forceinline__ int64_t word_at(const Weight &w, int64_t i, int64_t j) {
  const int r = static_cast<int>(i % 16), c = static_cast<int>(j % 64);
  return (i / 16 * w.ktiles + j / 64) * (kTileBytes / 4) + (r % 8 * 4 + c / 16) * 4 + r / 8 * 2 + c / 8 % 2;
}

__device__ __forceinline__ int64_t scale_at(const Weight &w, int64_t i, int64_t g) {
  return (i / 16 * w.groups + g) * 16 + i % 16;
}

// q of k j + e in a word.
__device__ __forceinline__ int nibble(uint32_t word, int e) {
  return static_cast<int>(word >> (e / 2 * 4 + e % 2 * 16) & 15u) - 8;
}

// A warp a row and group: the scale (given, or from the largest value), and the words.
template <typename T, bool GIVEN>
__global__ void __launch_bounds__(256) fill_kernel(const Weight w, uint32_t *packed, float *scale, const T *src,
                                                   int64_t row_stride, const float *scales, int64_t units) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  pdl_launch();
  pdl_wait();
  if (unit >= units) return;
  const int64_t i = unit / w.groups, g = unit % w.groups;
  const bool row = i < w.n;
  float s = 0.0f;
  if (GIVEN) {
    s = row ? scales[i * w.groups + g] : 1.0f;
  } else {
    float m = 0.0f;
    for (int e = lane; e < w.group; e += 32) {
      const int64_t j = g * w.group + e;
      const float v = row && j < w.k ? fabsf(static_cast<float>(src[i * row_stride + j])) : 0.0f;
      m = v > m || v != v ? v : m;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float v = __shfl_xor_sync(0xffffffffu, m, o);
      m = v > m || v != v ? v : m;
    }
    s = m == 0.0f ? 1.0f : m / 7.0f;
    if (s == 0.0f) s = m;  // the smallest subnormals
  }
  if (lane == 0) scale[scale_at(w, i, g)] = s;
  // The last group also fills its tile.
  const int64_t end = g == w.groups - 1 ? static_cast<int64_t>(w.ktiles) * 64 : (g + 1) * w.group;
  for (int64_t j = g * w.group + 8 * lane; j < end; j += 256) {
    uint32_t word = 0;
    for (int e = 0; e < 8; ++e) {
      int q = 0;
      if (row && j + e < w.k) {
        if (GIVEN) {
          q = static_cast<int>(src[i * row_stride + j + e]);
        } else {
          const float v = rintf(static_cast<float>(src[i * row_stride + j + e]) / s);
          q = v == v ? static_cast<int>(fminf(fmaxf(v, -8.0f), 7.0f)) : 0;
        }
        q = q < -8 ? -8 : q > 7 ? 7 : q;
      }
      word |= static_cast<uint32_t>(q + 8) << (e / 2 * 4 + e % 2 * 16);
    }
    packed[word_at(w, i, j)] = word;
  }
}

// A thread a word: eight values.
template <typename T>
__global__ void __launch_bounds__(256) values_kernel(const Weight w, T *out, int64_t row_stride, int64_t words) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  pdl_launch();
  pdl_wait();
  const int64_t per = up(w.k, 8);
  if (t >= words) return;
  const int64_t i = t / per, j = t % per * 8;
  const uint32_t word = w.packed[word_at(w, i, j)];
  const float s = w.scale[scale_at(w, i, j / w.group)];
  for (int e = 0; e < 8 && j + e < w.k; ++e)
    out[i * row_stride + j + e] = from_f32<T>(static_cast<float>(nibble(word, e)) * s);
}

struct ProductParams {
  Weight w;
  const void *x, *bias, *residual;
  void *out;
  int64_t rows, group_rows, x_group, x_row, res_row, out_row;
  int32_t bias_f32, out_f32, act;
  float scale;
};

// A warp an output.
template <typename T>
__global__ void __launch_bounds__(256) product_kernel(const ProductParams p) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  pdl_launch();
  pdl_wait();
  if (unit >= p.rows * p.w.n) return;
  const int64_t row = unit / p.w.n, i = unit % p.w.n;
  const T *const x = static_cast<const T *>(p.x) + row / p.group_rows * p.x_group + row % p.group_rows * p.x_row;
  float s = 0.0f;
  for (int64_t j = 8 * lane; j < p.w.k; j += 256) {
    const uint32_t word = p.w.packed[word_at(p.w, i, j)];
    float part = 0.0f;
    for (int e = 0; e < 8 && j + e < p.w.k; ++e) part += static_cast<float>(nibble(word, e)) * to_f32(x[j + e]);
    s += part * p.w.scale[scale_at(p.w, i, j / p.w.group)];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane != 0) return;
  if (p.bias) s += p.bias_f32 ? static_cast<const float *>(p.bias)[i] : to_f32(static_cast<const T *>(p.bias)[i]);
  float y = p.scale * activate_any(s, p.act);
  if (p.residual) y += to_f32(static_cast<const T *>(p.residual)[row * p.res_row + i]);
  if (p.out_f32) {
    static_cast<float *>(p.out)[row * p.out_row + i] = y;
  } else {
    static_cast<T *>(p.out)[row * p.out_row + i] = from_f32<T>(y);
  }
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

lm_status view(const lm_weight4 *a, Weight *w) {
  if (!a || a->n < 0 || a->k < 0) return LM_ERR_INVALID_ARG;
  if ((a->group != 32 && a->group != 64 && a->group != 128) || a->n > INT_MAX - 512 || a->k > INT_MAX - 512)
    return LM_ERR_UNSUPPORTED;
  w->packed = static_cast<const uint32_t *>(a->packed);
  w->scale = a->scale;
  w->n = a->n;
  w->k = a->k;
  w->group = a->group;
  w->ktiles = static_cast<int32_t>(up(a->k, 64));
  w->groups = static_cast<int32_t>(up(a->k, a->group));
  return LM_OK;
}

// ... of a weight with contents.
lm_status whole(const Weight &w) {
  if (!w.packed || !w.scale) return LM_ERR_INVALID_ARG;
  return aligned(w.packed, 16) && aligned(w.scale, 16) ? LM_OK : LM_ERR_MISALIGNED;
}

template <typename T, bool GIVEN>
lm_status fill(const Weight &w, const T *src, int64_t row_stride, const float *scales, cudaStream_t s) {
  const int64_t units = up(w.n, 16) * 16 * w.groups;
  if (up(units, 8) > INT_MAX) return LM_ERR_UNSUPPORTED;
  return launch_dependent(fill_kernel<T, GIVEN>, dim3(static_cast<unsigned>(up(units, 8))), 256, 0, s, 1, w,
                          const_cast<uint32_t *>(w.packed), const_cast<float *>(w.scale), src, row_stride, scales, units);
}

template <typename T>
lm_status values(const Weight &w, void *out, int64_t row_stride, cudaStream_t s) {
  const int64_t words = w.n * up(w.k, 8);
  if (up(words, 256) > INT_MAX) return LM_ERR_UNSUPPORTED;
  return launch_dependent(values_kernel<T>, dim3(static_cast<unsigned>(up(words, 256))), 256, 0, s, 1, w,
                          static_cast<T *>(out), row_stride, words);
}

}  // namespace
}  // namespace lm

extern "C" lm_status lm_weight4_size(const lm_weight4 *a, size_t *packed_bytes, size_t *scale_bytes) {
  lm::Weight w;
  if (!packed_bytes || !scale_bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::view(a, &w); st != LM_OK) return st;
  const size_t ntiles = static_cast<size_t>(lm::up(w.n, 16));
  *packed_bytes = ntiles * static_cast<size_t>(w.ktiles) * lm::kTileBytes;
  *scale_bytes = ntiles * static_cast<size_t>(w.groups) * 64;
  return LM_OK;
}

extern "C" lm_status lm_weight4_pack(const lm_weight4 *a, const int8_t *q, const float *scales, lm_stream_t stream) {
  lm::Weight w;
  if (lm_status st = lm::view(a, &w); st != LM_OK) return st;
  if (w.n == 0 || w.k == 0) return LM_OK;
  if (!q || !scales) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::whole(w); st != LM_OK) return st;
  if (!lm::aligned(scales, 4)) return LM_ERR_MISALIGNED;
  return lm::fill<int8_t, true>(w, q, w.k, scales, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" lm_status lm_weight4_quantize(const lm_weight4 *a, const void *weight, int64_t row_stride, int32_t dtype,
                                         lm_stream_t stream) {
  lm::Weight w;
  if (lm_status st = lm::view(a, &w); st != LM_OK) return st;
  if (row_stride < 0) return LM_ERR_INVALID_ARG;
  if (dtype != LM_F32 && dtype != LM_F16 && dtype != LM_BF16) return LM_ERR_UNSUPPORTED;
  if (w.n == 0 || w.k == 0) return LM_OK;
  if (!weight) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::whole(w); st != LM_OK) return st;
  if (!lm::aligned(weight, dtype == LM_F32 ? 4 : 2)) return LM_ERR_MISALIGNED;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == LM_F32) return lm::fill<float, false>(w, static_cast<const float *>(weight), row_stride, nullptr, s);
  if (dtype == LM_F16) return lm::fill<__half, false>(w, static_cast<const __half *>(weight), row_stride, nullptr, s);
  return lm::fill<__nv_bfloat16, false>(w, static_cast<const __nv_bfloat16 *>(weight), row_stride, nullptr, s);
}

extern "C" lm_status lm_weight4_values(const lm_weight4 *a, void *out, int64_t row_stride, int32_t dtype,
                                       lm_stream_t stream) {
  lm::Weight w;
  if (lm_status st = lm::view(a, &w); st != LM_OK) return st;
  if (row_stride < 0 || (w.n > 1 && row_stride < w.k)) return LM_ERR_INVALID_ARG;
  if (dtype != LM_F32 && dtype != LM_F16 && dtype != LM_BF16) return LM_ERR_UNSUPPORTED;
  if (w.n == 0 || w.k == 0) return LM_OK;
  if (!out) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::whole(w); st != LM_OK) return st;
  if (!lm::aligned(out, dtype == LM_F32 ? 4 : 2)) return LM_ERR_MISALIGNED;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == LM_F32   ? lm::values<float>(w, out, row_stride, s)
         : dtype == LM_F16 ? lm::values<__half>(w, out, row_stride, s)
                           : lm::values<__nv_bfloat16>(w, out, row_stride, s);
}

extern "C" int lm_linear4_expands(int64_t, int64_t, int64_t) { return 0; }

namespace lm {
namespace {

lm_status check4(const lm_linear_args *a, const lm_weight4 *wa, Weight *w) {
  if (lm_status st = linear_check(a); st != LM_OK) return st;
  if (lm_status st = view(wa, w); st != LM_OK) return st;
  return w->n == a->n && w->k == a->k ? LM_OK : LM_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace lm

extern "C" lm_status lm_linear4_workspace_size(const lm_linear_args *args, const lm_weight4 *weight, size_t *bytes) {
  lm::Weight w;
  if (!bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::check4(args, weight, &w); st != LM_OK) return st;
  *bytes = 256;
  return LM_OK;
}

extern "C" lm_status lm_linear4(const lm_linear_args *args, const lm_weight4 *weight, void *workspace,
                                size_t workspace_bytes, lm_stream_t stream) {
  using namespace lm;
  Weight w;
  size_t need = 0;
  if (lm_status st = check4(args, weight, &w); st != LM_OK) return st;
  if (lm_status st = lm_linear4_workspace_size(args, weight, &need); st != LM_OK) return st;
  const lm_linear_args &a = *args;
  const int64_t rows = a.groups * a.rows;
  if (rows == 0 || a.n == 0) return LM_OK;
  if (!a.out || (a.k > 0 && !a.x)) return LM_ERR_INVALID_ARG;
  if (a.k > 0)
    if (lm_status st = whole(w); st != LM_OK) return st;
  const int64_t out_size = a.out_dtype == LM_F32 ? 4 : 2;
  if (!aligned(a.x, 2) || !aligned(a.bias, a.bias_dtype == LM_F32 ? 4 : 2) || !aligned(a.residual, 2) ||
      !aligned(a.out, static_cast<size_t>(out_size)) || !aligned(workspace, 16))
    return LM_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < need) return LM_ERR_WORKSPACE;
  // The output's rows run into one another or into an input.
  const ByteRows out{a.out, rows, a.out_row_stride * out_size, a.n * out_size};
  if (rows > 1 && a.out_row_stride < a.n) return LM_ERR_INVALID_ARG;
  size_t packed_bytes = 0, scale_bytes = 0;
  (void)lm_weight4_size(weight, &packed_bytes, &scale_bytes);
  if (a.k > 0) {
    const ByteRows row{a.x, a.rows, a.x_row_stride * 2, a.k * 2};
    const ByteRows all = a.groups == 1 ? row
                         : a.rows == 1 ? ByteRows{a.x, a.groups, a.x_group_stride * 2, a.k * 2}
                                       : ByteRows{a.x, a.groups, a.x_group_stride * 2, (a.rows - 1) * row.step + row.size};
    if (rows_meet(out, all) || rows_meet(out, {w.packed, 1, 0, static_cast<int64_t>(packed_bytes)}) ||
        rows_meet(out, {w.scale, 1, 0, static_cast<int64_t>(scale_bytes)}))
      return LM_ERR_INVALID_ARG;
  }
  if (a.bias && rows_meet(out, {a.bias, 1, 0, a.n * (a.bias_dtype == LM_F32 ? 4 : 2)})) return LM_ERR_INVALID_ARG;
  const bool same = a.residual == a.out && out_size == 2 && (rows == 1 || a.residual_row_stride == a.out_row_stride);
  if (a.residual && !same && rows_meet(out, {a.residual, rows, a.residual_row_stride * 2, a.n * 2}))
    return LM_ERR_INVALID_ARG;
  ProductParams p = {};
  p.w = w;
  p.x = a.x;
  p.bias = a.bias;
  p.residual = a.residual;
  p.out = a.out;
  p.rows = rows;
  p.group_rows = a.rows;
  p.x_group = a.x_group_stride;
  p.x_row = a.x_row_stride;
  p.res_row = a.residual_row_stride;
  p.out_row = a.out_row_stride;
  p.bias_f32 = a.bias_dtype == LM_F32;
  p.out_f32 = a.out_dtype == LM_F32;
  p.act = a.activation;
  p.scale = a.scale;
  const int64_t ctas = up(rows * a.n, 8);
  if (ctas > INT_MAX) return LM_ERR_UNSUPPORTED;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launch_dependent(a.dtype == LM_F16 ? product_kernel<__half> : product_kernel<__nv_bfloat16>,
                          dim3(static_cast<unsigned>(ctas)), 256, 0, s, 1, p);
}
