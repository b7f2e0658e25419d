// linear4.cu -- weights of 4 bits with group scales: their layout, rounding and values, and
// y = residual + scale * act(x W^T + bias) with such a weight.
//
// Few rows of x: the weight's bytes bound the call.  They are laid out so that a lane's 16 bytes of
// a tile are its operands of four m16n8k16 products with W as the 16 rows, and 16 bytes of x twice the
// other operand: neither goes through shared memory, and a nibble becomes a 16-bit float by an OR into
// the mantissa of 1024 (f16) or 128 (bf16) and an exact subtraction.  (tcgen05 takes no operand that has to
// be converted first without a pass through shared memory.)  A warp sums a tile of 16 outputs over a part of
// k, a group's products in 32 bits and then times its scale; the warps of a CTA share out tiles and
// k, meet in shared memory, and write whole lines.
//
// Many rows: products bound it, and the legacy matrix instruction with them.  The values are expanded into
// the workspace, rounded to x's type, and linear.cu's kernel takes them.
#include <climits>

#include "activate.cuh"
#include "half.cuh"
#include "internal.h"
#include "mma.cuh"
#include "operand.cuh"
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
  return (i / 16 * w.ktiles + j / 64) * (kTileBytes / 4) + (r % 8 * 4 + c % 32 / 8) * 4 + r / 8 * 2 + c / 32;
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

// A thread a word: eight values.  WHOLE: rows of 16-byte vectors, zeros past k.
template <typename T, bool WHOLE>
__global__ void __launch_bounds__(256) values_kernel(const Weight w, T *out, int64_t row_stride, int64_t words) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  pdl_launch();
  pdl_wait();
  const int64_t per = up(w.k, 8);
  if (t >= words) return;
  const int64_t i = t / per, j = t % per * 8;
  const uint32_t word = w.packed[word_at(w, i, j)];
  const float s = w.scale[scale_at(w, i, j / w.group)];
  if constexpr (WHOLE) {
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      v[e / 2] = pack2<T>(j + e < w.k ? static_cast<float>(nibble(word, e)) * s : 0.0f,
                          j + e + 1 < w.k ? static_cast<float>(nibble(word, e + 1)) * s : 0.0f);
    *reinterpret_cast<uint4 *>(out + i * row_stride + j) = make_uint4(v[0], v[1], v[2], v[3]);
  } else {
    for (int e = 0; e < 8 && j + e < w.k; ++e)
      out[i * row_stride + j + e] = from_f32<T>(static_cast<float>(nibble(word, e)) * s);
  }
}

struct ProductParams {
  Weight w;
  const void *x, *bias, *residual;
  void *out;
  int64_t x_group, x_row, res_row, out_row;
  int32_t rows, group_rows, ntiles, parts;  // parts: warps that share out a tile's k
  int32_t bias_f32, out_f32, act;
  float scale;
};

constexpr int kWarps = 8;

__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) { return (w & mask) | bits; }

// The four pairs of a word (k 0 1, 2 3, 4 5, 6 7) as 16-bit floats of -8 .. 7.
template <typename T>
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&v)[4]);
template <>
__device__ __forceinline__ void widen<__half>(uint32_t w, uint32_t (&v)[4]) {
  // Nibble q + 8 in the low bits of 1024's mantissa is 1032 + q, four bits up 1152 + 16 q.
  const __half2 low = __floats2half2_rn(1032.0f, 1032.0f), sixteenth = __floats2half2_rn(0.0625f, 0.0625f),
                high = __floats2half2_rn(-72.0f, -72.0f);
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t a = and_or(w >> (4 * i), 0x000f000fu, 0x64006400u), b = and_or(w >> (4 * i), 0x00f000f0u, 0x64006400u);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), low);
    const __half2 y = __hfma2(*reinterpret_cast<const __half2 *>(&b), sixteenth, high);
    v[i] = *reinterpret_cast<const uint32_t *>(&x);
    v[i + 1] = *reinterpret_cast<const uint32_t *>(&y);
  }
}
template <>
__device__ __forceinline__ void widen<__nv_bfloat16>(uint32_t w, uint32_t (&v)[4]) {
  const __nv_bfloat162 low = __floats2bfloat162_rn(136.0f, 136.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = and_or(w >> (4 * i), 0x000f000fu, 0x43004300u);  // 128 + 8 + q
    const __nv_bfloat162 x = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), low);
    v[i] = *reinterpret_cast<const uint32_t *>(&x);
  }
}

// A weight's 16 bytes pass once: they leave the L1 to x.
__device__ __forceinline__ uint4 load_once(const uint32_t *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Eight elements of a row from k on, zeros past its end.
template <typename T>
__device__ __forceinline__ uint4 load8(const T *row, int k, int end) {
  if (row && k + 8 <= end) return *reinterpret_cast<const uint4 *>(row + k);
  uint32_t v[4] = {0, 0, 0, 0};
  if (row && k < end) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k + j < end) v[j / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(row + k + j)) << (16 * (j % 2));
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// One output element.
template <typename T>
__device__ __forceinline__ void put(const ProductParams &p, float s, int row, int n) {
  if (p.bias) s += p.bias_f32 ? static_cast<const float *>(p.bias)[n] : to_f32(static_cast<const T *>(p.bias)[n]);
  float y = p.scale * activate_any(s, p.act);
  if (p.residual) y += to_f32(static_cast<const T *>(p.residual)[row * p.res_row + n]);
  if (p.out_f32) {
    static_cast<float *>(p.out)[row * p.out_row + n] = y;
  } else {
    static_cast<T *>(p.out)[row * p.out_row + n] = from_f32<T>(y);
  }
}

// NT: blocks of eight rows of x; blockIdx.y counts such tiles.  SMALL: groups of 32, two to a tile.
template <typename T, int NT, bool SMALL>
__global__ void __launch_bounds__(32 * kWarps) product_kernel(const ProductParams p) {
  constexpr int AHEAD = NT <= 2 ? 4 : 2;  // tiles whose bytes are on their way
  constexpr int SCALES = SMALL ? 2 : 1;
  __shared__ float sums[kWarps][8 * NT][16 + 1];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, r = lane / 4, c = lane % 4;
  const int part = warp % p.parts, per = kWarps / p.parts;
  const int tile = static_cast<int>(blockIdx.x) * per + warp / p.parts;
  const int row0 = static_cast<int>(blockIdx.y) * 8 * NT, k = static_cast<int>(p.w.k);
  const bool any = tile < p.ntiles;
  const int begin = any ? static_cast<int>(static_cast<int64_t>(p.w.ktiles) * part / p.parts) : 0;
  const int end = any ? static_cast<int>(static_cast<int64_t>(p.w.ktiles) * (part + 1) / p.parts) : 0;
  pdl_launch();
  pdl_wait();
  const uint32_t *const packed = p.w.packed + static_cast<int64_t>(tile) * p.w.ktiles * (kTileBytes / 4) + lane * 4;
  const float *const scales = p.w.scale + static_cast<int64_t>(tile) * p.w.groups * 16 + r;
  const T *x[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = row0 + 8 * t + r;
    x[t] = row < p.rows ? static_cast<const T *>(p.x) + row / p.group_rows * p.x_group + row % p.group_rows * p.x_row
                        : nullptr;
  }
  float total[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) total[t][j] = 0.0f;

  uint4 w[AHEAD];
  float s[AHEAD][SCALES][2];
  auto fetch = [&](int u, int kt) {
    w[u] = load_once(packed + static_cast<int64_t>(kt) * (kTileBytes / 4));
#pragma unroll
    for (int h = 0; h < SCALES; ++h) {
      int g = SMALL ? 2 * kt + h : kt * 64 / p.w.group;
      if (SMALL && g >= p.w.groups) g = p.w.groups - 1;  // (its half of the tile is zeros)
      s[u][h][0] = scales[g * 16];
      s[u][h][1] = scales[g * 16 + 8];
    }
  };
#pragma unroll
  for (int u = 0; u < AHEAD; ++u)
    if (begin + u < end) fetch(u, begin + u);
  for (int base = begin; base < end; base += AHEAD) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int kt = base + u;
      if (kt >= end) break;
      uint32_t v[4][4];  // words: row r, the tile's first and second half of k; row r + 8
      widen<T>(w[u].x, v[0]);
      widen<T>(w[u].y, v[1]);
      widen<T>(w[u].z, v[2]);
      widen<T>(w[u].w, v[3]);
      float f[SCALES][2];
#pragma unroll
      for (int h = 0; h < SCALES; ++h) {
        f[h][0] = s[u][h][0];
        f[h][1] = s[u][h][1];
      }
      if (kt + AHEAD < end) fetch(u, kt + AHEAD);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 b = load8<T>(x[t], kt * 64 + 32 * h + 8 * c, k);
          const uint32_t a0[4] = {v[h][0], v[h + 2][0], v[h][1], v[h + 2][1]};
          const uint32_t a1[4] = {v[h][2], v[h + 2][2], v[h][3], v[h + 2][3]};
          mma16816<T>(d, a0, b.x, b.y);
          mma16816<T>(d, a1, b.z, b.w);
          if (SMALL || h == 1) {
            const int g = SMALL ? h : 0;
            total[t][0] = fmaf(f[g][0], d[0], total[t][0]);
            total[t][1] = fmaf(f[g][0], d[1], total[t][1]);
            total[t][2] = fmaf(f[g][1], d[2], total[t][2]);
            total[t][3] = fmaf(f[g][1], d[3], total[t][3]);
            d[0] = d[1] = d[2] = d[3] = 0.0f;
          }
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    sums[warp][8 * t + 2 * c][r] = total[t][0];
    sums[warp][8 * t + 2 * c + 1][r] = total[t][1];
    sums[warp][8 * t + 2 * c][r + 8] = total[t][2];
    sums[warp][8 * t + 2 * c + 1][r + 8] = total[t][3];
  }
  __syncthreads();
  const int wide = 16 * per, rows = min(8 * NT, p.rows - row0);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * wide;
  for (int i = threadIdx.x; i < rows * wide; i += 32 * kWarps) {
    const int row = i / wide, at = i % wide;
    if (n0 + at >= p.w.n) continue;
    float sum = 0.0f;
    for (int q = 0; q < p.parts; ++q) sum += sums[at / 16 * p.parts + q][row][at % 16];
    put<T>(p, sum, row0 + row, static_cast<int>(n0) + at);
  }
}

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

// From this many rows on the products cost more than expanding the weight.
bool expands(int64_t rows, int64_t, int64_t) { return rows > 128; }

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
  return launch_dependent(values_kernel<T, false>, dim3(static_cast<unsigned>(up(words, 256))), 256, 0, s, 1, w,
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

extern "C" int lm_linear4_expands(int64_t rows, int64_t n, int64_t k) { return lm::expands(rows, n, k); }

namespace lm {
namespace {

lm_status check4(const lm_linear_args *a, const lm_weight4 *wa, Weight *w) {
  if (lm_status st = linear_check(a); st != LM_OK) return st;
  if (lm_status st = view(wa, w); st != LM_OK) return st;
  return w->n == a->n && w->k == a->k ? LM_OK : LM_ERR_INVALID_ARG;
}

size_t padded(size_t n) { return (n + 255) / 256 * 256; }

// linear.cu's arguments for the expanded weight at `at`.
lm_linear_args expanded(const lm_linear_args &a, const void *at) {
  lm_linear_args e = a;
  e.weight = at;
  e.weight_row_stride = up(a.k, 8) * 8;
  return e;
}

// Bytes: what linear.cu takes (or a copy of x), then the expanded weight.
lm_status sizes(const lm_linear_args &a, size_t *first, size_t *all) {
  if (expands(a.groups * a.rows, a.n, a.k)) {
    const lm_linear_args e = expanded(a, reinterpret_cast<const void *>(static_cast<uintptr_t>(256)));
    if (lm_status st = lm_linear_workspace_size(&e, first); st != LM_OK) return st;
    *first = padded(*first);
    *all = *first + padded(static_cast<size_t>(a.n) * static_cast<size_t>(up(a.k, 8)) * 16);
  } else {
    *first = *all = 256 + padded(operand(a.x, a.groups, a.rows, a.k, a.x_group_stride, a.x_row_stride).bytes);
  }
  return LM_OK;
}

template <typename T, int NT>
lm_status product_as(const ProductParams &p, dim3 grid, cudaStream_t s) {
  return launch_dependent(p.w.group == 32 ? product_kernel<T, NT, true> : product_kernel<T, NT, false>, grid, 32 * kWarps,
                          0, s, 1, p);
}

template <typename T>
lm_status product(ProductParams p, int sms, cudaStream_t s) {
  const int nt = p.rows <= 8 ? 1 : p.rows <= 16 ? 2 : p.rows <= 32 ? 4 : 8;
  const int64_t blocks = up(p.rows, 8 * nt);
  // As many parts of k as give every SM a dozen warps.
  p.parts = 1;
  while (p.parts < kWarps && 2 * p.parts <= p.w.ktiles && p.ntiles * blocks * p.parts < 12ll * sms) p.parts *= 2;
  const dim3 grid(static_cast<unsigned>(up(p.ntiles, kWarps / p.parts)), static_cast<unsigned>(blocks));
  return nt == 1   ? product_as<T, 1>(p, grid, s)
         : nt == 2 ? product_as<T, 2>(p, grid, s)
         : nt == 4 ? product_as<T, 4>(p, grid, s)
                   : product_as<T, 8>(p, grid, s);
}

}  // namespace
}  // namespace lm

extern "C" lm_status lm_linear4_workspace_size(const lm_linear_args *args, const lm_weight4 *weight, size_t *bytes) {
  lm::Weight w;
  size_t first = 0;
  if (!bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::check4(args, weight, &w); st != LM_OK) return st;
  return lm::sizes(*args, &first, bytes);
}

extern "C" lm_status lm_linear4(const lm_linear_args *args, const lm_weight4 *weight, void *workspace,
                                size_t workspace_bytes, lm_stream_t stream) {
  using namespace lm;
  Weight w;
  size_t first = 0, need = 0;
  if (lm_status st = check4(args, weight, &w); st != LM_OK) return st;
  const lm_linear_args &a = *args;
  if (lm_status st = sizes(a, &first, &need); st != LM_OK) return st;
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
  Operand x = operand(a.x, a.groups, a.rows, a.k, a.x_group_stride, a.x_row_stride);
  if (a.k > 0) {
    const ByteRows row{x.p, x.rows, x.row_stride * 2, a.k * 2};
    const ByteRows all = x.groups == 1 ? row
                                       : ByteRows{x.p, x.groups, x.group_stride * 2, (x.rows - 1) * row.step + row.size};
    if (rows_meet(out, all) || rows_meet(out, {w.packed, 1, 0, static_cast<int64_t>(packed_bytes)}) ||
        rows_meet(out, {w.scale, 1, 0, static_cast<int64_t>(scale_bytes)}))
      return LM_ERR_INVALID_ARG;
  }
  if (a.bias && rows_meet(out, {a.bias, 1, 0, a.n * (a.bias_dtype == LM_F32 ? 4 : 2)})) return LM_ERR_INVALID_ARG;
  const bool same = a.residual == a.out && out_size == 2 && (rows == 1 || a.residual_row_stride == a.out_row_stride);
  if (a.residual && !same && rows_meet(out, {a.residual, rows, a.residual_row_stride * 2, a.n * 2}))
    return LM_ERR_INVALID_ARG;

  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool half = a.dtype == LM_F16;
  if (expands(rows, a.n, a.k)) {
    void *const to = static_cast<char *>(workspace) + first;
    if (a.k > 0) {
      const int64_t words = a.n * up(a.k, 8), ctas = up(words, 256);
      if (ctas > INT_MAX) return LM_ERR_UNSUPPORTED;
      const dim3 grid(static_cast<unsigned>(ctas));
      if (lm_status st = half ? launch_dependent(values_kernel<__half, true>, grid, 256, 0, s, 1, w,
                                                 static_cast<__half *>(to), up(a.k, 8) * 8, words)
                              : launch_dependent(values_kernel<__nv_bfloat16, true>, grid, 256, 0, s, 1, w,
                                                 static_cast<__nv_bfloat16 *>(to), up(a.k, 8) * 8, words);
          st != LM_OK)
        return st;
    }
    const lm_linear_args e = expanded(a, to);
    return lm_linear(&e, workspace, first, stream);
  }
  if (x.pack)
    if (lm_status st = pack(&x, a.k, static_cast<char *>(workspace) + 256, s); st != LM_OK) return st;
  ProductParams p = {};
  p.w = w;
  p.x = x.p;
  p.bias = a.bias;
  p.residual = a.residual;
  p.out = a.out;
  p.rows = static_cast<int32_t>(rows);
  p.group_rows = static_cast<int32_t>(x.rows);
  p.x_group = x.group_stride;
  p.x_row = x.row_stride;
  p.res_row = a.residual_row_stride;
  p.out_row = a.out_row_stride;
  p.ntiles = static_cast<int32_t>(up(a.n, 16));
  p.bias_f32 = a.bias_dtype == LM_F32;
  p.out_f32 = a.out_dtype == LM_F32;
  p.act = a.activation;
  p.scale = a.scale;
  DeviceInfo dev;
  if (lm_status st = current_device_info(&dev); st != LM_OK) return st;
  return half ? product<__half>(p, dev.sm_count, s) : product<__nv_bfloat16>(p, dev.sm_count, s);
}
