// linear4.cu -- weights of 4 bits with group scales: their layout, rounding and values, and
// y = residual + scale * act(x W^T + bias) with such a weight.
//
// Few rows of x: the weight's bytes bound the call.  They are laid out so that a lane's 16 bytes of
// a tile are its operands of four m16n8k16 products with W as the 16 rows, and 16 bytes of x twice the
// other operand: neither goes through shared memory, and a nibble becomes a 16-bit float by an OR into
// the mantissa of 1024 (f16) or 128 (bf16) and an exact subtraction.  (For tcgen05 a converted operand has to be
// written to shared or tensor memory first.)  A warp sums a tile of 16 outputs over a part of
// k, a group's products in 32 bits and then times its scale; the warps of a CTA share out tiles and
// k, meet in shared memory, and write whole lines.
//
// More rows: linear.cu's tiles on tcgen05, with warps that widen W's bytes into the operand, rounded to x's
// type.  Many rows: the values are expanded into the workspace, and linear.cu's kernel takes them.
//
// Measured, in a graph: 5 x 1024 -> 4096 3.3 us; 5 x 1024 -> 50001 10.6 us for 28.8 MB (2.7 TB/s; issue slots 55% full, a
// hundred instructions a tile), 16 rows 17; 128 rows 18.6 to 20 (16-bit weights: 320 rows 31); 320 x 4096 -> 1024 11.5;
// 3000 x 1024 -> 4096 22.6, of which the expansion is 3.
#include <climits>
#include <type_traits>

#include "activate.cuh"
#include "half.cuh"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "mma.cuh"
#include "operand.cuh"
#include "pdl.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "waits.cuh"

namespace lm {
namespace {

constexpr int kTileBytes = 512;    // 16 rows by 64 k
constexpr int kBlockBytes = 4096;  // eight of them: 128 rows by 64 k

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
  return ((i / 128 * w.ktiles + j / 64) * 8 + i % 128 / 16) * (kTileBytes / 4) + (r % 8 * 4 + c % 32 / 8) * 4 + r / 8 * 2 +
         c / 32;
}

__device__ __forceinline__ int64_t scale_at(const Weight &w, int64_t i, int64_t g) {
  return (i / 128 * w.groups + g) * 128 + i % 128;
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
  int64_t x_group, x_row, res_row, out_row;
  int32_t rows, group_rows, ntiles, parts;  // parts: warps that share out a tile's k
  int32_t group_tiles;  // log2 of a group's tiles of k
  int32_t bias_f32, out_f32, act;
  float scale;
};

constexpr int kMostWarps = 16;  // of a CTA
constexpr int kSide = 2;  // tiles of 16 outputs that a warp works on

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

__device__ __forceinline__ void sts_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Eight elements of a row from k on, zeros past its end.
template <typename T>
__device__ __forceinline__ uint4 load8(const T *row, int k, int end) {
  if (k + 8 <= end) return *reinterpret_cast<const uint4 *>(row + k);
  uint32_t v[4] = {0, 0, 0, 0};
  if (k < end) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k + j < end) v[j / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(row + k + j)) << (16 * (j % 2));
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// One output element.
template <typename T>
__device__ __forceinline__ void put_any(const ProductParams &p, float s, int row, int n) {
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
// A warp has two tiles of 16 outputs side by side, which share its operands of x and give it products
// that do not wait for one another.
// MOST: warps of a CTA, at most; with 8 the registers are held to what lets three such CTAs share an SM.
template <typename T, int NT, bool SMALL, int MOST>
__global__ void __launch_bounds__(32 * MOST, MOST == 8 ? (NT == 1 ? 3 : 2) : 1) product_kernel(const ProductParams p) {
  constexpr int SCALES = SMALL ? 2 : 1;
  constexpr int PITCH = 16 * kSide + 1;
  extern __shared__ float sums[];  // [warps][8 * NT][PITCH]
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, r = lane / 4, c = lane % 4;
  const int part = warp % p.parts, per = static_cast<int>(blockDim.x) / 32 / p.parts;
  const int tile = (static_cast<int>(blockIdx.x) * per + warp / p.parts) * kSide;
  const int row0 = static_cast<int>(blockIdx.y) * 8 * NT, k = static_cast<int>(p.w.k);
  const bool any = tile < p.ntiles;
  const int begin = any ? static_cast<int>(static_cast<int64_t>(p.w.ktiles) * part / p.parts) : 0;
  const int end = any ? static_cast<int>(static_cast<int64_t>(p.w.ktiles) * (part + 1) / p.parts) : 0;
  pdl_launch();
  pdl_wait();
  // (A row past the last reads the first; its sums are not written.)
  const uint32_t *const packed =
      p.w.packed + (static_cast<int64_t>(tile / 8) * p.w.ktiles * 8 + tile % 8) * (kTileBytes / 4) + lane * 4;
  const float *const scales = p.w.scale + static_cast<int64_t>(tile / 8) * p.w.groups * 128 + tile % 8 * 16 + r;
  const T *x[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = row0 + 8 * t + r < p.rows ? row0 + 8 * t + r : row0;
    x[t] = static_cast<const T *>(p.x) + row / p.group_rows * p.x_group + row % p.group_rows * p.x_row + 8 * c;
  }
  float total[NT][kSide][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < kSide; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) total[t][m][j] = 0.0f;

  uint4 w[2][kSide], b[2][NT][2];
  float s[2][kSide][SCALES][2];
  auto fetch = [&](int u, int kt) {
#pragma unroll
    for (int m = 0; m < kSide; ++m) {
      w[u][m] = load_once(packed + m * (kTileBytes / 4) + static_cast<int64_t>(kt) * (kBlockBytes / 4));
#pragma unroll
      for (int h = 0; h < SCALES; ++h) {
        int g = SMALL ? 2 * kt + h : kt >> p.group_tiles;
        if (SMALL && g >= p.w.groups) g = p.w.groups - 1;  // (its half of the tile is zeros)
        const float *const at = scales + m * 16 + static_cast<int64_t>(g) * 128;
        s[u][m][h][0] = at[0];
        s[u][m][h][1] = at[8];
      }
    }
    if ((kt + 1) * 64 <= k) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) b[u][t][h] = *reinterpret_cast<const uint4 *>(x[t] + kt * 64 + 32 * h);
    } else {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) b[u][t][h] = load8<T>(x[t] - 8 * c, kt * 64 + 32 * h + 8 * c, k);
    }
  };
  auto multiply = [&](int u) {
#pragma unroll
    for (int m = 0; m < kSide; ++m) {
      uint32_t v[4][4];  // words: row r, the tile's first and second half of k; row r + 8
      widen<T>(w[u][m].x, v[0]);
      widen<T>(w[u][m].y, v[1]);
      widen<T>(w[u][m].z, v[2]);
      widen<T>(w[u][m].w, v[3]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 &o = b[u][t][h];
          const uint32_t a0[4] = {v[h][0], v[h + 2][0], v[h][1], v[h + 2][1]};
          const uint32_t a1[4] = {v[h][2], v[h + 2][2], v[h][3], v[h + 2][3]};
          mma16816<T>(d, a0, o.x, o.y);
          mma16816<T>(d, a1, o.z, o.w);
          if (SMALL || h == 1) {
            const float *const f = s[u][m][SMALL ? h : 0];
            total[t][m][0] = fmaf(f[0], d[0], total[t][m][0]);
            total[t][m][1] = fmaf(f[0], d[1], total[t][m][1]);
            total[t][m][2] = fmaf(f[1], d[2], total[t][m][2]);
            total[t][m][3] = fmaf(f[1], d[3], total[t][m][3]);
            d[0] = d[1] = d[2] = d[3] = 0.0f;
          }
        }
      }
    }
  };
  // Two tiles on their way.
  if (begin < end) fetch(0, begin);
  if (begin + 1 < end) fetch(1, begin + 1);
#pragma unroll 1
  for (int kt = begin; kt < end; kt += 2) {
    multiply(0);
    if (kt + 2 < end) fetch(0, kt + 2);
    if (kt + 1 < end) {
      multiply(1);
      if (kt + 3 < end) fetch(1, kt + 3);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < kSide; ++m) {
      float *const to = sums + (warp * 8 * NT + 8 * t + 2 * c) * PITCH + 16 * m + r;
      to[0] = total[t][m][0];
      to[PITCH] = total[t][m][1];
      to[8] = total[t][m][2];
      to[PITCH + 8] = total[t][m][3];
    }
  __syncthreads();
  constexpr int WIDE = 16 * kSide;
  const int wide = WIDE * per, rows = min(8 * NT, p.rows - row0);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * wide;
  for (int i = threadIdx.x; i < rows * wide; i += blockDim.x) {
    const int row = i / wide, at = i % wide;
    if (n0 + at >= p.w.n) continue;
    float sum = 0.0f;
    for (int q = 0; q < p.parts; ++q) sum += sums[((at / WIDE * p.parts + q) * 8 * NT + row) * PITCH + at % WIDE];
    put_any<T>(p, sum, row0 + row, static_cast<int>(n0) + at);
  }
}

// ---- more rows: tcgen05 ----

constexpr int kMaxStages = 8, kMaxRaw = 4;
constexpr int kChunk = 4;                       // blocks of k that are fetched at once
constexpr int kSlotBytes = kChunk * (kBlockBytes + 1024);  // their packed bytes, then their scales
constexpr int kWiden = 8, kEpilogue = 8;        // warps
constexpr int kThreads = 32 * (4 + kWiden + kEpilogue);

struct TileParams {
  LinearParams l;
  const uint8_t *packed;
  const float *scale;
  int32_t groups, small, group_tiles, raw;
};

__device__ uint32_t g_linear4_error;

struct alignas(16) Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t raw_full[kMaxRaw], raw_empty[kMaxRaw];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
};

// The group that block kb of k starts with.
__device__ __forceinline__ int group_at(const TileParams &p, int kb) { return p.small ? 2 * kb : kb >> p.group_tiles; }

// A ring's position.
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n, int by = 1) {
    at += by;
    if (at >= n) {
      at -= n;
      phase ^= 1;
    }
  }
};

// The eight values of a word: whole numbers times the scale in 32 bits, rounded once (as lm_weight4_values).
template <typename T>
__device__ __forceinline__ void widen_scaled(uint32_t word, float s, uint32_t (&v)[4]) {
  widen<T>(word, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = unpack2<T>(v[i]);
    v[i] = pack2<T>(q.x * s, q.y * s);
  }
}

// The values of all blocks in rows of `pitch` (a multiple of 8) elements, zeros past k: a warp a tile of 16 rows,
// a lane four vectors of 16 bytes.
template <typename T>
__global__ void __launch_bounds__(256) expand_kernel(const Weight w, T *out, int pitch) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
  const int64_t block = blockIdx.y;
  const int kb = blockIdx.x, small = w.group == 32 ? 1 : 0;
  const int g = small ? 2 * kb : kb * 64 / w.group;
  pdl_launch();
  pdl_wait();
  const uint4 v = load_once(w.packed + ((block * w.ktiles + kb) * 8 + warp) * (kTileBytes / 4) + lane * 4);
  const float *const s = w.scale + (block * w.groups + g) * 128 + 16 * warp + r;
  const bool there = !small || g + 1 < w.groups;
  const int j = kb * 64 + 8 * c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = block * 128 + 16 * warp + r + 8 * h;
    if (row >= w.n) break;
    uint32_t x[4];
    T *const to = out + row * pitch + j;
    widen_scaled<T>(h ? v.z : v.x, s[8 * h], x);
    if (j < pitch) *reinterpret_cast<uint4 *>(to) = make_uint4(x[0], x[1], x[2], x[3]);
    widen_scaled<T>(h ? v.w : v.y, there ? s[8 * h + 128 * small] : 0.0f, x);
    if (j + 32 < pitch) *reinterpret_cast<uint4 *>(to + 32) = make_uint4(x[0], x[1], x[2], x[3]);
  }
}

// A scale as two 16-bit floats, twice each: its rounded value and what that leaves off.
template <typename T>
struct Scale {
  uint32_t high, low;
};

// Both of a number, rounded; of bf16 at most its largest value.
template <typename T>
__device__ __forceinline__ uint32_t first_part(float s) {
  if (std::is_same<T, __half>::value) return pack2<T>(s, s);
  uint32_t r;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %1;" : "=r"(r) : "f"(s));
  return r;
}

template <typename T>
__device__ __forceinline__ Scale<T> split_scale(float s) {
  Scale<T> o;
  o.high = first_part<T>(s);
  const float low = s - unpack2<T>(o.high).x;
  o.low = pack2<T>(low, low);
  return o;
}

// Whether the parts stand for the scale.  Those of f16 do up to its largest value (past it the second may be infinite, and
// 0 times it NaN) and, because its steps end at 2^-24, down to 2^-10 (see widen_scaled).  Those of bf16 always do: a
// finite scale leaves a finite second part, an infinite one an infinite, and 0 times the scale is 0 or NaN.
template <typename T>
__device__ __forceinline__ bool splits(float s) {
  const float a = fabsf(s);
  return !std::is_same<T, __half>::value || (a >= 0x1p-10f && a <= 65504.0f);
}

__device__ __forceinline__ __half2 as2(uint32_t v, __half) { return *reinterpret_cast<const __half2 *>(&v); }
__device__ __forceinline__ __nv_bfloat162 as2(uint32_t v, __nv_bfloat16) {
  return *reinterpret_cast<const __nv_bfloat162 *>(&v);
}
// The eight values of a word, two instructions a pair: q * high + (q * low rounded), rounded once.  In bf16 the
// parts lose 2^-17 of the value, 2^-8 of the last rounding; in f16, whose least step is 2^-24, 8 * 2^-25 for scales
// down to 2^-10, a sixteenth of it (other scales go through 32 bits).
template <typename T>
__device__ __forceinline__ void widen_scaled(uint32_t word, const Scale<T> &s, uint32_t (&v)[4]) {
  widen<T>(word, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto q = as2(v[i], T()), y = __hfma2(q, as2(s.high, T()), __hmul2(q, as2(s.low, T())));
    v[i] = *reinterpret_cast<const uint32_t *>(&y);
  }
}

// ... by whichever way is the scale's.
template <typename T>
__device__ __forceinline__ void widen_any(uint32_t word, float s, uint32_t (&v)[4]) {
  if (splits<T>(s)) {
    widen_scaled<T>(word, split_scale<T>(s), v);
  } else {
    widen_scaled<T>(word, s, v);
  }
}

// TILES tiles of 16 rows of a block into the operand at `to`.
template <typename T, int TILES>
__device__ __forceinline__ void widen_stage(const uint8_t *slot, const float *scales, int other, bool there, uint32_t to,
                                            uint32_t low, uint32_t high, bool odd, int lane) {
  // (Odd rows' halves change places here.)
  uint4 v[TILES];
  float f[TILES][2][2];
  bool parts = true;
#pragma unroll
  for (int j = 0; j < TILES; ++j) {
    const uint4 u = reinterpret_cast<const uint4 *>(slot + j * kTileBytes)[lane];
    v[j] = odd ? make_uint4(u.y, u.x, u.w, u.z) : u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float first = scales[16 * j + 8 * h], second = there ? scales[other + 16 * j + 8 * h] : 0.0f;
      f[j][h][0] = odd ? second : first;
      f[j][h][1] = odd ? first : second;
      parts = parts && splits<T>(f[j][h][0]) && splits<T>(f[j][h][1]);
    }
  }
  if (std::is_same<T, __half>::value && !__all_sync(0xffffffffu, parts)) {  // a warp's other rows get the same bits either way
#pragma unroll 1
    for (int h = 0; h < 2 * TILES; ++h) {
      const uint4 u = reinterpret_cast<const uint4 *>(slot + h / 2 * kTileBytes)[lane];
      const float first = scales[8 * h], second = there ? scales[other + 8 * h] : 0.0f;
      uint32_t x[4], y[4];
      widen_any<T>(h % 2 ? u.z : u.x, first, x);
      widen_any<T>(h % 2 ? u.w : u.y, second, y);
      const uint32_t at = to + h * 1024;
      sts_v4(at + (odd ? high : low), x[0], x[1], x[2], x[3]);
      sts_v4(at + (odd ? low : high), y[0], y[1], y[2], y[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // rows r and r + 8
        uint32_t x[4];
        const uint32_t at = to + j * 2048 + h * 1024;
        widen_scaled<T>(h ? v[j].z : v[j].x, split_scale<T>(f[j][h][0]), x);
        sts_v4(at + low, x[0], x[1], x[2], x[3]);
        widen_scaled<T>(h ? v[j].w : v[j].y, split_scale<T>(f[j][h][1]), x);
        sts_v4(at + high, x[0], x[1], x[2], x[3]);
      }
    }
  }
}

// linear.cu's kernel (a CTA a tile, or a cluster that shares out k), but for W's tiles: bulk copies bring their packed
// bytes and scales, and eight warps turn them into the operand's swizzled layout.
//
// A stage's way through a warp takes several hundred cycles of waiting for one another, so that GROUPS groups
// of warps widen as many stages at once, in turn.  A wait tells whether the phase before was the last to
// end, not which one it was; a group's own last fill shows that what came as many fills before as there are stages
// has been used, which is enough where there are no more groups than stages.
//
// KB: blocks of k of a stage.  With two the waits for barriers come half as often (64 x 1024 -> 50001 17.9 us, with
// one 19.5; 64 x 4096 -> 8192 16.0, 16.8; nowhere slower); from 128 columns of x on there would be room for two
// stages, too few.  (Of 19.5 us the copies, barriers and three rounds of tiles alone took 13.4, the widening 4.)
template <typename T, bool SPLIT, int GROUPS, int KB>
__global__ void __launch_bounds__(kThreads, 1) tile_kernel(const __grid_constant__ CUtensorMap col_map, const TileParams tp) {
  constexpr int GROUP_WARPS = kWiden / GROUPS, TILES = KB * 8 / GROUP_WARPS;
  static_assert(8 % TILES == 0 && kChunk % KB == 0, "a warp's tiles are of one block, a chunk's stages its own");
  const LinearParams &p = tp.l;
  extern __shared__ __align__(1024) uint8_t ring[];
  const int block_bytes = kLanes * 128 + p.bn * 128, stage_bytes = KB * block_bytes;  // a block: W's tile, then x's
  uint8_t *const raw = ring + p.stages * stage_bytes;
  Barriers &b = *reinterpret_cast<Barriers *>(raw + tp.raw * kSlotBytes);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0), lane = threadIdx.x % 32;
  const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = SPLIT ? static_cast<int>(blockIdx.x) / p.splits : static_cast<int>(blockIdx.x);
  const int step = SPLIT ? p.tiles : static_cast<int>(gridDim.x);
  const int k_begin = SPLIT ? static_cast<int>(static_cast<int64_t>(p.kblocks) * rank / p.splits) : 0;
  const int k_end = SPLIT ? static_cast<int>(static_cast<int64_t>(p.kblocks) * (rank + 1) / p.splits) : p.kblocks;

  // (By many threads: one thread took a microsecond for all of them.)
  if (warp == 0) {
    if (lane < p.stages) {
      mbar_init(&b.full[lane], 1 + GROUP_WARPS + (lane == 0 && static_cast<int>(blockIdx.x) == p.withheld ? 1 : 0));
      mbar_init(&b.empty[lane], 1);
    }
    if (lane < tp.raw) {
      mbar_init(&b.raw_full[lane], 1);
      mbar_init(&b.raw_empty[lane], kWiden);
    }
    if (lane < 2) {
      mbar_init(&b.acc_full[lane], 1);
      mbar_init(&b.acc_empty[lane], kEpilogue);
    }
    if (lane == 0) {
      mbar_init(&b.drain, 1);
      b.abort = 0;
      tma_prefetch_map(&col_map);
    }
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc<false>(&b.tmem, static_cast<uint32_t>(p.tmem_cols));
  tcgen05_fence_before();
  __syncthreads();
  __syncwarp();
  pdl_launch();
  pdl_wait();
  tcgen05_fence_after();
  const uint32_t tmem = b.tmem;
  volatile int *const abort = &b.abort;

  if (warp == 0) {  // tiles of x
    Ring s;
    int fills = 0;
    bool ok = true;
    for (int t = first; t < p.tiles && ok; t += step) {
      const Tile tile = tile_at(p, t, 0);
      for (int kb = k_begin; kb < k_end; kb += KB) {
        if (fills >= p.stages) ok = mbar_wait_warp(&b.empty[s.at], s.phase ^ 1, p.wait_ns, abort, p.err);
        if (!ok) break;
        if (elect_one()) {
          const int count = min(KB, k_end - kb);
          mbar_arrive_expect_tx(&b.full[s.at], static_cast<uint32_t>(count * p.bn * 128));
          for (int i = 0; i < count; ++i)
            tma_load_3d<false>(ring + s.at * stage_bytes + i * block_bytes + kLanes * 128, &col_map, (kb + i) * kBk,
                               tile.col0, tile.group, smem_u32(&b.full[s.at]));
        }
        __syncwarp();
        ++fills;
        s.next(p.stages);
      }
    }
    // No copy outlives the CTA, whatever the other warps did.
    for (int f = fills > p.stages ? fills - p.stages : 0; f < fills; ++f)
      if (!mbar_drain(&b.full[f % p.stages], (f / p.stages) & 1, p.wait_ns, p.err)) break;
  } else if (warp == 3) {  // packed bytes and scales, several blocks at once: issuing a copy takes some 200 cycles
    Ring s;
    int fills = 0;
    bool ok = true;
    for (int t = first; t < p.tiles && ok; t += step) {
      const int64_t block = tile_at(p, t, 0).lane0 / kLanes;
      const uint8_t *const bytes = tp.packed + block * p.kblocks * kBlockBytes;
      const float *const scales = tp.scale + block * tp.groups * kLanes;
      for (int kb = k_begin; kb < k_end; kb += kChunk) {
        if (fills >= tp.raw) ok = mbar_wait_warp(&b.raw_empty[s.at], s.phase ^ 1, p.wait_ns, abort, p.err);
        if (!ok) break;
        if (elect_one()) {
          const int end = min(kb + kChunk, k_end), g = group_at(tp, kb);
          const int g_end = min(group_at(tp, end - 1) + 1 + tp.small, tp.groups);
          const uint32_t size = static_cast<uint32_t>(end - kb) * kBlockBytes, factors = static_cast<uint32_t>(g_end - g) * 512;
          uint8_t *const to = raw + s.at * kSlotBytes;
          mbar_arrive_expect_tx(&b.raw_full[s.at], size + factors);
          bulk_g2s_plain(to, bytes + static_cast<int64_t>(kb) * kBlockBytes, size, &b.raw_full[s.at]);
          bulk_g2s_plain(to + kChunk * kBlockBytes, scales + static_cast<int64_t>(g) * kLanes, factors, &b.raw_full[s.at]);
        }
        __syncwarp();
        ++fills;
        s.next(tp.raw);
      }
    }
    for (int f = fills > tp.raw ? fills - tp.raw : 0; f < fills; ++f)
      if (!mbar_drain(&b.raw_full[f % tp.raw], (f / tp.raw) & 1, p.wait_ns, p.err)) break;
  } else if (warp == 1) {  // products
    Ring s;
    int tiles = 0;
    bool ok = true;
    const uint32_t ring_a = smem_u32(ring);
    for (int t = first; t < p.tiles && ok; t += step, ++tiles) {
      const int half = tiles & 1;
      if (tiles >= 2) ok = mbar_wait_warp(&b.acc_empty[half], ((tiles >> 1) - 1) & 1, p.wait_ns, abort, p.err);
      tcgen05_fence_after();
      const uint32_t d = tmem + static_cast<uint32_t>(half * (p.tmem_cols / 2));
      for (int kb = k_begin; kb < k_end && ok; kb += KB) {
        ok = mbar_wait_warp(&b.full[s.at], s.phase, p.wait_ns, abort, p.err);
        if (!ok) break;
        tcgen05_fence_after();
        const uint64_t a = smem_desc_k128(ring_a + s.at * stage_bytes);
        const uint64_t c = smem_desc_k128(ring_a + s.at * stage_bytes + kLanes * 128);
        const bool second = KB == 2 && kb + 1 < k_end;
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kBk / 16; ++i)
            tcgen05_mma_f16<false>(d, a + 2 * i, c + 2 * i, p.idesc, kb > k_begin || i > 0);
          if (second) {
            const uint64_t next = static_cast<uint64_t>(block_bytes >> 4);
#pragma unroll
            for (int i = 0; i < kBk / 16; ++i)
              tcgen05_mma_f16<false>(d, a + next + 2 * i, c + next + 2 * i, p.idesc, true);
          }
          tcgen05_commit<false>(&b.empty[s.at]);
        }
        __syncwarp();
        s.next(p.stages);
      }
      if (ok && elect_one()) tcgen05_commit<false>(&b.acc_full[half]);
      __syncwarp();
    }
    if (!ok) {  // products in flight end before the tensor memory is given back
      if (elect_one()) tcgen05_commit<false>(&b.drain);
      mbar_drain(&b.drain, 0, p.wait_ns, p.err);
    }
  } else if (warp >= 4 && warp < 4 + kWiden) {
    // Of a tile of 16 rows lane 4 r + c has rows r and r + 8 at k 8 c .. + 7 and 32 + 8 c .. + 7, chunks c
    // and 4 + c of 16 bytes in a row of 128.  Odd rows store their second chunk first: eight lanes then
    // meet every bank once.
    const int e = warp - 4, group = e / GROUP_WARPS, r = lane / 4, c = lane % 4, odd = r & 1;
    const int tile0 = e % GROUP_WARPS * TILES % 8, block = e % GROUP_WARPS * TILES / 8;  // of the stage's
    const uint32_t low = static_cast<uint32_t>((16 * tile0 + r) * 128 + (((odd ? 4 + c : c) ^ r) * 16));
    const uint32_t high = static_cast<uint32_t>((16 * tile0 + r) * 128 + (((odd ? c : 4 + c) ^ r) * 16));
    const uint32_t ring_a = smem_u32(ring);
    // Every warp waits for every chunk of blocks and gives it back; the stages are the groups' in turn.
    Ring s, q;
    s.next(p.stages, group);
    int fill = 0;
    bool ok = true;
    for (int t = first; t < p.tiles && ok; t += step)
      for (int chunk = k_begin; chunk < k_end && ok; chunk += kChunk) {
        ok = mbar_wait_warp(&b.raw_full[q.at], q.phase, p.wait_ns, abort, p.err);
        const int end = min(chunk + kChunk, k_end);
        for (int first_kb = chunk; first_kb < end && ok; first_kb += KB, ++fill) {
          if (fill % GROUPS != group) continue;
          const int kb = first_kb + block;
          const uint8_t *const slot = raw + q.at * kSlotBytes + (kb - chunk) * kBlockBytes;
          const int g = group_at(tp, kb) - group_at(tp, chunk);
          const float *const scales =
              reinterpret_cast<const float *>(raw + q.at * kSlotBytes + kChunk * kBlockBytes) + g * kLanes + 16 * tile0 + r;
          // A second group that the block lacks has zeros for numbers, whatever lies in its scales' place.
          const int other = tp.small ? kLanes : 0;
          const bool there = !tp.small || 2 * kb + 1 < tp.groups;
          if (fill >= p.stages) ok = mbar_wait_warp(&b.empty[s.at], s.phase ^ 1, p.wait_ns, abort, p.err);
          if (!ok) break;
          if (kb < end)  // (a last stage may have one block)
            widen_stage<T, TILES>(slot + tile0 * kTileBytes, scales, other, there,
                                  ring_a + s.at * stage_bytes + block * block_bytes, low, high, odd, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b.full[s.at]);
          s.next(p.stages, GROUPS);
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&b.raw_empty[q.at]);
        q.next(tp.raw);
      }
  } else if (warp >= 4 + kWiden) {
    const int e = warp - 4 - kWiden;
    int tiles = 0;
    for (int t = first; t < p.tiles; t += step, ++tiles) {
      const Tile tile = tile_at(p, t, 0);
      const int half = tiles & 1;
      T residual[16];
      if (!SPLIT && p.residual) {
#pragma unroll
        for (int j = 0; j < 16; ++j) residual[j] = from_f32<T>(0.0f);
        const int c = e / 4 * 16, cols = min(p.bn, p.rows - tile.col0);
        if (c < cols)
          residual_rows<T>(p, residual, static_cast<int64_t>(tile.group) * p.rows + tile.col0 + c, min(16, cols - c),
                           tile.lane0 + 32 * (e % 4) + lane);
      }
      // One decision per warp: tensor memory loads are executed by whole warps.
      if (!mbar_wait_warp(&b.acc_full[half], (tiles >> 1) & 1, p.wait_ns, abort, p.err)) break;
      tcgen05_fence_after();
      const uint32_t acc = tmem + static_cast<uint32_t>(half * (p.tmem_cols / 2));
      if (SPLIT) {
        // Products are complete: the ring is free to hold the partial sums.
        float *const partial = reinterpret_cast<float *>(ring);
        for (int c = e / 4 * 16; c < p.bn; c += 4 * kEpilogue) {
          uint32_t r[16];
          tmem_ld16(acc + (static_cast<uint32_t>(32 * (e % 4)) << 16) + c, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) partial[(c + j) * kLanes + 32 * (e % 4) + lane] = __uint_as_float(r[j]);
        }
      } else {
        if (p.residual) {
          epilogue_act<T, true, kEpilogue>(p, tile, acc, e, residual);
        } else {
          epilogue_act<T, false, kEpilogue>(p, tile, acc, e, residual);
        }
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.acc_empty[half]);
      }
    }
  }

  __syncwarp();
  if (SPLIT) {
    __syncthreads();
    cluster_sync_all();
    if (!*abort && first < p.tiles)
      finish_split_act<T>(p, tile_at(p, first, 0), smem_u32(ring), rank, threadIdx.x, kThreads);
    cluster_sync_all();  // no CTA leaves while another reads its sums
  }
  tcgen05_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort) atomicOr(&g_linear4_error, kErrMbarTimeout);
  if (warp == 2) {
    tcgen05_fence_after();
    tmem_dealloc<false>(tmem, static_cast<uint32_t>(p.tmem_cols));
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

// Whether the warps' products take a call: up to 16 rows read the weight once, more read it from L2 for every 16
// (32 rows x 1024 -> 4096: 4.5 us, 6.7 on tcgen05; 64 x 4096 -> 1024: 5.6, 7.9; 32 x 2048 -> 6000 9.3, 11.6; 64 x 1024 ->
// 4096 6.7, 7.5; but 48 x 2048 -> 4096 9.1, 8.1, 64 x 1024 -> 6000 10.0, 7.6 and 32 x 1024 -> 50001 29, 18).
bool few(int64_t rows, int64_t n, int64_t k) {
  return rows <= 16 || (rows <= 64 && up(rows, 16) * n <= (k <= 1024 ? 16384 : 12000));
}

// From this many rows on the products cost more than expanding the weight.  (us, tiles and expanded: 768 rows x 1024 -> 4096
// 9.7, 11.3, 3000 rows 24.1, 20.8; 4096 -> 4096 23.9, 23.9 and 74.6, 59.3; 2048 -> 8192 24.7, 23.7 and 77.8, 60.4; 1024 ->
// 50001 60.3, 71.3 and 234, 208.  Of nine weights seven cross between 256 and 2048 rows, whatever n and k, and the smallest,
// 512 -> 512 and 256 -> 1024, stay 2 to 12% apart.  The rule's choice is up to 18% slower than the other at 768 and 1024 rows
// (8192 -> 2048 31.5, 26.6; 1024 -> 4096 13.2, 11.3), 8% elsewhere, and 30% at 512 x 4096 -> 4096 (25.7, 19.7).)
bool expands(int64_t rows, int64_t n, int64_t) { return rows > 768 && n <= 65535 * 128; }

// ... of a weight with contents.
lm_status whole(const Weight &w) {
  if (!w.packed || !w.scale) return LM_ERR_INVALID_ARG;
  return aligned(w.packed, 16) && aligned(w.scale, 16) ? LM_OK : LM_ERR_MISALIGNED;
}

template <typename T, bool GIVEN>
lm_status fill(const Weight &w, const T *src, int64_t row_stride, const float *scales, cudaStream_t s) {
  const int64_t units = up(w.n, 128) * 128 * w.groups;
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
  const size_t blocks = static_cast<size_t>(lm::up(w.n, 128));
  *packed_bytes = blocks * static_cast<size_t>(w.ktiles) * lm::kBlockBytes;
  *scale_bytes = blocks * static_cast<size_t>(w.groups) * 512;
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

// Warps that share out the k of a pair of tiles: a warp's time is about its tiles of k and one more, times the rounds
// in which an SM's 24 warps (16 with two blocks of rows) come by.  Rounds of small CTAs overlap, so
// that they count half; a CTA of 16 warps has the SM to itself.  Within 5% of the best of all on 74 problems (k 256 to
// 4096, 512 to 50001 outputs); 16 rows x 512 -> 8192 3.8 us, with two dozen warps an SM as the rule 4.8.
int best_parts(int64_t ktiles, int64_t pairs, int nt, int sms) {
  int best = 1;
  float least = 3.0e38f;
  for (int parts = 1; parts <= kMostWarps && parts <= ktiles; parts *= 2) {
    const int64_t room = (nt == 1 && parts <= 8 ? 24ll : 16ll) * sms, warps = pairs * parts;
    const float whole = static_cast<float>(up(warps, room));
    const float share = static_cast<float>(warps) / static_cast<float>(room);
    const float rounds = parts > 8 || share < 1.0f ? whole : 0.5f * (whole + share);
    const float t = rounds * (1.0f + static_cast<float>(up(ktiles, parts)));
    if (t < least) {
      least = t;
      best = parts;
    }
  }
  return best;
}

// CTAs of four warps or, where more share out a tile's k, of those: small ones even out over the SMs.
template <typename T, int NT>
lm_status product_as(ProductParams p, int sms, cudaStream_t s) {
  const int64_t pairs = up(p.ntiles, kSide), blocks = up(p.rows, 8 * NT);
  p.parts = best_parts(p.w.ktiles, pairs * blocks, NT, sms);
  const int warps = p.parts > 4 ? p.parts : 4;
  const dim3 grid(static_cast<unsigned>(up(pairs, warps / p.parts)), static_cast<unsigned>(blocks));
  const auto kernel = warps > 8 ? (p.w.group == 32 ? product_kernel<T, NT, true, 16> : product_kernel<T, NT, false, 16>)
                                : (p.w.group == 32 ? product_kernel<T, NT, true, 8> : product_kernel<T, NT, false, 8>);
  const int shared = warps * 8 * NT * (16 * kSide + 1) * 4;
  return launch_dependent(kernel, grid, 32 * warps, static_cast<size_t>(shared), s, 1, p);
}

template <typename T>
lm_status product(const ProductParams &p, int sms, cudaStream_t s) {
  return p.rows <= 8 ? product_as<T, 1>(p, sms, s) : product_as<T, 2>(p, sms, s);
}

// How the tiles' kernel cuts a call.
struct Cut {
  int bn, splits;
  int64_t tiles;
};

// The cut with the least estimated time, in microseconds: linear.cu's model, with what a block's widening takes
// (in a cluster, too).  Of 24 problems (32 to 768 rows, k 500 to 8192, 512 to 50001 outputs) its choice is within 4% of
// the best of all cuts (500 x 1024 -> 1024 7.7 us; a cut over k 8.9).
Cut best_cut(int64_t n, int64_t rows, int64_t groups, int kblocks, bool activation, int sms, const Resident &held) {
  Cut best = {16, 1, 0};
  float least = 3.0e38f;
  const float column = activation ? 0.017f : 0.013f;
  auto consider = [&](int bn, int splits) {
    const int64_t tiles = up(n, kLanes) * up(rows, bn) * groups;
    if (splits > 1 && tiles > held.split[splits]) return;
    const int64_t rounds = up(tiles, splits > 1 ? held.split[splits] : sms);
    const float products = 0.0011f * static_cast<float>(bn);
    const float widening = splits > 1 ? 0.3f : bn <= 96 ? 0.22f : 0.25f;
    const float blocks = static_cast<float>(up(kblocks, splits)) * (products > widening ? products : widening);
    float t = 3.0f + blocks;
    t += splits > 1 ? 2.0f + 0.03f * static_cast<float>(bn) / static_cast<float>(splits) + 0.008f * static_cast<float>(bn)
                    : column * static_cast<float>(bn);
    const float epi = 0.5f + column * static_cast<float>(bn);
    t += static_cast<float>(rounds - 1) * (blocks > epi ? blocks : epi);
    if (t < least) {
      least = t;
      best = {bn, splits, tiles};
    }
  };
  const int most = rows < kMaxBn ? static_cast<int>(up(rows, 16) * 16) : kMaxBn;
  auto splits = [&](int bn) {
    for (int s = 1; s <= kMaxSplits && (s == 1 || s <= kblocks); s *= 2) consider(bn, s);
  };
  for (int bn = 16; bn <= most; bn += bn < 64 ? 16 : 32) splits(bn);
  splits(static_cast<int>(up(up(rows, up(rows, kMaxBn)), 16) * 16));
  return best;
}

template <typename T>
lm_status tiles(const lm_linear_args &a, const Weight &w, const Operand &x, const DeviceInfo &dev, void *workspace,
                const WaitFault *fault, cudaStream_t s) {
  TileParams tp = {};
  LinearParams &p = tp.l;
  tp.packed = reinterpret_cast<const uint8_t *>(w.packed);
  tp.scale = w.scale;
  tp.groups = w.groups;
  tp.small = w.group == 32;
  tp.group_tiles = w.group == 128 ? 1 : 0;
  p.bias = a.bias;
  p.residual = a.residual;
  p.out = a.out;
  p.out_row = a.out_row_stride;
  p.res_row = a.residual_row_stride;
  p.rows = static_cast<int32_t>(x.rows);
  p.n = static_cast<int32_t>(a.n);
  p.kblocks = w.ktiles;
  p.bias_f32 = a.bias_dtype == LM_F32;
  p.out_f32 = a.out_dtype == LM_F32;
  p.act = a.activation;
  p.scale = a.scale;
  p.err = static_cast<uint32_t *>(workspace);
  p.wait_ns = fault ? fault->wait_ns : kWaitTimeoutNs;
  p.withheld = fault ? static_cast<int32_t>(fault->withheld_cta) : -1;
  Resident held;
  if (lm_status st = resident_clusters(dev, &held); st != LM_OK) return st;
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const Cut cut = best_cut(a.n, x.rows, x.groups, p.kblocks, p.act > LM_ACT_RELU, dev.sm_count, held);
  if (cut.tiles > INT_MAX / 16) return LM_ERR_UNSUPPORTED;
  p.bn = cut.bn;
  p.splits = cut.splits;
  p.tiles = static_cast<int32_t>(cut.tiles);
  p.lane_step = kLanes;
  p.lane_tiles = static_cast<int32_t>(up(p.n, kLanes));
  p.col_tiles = static_cast<int32_t>(up(p.rows, p.bn));
  p.lanes_inside = 0;  // a tile of W's columns go round inside: its bytes come from L2
  p.tmem_cols = 32;
  while (p.tmem_cols < 2 * p.bn) p.tmem_cols *= 2;
  const bool two = p.bn <= 96;  // blocks a stage: see the kernel
  const int stage_bytes = (two ? 2 : 1) * (kLanes * 128 + p.bn * 128);
  const int room = 227 * 1024 - static_cast<int>(sizeof(Barriers));
  p.stages = (room - 3 * kSlotBytes) / stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  tp.raw = (room - p.stages * stage_bytes) / kSlotBytes;
  if (tp.raw > kMaxRaw) tp.raw = kMaxRaw;
  const bool four = !two && p.stages >= 4;
  if (p.stages < (four ? 4 : 2) || tp.raw < 2) return LM_ERR_UNSUPPORTED;
  p.idesc = idesc_f16(bf16, kLanes, static_cast<uint32_t>(p.bn));
  CUtensorMap cols = {};
  if (lm_status st = make_map(&cols, x, a.k, p.bn, bf16); st != LM_OK) return st;
  const int smem = p.stages * stage_bytes + tp.raw * kSlotBytes + static_cast<int>(sizeof(Barriers));
  const bool split = p.splits > 1;
  const auto kernel = split ? (two    ? tile_kernel<T, true, 2, 2>
                               : four ? tile_kernel<T, true, 4, 1>
                                      : tile_kernel<T, true, 2, 1>)
                            : (two    ? tile_kernel<T, false, 2, 2>
                               : four ? tile_kernel<T, false, 4, 1>
                                      : tile_kernel<T, false, 2, 1>);
  if (lm_status st = ensure_smem_attribute(reinterpret_cast<const void *>(kernel), smem); st != LM_OK) return st;
  const int grid = split ? p.tiles * p.splits : p.tiles < dev.sm_count ? p.tiles : dev.sm_count;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(grid)), kThreads, static_cast<size_t>(smem), s,
                          split ? p.splits : 1, cols, tp);
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

namespace lm {
namespace {

lm_status run(const lm_linear_args *args, const lm_weight4 *weight, void *workspace, size_t workspace_bytes,
              lm_stream_t stream, const WaitFault *fault) {
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
      if (up(a.n, 128) > 65535) return LM_ERR_UNSUPPORTED;
      const dim3 grid(static_cast<unsigned>(w.ktiles), static_cast<unsigned>(up(a.n, 128)));
      const int pitch = static_cast<int>(up(a.k, 8) * 8);
      if (lm_status st = half ? launch_dependent(expand_kernel<__half>, grid, 256, 0, s, 1, w, static_cast<__half *>(to), pitch)
                              : launch_dependent(expand_kernel<__nv_bfloat16>, grid, 256, 0, s, 1, w,
                                                 static_cast<__nv_bfloat16 *>(to), pitch);
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
  p.group_tiles = w.group == 128 ? 1 : 0;
  p.bias_f32 = a.bias_dtype == LM_F32;
  p.out_f32 = a.out_dtype == LM_F32;
  p.act = a.activation;
  p.scale = a.scale;
  DeviceInfo dev;
  if (lm_status st = current_device_info(&dev); st != LM_OK) return st;
  if (few(rows, a.n, a.k) || a.k == 0)
    return half ? product<__half>(p, dev.sm_count, s) : product<__nv_bfloat16>(p, dev.sm_count, s);
  return half ? tiles<__half>(a, w, x, dev, workspace, fault, s) : tiles<__nv_bfloat16>(a, w, x, dev, workspace, fault, s);
}

}  // namespace

lm_status linear4_error(uint32_t *value, bool clear, cudaStream_t s) { return read_sticky(g_linear4_error, value, clear, s); }

}  // namespace lm

extern "C" lm_status lm_linear4(const lm_linear_args *args, const lm_weight4 *weight, void *workspace,
                                size_t workspace_bytes, lm_stream_t stream) {
  return lm::run(args, weight, workspace, workspace_bytes, stream, nullptr);
}

extern "C" lm_status lm_debug_linear4_withhold(const lm_linear_args *args, const lm_weight4 *weight, void *workspace,
                                               size_t workspace_bytes, int64_t withheld_cta, uint64_t wait_ns,
                                               lm_stream_t stream) {
  if (withheld_cta < 0 || withheld_cta > INT_MAX || wait_ns < 100000ull || wait_ns > lm::kWaitTimeoutNs)
    return LM_ERR_INVALID_ARG;
  const lm::WaitFault fault{withheld_cta, wait_ns};
  return lm::run(args, weight, workspace, workspace_bytes, stream, &fault);
}
