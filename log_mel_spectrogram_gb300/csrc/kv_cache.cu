// kv_cache.cu -- the 8-bit key/value cache: quantising tokens into blocks,
// reading them back, and letting the block tables follow a beam step.
//
// A block of `block` tokens of one head is one contiguous tile of
// block * head_dim bytes with one scale.  One "unit" below is such a tile of
// keys or of values: block * head_dim / 64 threads work on it, 64 elements
// (eight 8-element vectors) each, so that a unit's new tokens stay in
// registers between the maximum and the rounding and are read once.
//
// Measured: 64 rows of up to 1500 tokens, 16 heads of 64, with their values
// read back, 131 us (6.3 TB/s, 94% of copy bandwidth).  One token of 320 rows,
// values read back, 13.8 us against 9.1 of traffic: length, table and scale are
// loads that wait for one another, in two rounds of CTAs.
#include <climits>

#include "half.cuh"
#include "internal.h"
#include "kv_cache.cuh"
#include "pdl.cuh"
#include "ptx.cuh"

namespace lm {

namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;  // 8-element vectors per thread

struct AppendParams {
  KvView c;
  const void *src[2];            // k, v
  int64_t row_s[2], tok_s[2], head_s[2];
  void *values[2];
  const int32_t *counts;
  int32_t tokens, spans;         // spans: blocks per row that a step can touch
  uint32_t units;                // rows * spans * heads
  bool vec;                      // 16-byte loads of src are aligned
};

// Eight signed bytes as f32: with the sign bit flipped a byte is b + 128, and
// 0x4b000000 | that is 2^23 + 128 + b.  (Conversion instructions run at an
// eighth of this rate.)
__device__ __forceinline__ void bytes_to_f32(uint2 w, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u = (j < 4 ? w.x : w.y) ^ 0x80808080u;
    x[j] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + (j & 3))) - 8388736.0f;
  }
}

// The largest |x| of two packed values and an earlier result; NaN stays NaN.
template <typename T>
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t w);
template <>
__device__ __forceinline__ uint32_t max_abs2<__half>(uint32_t m, uint32_t w) {
  const __half2 r = __hmax2_nan(*reinterpret_cast<__half2 *>(&m), __habs2(*reinterpret_cast<__half2 *>(&w)));
  return *reinterpret_cast<const uint32_t *>(&r);
}
template <>
__device__ __forceinline__ uint32_t max_abs2<__nv_bfloat16>(uint32_t m, uint32_t w) {
  const __nv_bfloat162 r =
      __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&m), __habs2(*reinterpret_cast<__nv_bfloat162 *>(&w)));
  return *reinterpret_cast<const uint32_t *>(&r);
}

struct Eight {
  float x[8];
};

// The nearest integers of x / scale, ties to even, NaN as 0: the definition.
__device__ __noinline__ Eight divide8(Eight v, float scale) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v.x[j] = static_cast<float>(static_cast<int>(rintf(__fdiv_rn(v.x[j], scale))));
  return v;
}

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it leaves an integer in the low bits

// The low bytes of eight integers q, given as q + kMagic.
__device__ __forceinline__ uint2 pack_bytes(const float (&t)[8]) {
  uint32_t u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(t[j]);
  return make_uint2(
      __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410),
      __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410));
}

// x / scale to the nearest integer, ties to even, as __fdiv_rn and rintf give
// it, for eight values with |x / scale| <= 128, without the division.  The
// product with 1 / scale is within 2^-22 * 128 of the quotient, so that only
// values within 2^-14 of a half can differ, and those take the division.
// Returns the integers' bytes; q holds them as floats.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float scale, float inv, bool plain, float (&q)[8]) {
  float t[8], off = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    t[j] = fmaf(x[j], inv, kMagic);
    q[j] = t[j] - kMagic;
    off = fmaxf(off, fabsf(fmaf(x[j], inv, -q[j])));
  }
  if (!(off < 0.5f - 6.2e-5f) || plain) {
    Eight v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v.x[j] = x[j];
    v = divide8(v, scale);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      q[j] = v.x[j];
      t[j] = q[j] + kMagic;
    }
  }
  return pack_bytes(t);
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint32_t (&w)[4], float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f2 = unpack2<T>(w[j]);
    f[2 * j] = f2.x;
    f[2 * j + 1] = f2.y;
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&q)[8], float scale) {
  return make_uint4(pack2<T>(q[0] * scale, q[1] * scale), pack2<T>(q[2] * scale, q[3] * scale),
                    pack2<T>(q[4] * scale, q[5] * scale), pack2<T>(q[6] * scale, q[7] * scale));
}

// One unit: row r's span s of head h.  D and BS are the head dimension and
// the tokens of a block; NT threads work on the unit.
template <typename T, int D, int BS>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const AppendParams p) {
  constexpr int NT = BS * D / 64;
  constexpr int PER = kThreads / NT;  // units per CTA
  __shared__ float part[kThreads / 32];
  pdl_launch();
  pdl_wait();
  const int tid = threadIdx.x % NT;
  const uint32_t unit = blockIdx.x * PER + threadIdx.x / NT;
  const int which = blockIdx.y;
  const bool in = unit < p.units;
  const uint32_t uu = in ? unit : 0;
  const uint32_t rs = uu / static_cast<uint32_t>(p.c.heads);
  const int h = static_cast<int>(uu - rs * p.c.heads);
  const int r = static_cast<int>(rs / static_cast<uint32_t>(p.spans));
  const int span = static_cast<int>(rs - static_cast<uint32_t>(r) * p.spans);

  const int held = min(max(p.c.lens[r], 0), p.c.width * BS);
  const int fresh = p.counts ? min(max(p.counts[r], 0), p.tokens) : p.tokens;
  const int col = held / BS + span;
  const int base = col * BS;  // first token of the block
  // Row r's tokens end here; what lies past the table is dropped.
  const int end = static_cast<int>(min(static_cast<int64_t>(held) + fresh, static_cast<int64_t>(p.c.width) * BS));
  const int blk = in && col < p.c.width ? p.c.table[static_cast<int64_t>(r) * p.c.width + col] : -1;
  const bool ok = blk >= 0 && blk < p.c.blocks && base < end;
  const int64_t tile = ok ? (static_cast<int64_t>(blk) * p.c.heads + h) : 0;
  int8_t *const q8 = (which ? p.c.v8 : p.c.k8) + (p.c.layer_tiles + tile) * BS * D;
  float *const qs = (which ? p.c.v_scale : p.c.k_scale) + p.c.layer_tiles + tile;
  const bool had = ok && base < held;  // the block holds tokens already
  const float before = had ? *qs : 0.0f;

  // Vector i of this thread: token tok0 + i * STEP of the block, elements d ..
  // d + 7.  A new token's values, or an old one's bytes.
  constexpr int STEP = NT / (D / 8);
  const int tok0 = tid / (D / 8), d = tid % (D / 8) * 8;
  const int old = ok ? min(held - base, BS) : 0, all = ok ? min(end - base, BS) : 0;  // tokens of the block
  const T *const src = static_cast<const T *>(p.src[which]) + r * p.row_s[which] + h * p.head_s[which] +
                       (static_cast<int64_t>(base) + tok0 - held) * p.tok_s[which] + d;
  const int64_t src_step = STEP * p.tok_s[which];
  int8_t *const dst = q8 + tok0 * D + d;
  // A block that the step fills from its first token, as most of a prompt's:
  // no conditions on the tokens.
  const bool full = old <= 0 && all == BS && p.vec;
  uint32_t x[kVecs][4];
  if (full) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint4 w = *reinterpret_cast<const uint4 *>(src + i * src_step);
      x[i][0] = w.x;
      x[i][1] = w.y;
      x[i][2] = w.z;
      x[i][3] = w.w;
    }
  } else
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int tok = tok0 + i * STEP;
    x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0;
    if (tok < old) {
      const uint2 w = *reinterpret_cast<const uint2 *>(dst + i * STEP * D);
      x[i][0] = w.x;
      x[i][1] = w.y;
    } else if (tok < all) {
      const T *const s = src + i * src_step;
      if (p.vec) {
        const uint4 w = *reinterpret_cast<const uint4 *>(s);
        x[i][0] = w.x;
        x[i][1] = w.y;
        x[i][2] = w.z;
        x[i][3] = w.w;
      } else {
        const uint16_t *const s16 = reinterpret_cast<const uint16_t *>(s);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = s16[2 * j] | static_cast<uint32_t>(s16[2 * j + 1]) << 16;
      }
    }
  }
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if (tok0 + i * STEP >= old)
#pragma unroll
      for (int j = 0; j < 4; ++j) most = max_abs2<T>(most, x[i][j]);
  }
  const float2 m2 = unpack2<T>(most);
  float top = fmaxf(m2.x, m2.y);
  if (m2.x != m2.x || m2.y != m2.y) top = __int_as_float(0x7f800000);
  // The unit's maximum.
#pragma unroll
  for (int o = (NT < 32 ? NT : 32) / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (NT > 32) {
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
    __syncthreads();
    const int w0 = threadIdx.x / NT * (NT / 32);
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) top = fmaxf(top, part[w0 + w]);
  }
  // (A product by definition, as in logmel.h: one in twenty maxima gives one unit in the last
  // place more or less than top / 127.)
  float now = fmaxf(before, top * (1.0f / 127.0f));
  if (now == 0.0f) now = 1.0f;
  const float shrink = had ? before / now : 1.0f, inv = 1.0f / now;
  const bool plain = !(inv > 0.0f && inv < INFINITY);  // an infinite or subnormal scale has no inverse to go by
  // Every thread of the unit has read the old scale before one writes it.
  if (NT <= 32) __syncwarp();
  if (ok && tid == 0) *qs = now;

  T *const values = static_cast<T *>(p.values[which]);
  T *const out = values && in ? values + ((static_cast<int64_t>(rs) * BS + tok0) * p.c.heads + h) * D + d : nullptr;
  const int64_t out_step = static_cast<int64_t>(STEP) * p.c.heads * D;
  if (full) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float f[8], q[8];
      unpack8<T>(x[i], f);
      *reinterpret_cast<uint2 *>(dst + i * STEP * D) = quantise8(f, now, inv, plain, q);
      if (out) __stcs(reinterpret_cast<uint4 *>(out + i * out_step), pack8<T>(q, now));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int tok = tok0 + i * STEP;
    uint2 *const at = reinterpret_cast<uint2 *>(dst + i * STEP * D);
    float q[8];
    if (tok >= all) {
      if (out) __stcs(reinterpret_cast<uint4 *>(out + i * out_step), make_uint4(0, 0, 0, 0));
      continue;
    }
    if (tok >= old) {
      float f[8];
      unpack8<T>(x[i], f);
      *at = quantise8(f, now, inv, plain, q);
    } else {
      bytes_to_f32(make_uint2(x[i][0], x[i][1]), q);
      if (shrink != 1.0f) {
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          t[j] = static_cast<float>(static_cast<int>(rintf(q[j] * shrink))) + kMagic;  // NaN as 0
          q[j] = t[j] - kMagic;
        }
        *at = pack_bytes(t);
      }
    }
    if (out) __stcs(reinterpret_cast<uint4 *>(out + i * out_step), pack8<T>(q, now));
  }
}

constexpr int kReadTokens = 4;  // consecutive tokens of a thread

struct ReadParams {
  KvView c;
  void *out[2];
  int32_t start, count, dim_shift;  // dim_shift: log2 of a head's 8-element vectors
  uint32_t per_token, units;        // vectors of a token; of a row, by kReadTokens
};

// A thread has one vector of kReadTokens tokens in a row: one division, and one
// look into the table a block, for all of them (100 instructions a vector otherwise,
// and bound by them).  Grid: (part of a row's vectors, row, layer and keys or
// values).  The open blocks of 320 rows, 4 layers of 16 heads of 64: 36.5 -> 30.0
// us, 197 MB at 6.6 TB/s.
template <typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams p) {
  pdl_launch();
  pdl_wait();
  const uint32_t unit = blockIdx.x * kThreads + threadIdx.x;
  if (unit >= p.units) return;
  const int which = blockIdx.z & 1, r = blockIdx.y;
  const int64_t layer = blockIdx.z >> 1;
  const int32_t *const table = p.c.table + static_cast<int64_t>(r) * p.c.width;
  const int64_t tiles = p.c.layer_tiles + layer * p.c.blocks * p.c.heads;
  const int8_t *const x8 = which ? p.c.v8 : p.c.k8;
  const float *const xs = which ? p.c.v_scale : p.c.k_scale;
  const uint32_t len = static_cast<uint32_t>(max(p.c.lens[r], 0));
  const uint32_t group = unit / p.per_token, e = unit - group * p.per_token;
  const uint32_t t0 = group * kReadTokens, in_block = p.c.block - 1;
  const int block_shift = 31 - __clz(p.c.block);
  const uint32_t head = e >> p.dim_shift, vec = e & ((1u << p.dim_shift) - 1);
  uint2 q[kReadTokens];
  float s[kReadTokens];
  const int8_t *block = nullptr;  // of the head and vector, where there is one
  float scale = 0.0f;
#pragma unroll
  for (int i = 0; i < kReadTokens; ++i) {
    const uint32_t tok = static_cast<uint32_t>(p.start) + t0 + i;
    if (i == 0 || (tok & in_block) == 0) {
      const uint32_t col = tok >> block_shift;
      const int blk = tok < len && col < static_cast<uint32_t>(p.c.width) ? table[col] : -1;
      block = nullptr;
      scale = 0.0f;
      if (blk >= 0 && blk < p.c.blocks) {
        const int64_t tile = tiles + static_cast<int64_t>(blk) * p.c.heads + head;
        scale = xs[tile];
        block = x8 + (tile << block_shift) * p.c.head_dim + vec * 8;
      }
    }
    const bool in = block && tok < len;
    s[i] = in ? scale : 0.0f;
    q[i] = in ? *reinterpret_cast<const uint2 *>(block + (tok & in_block) * p.c.head_dim) : make_uint2(0, 0);
  }
  uint4 *out = reinterpret_cast<uint4 *>(p.out[which]) +
               ((layer * p.c.rows + r) * static_cast<int64_t>(p.count) + t0) * p.per_token + e;
#pragma unroll
  for (int i = 0; i < kReadTokens; ++i, out += p.per_token) {
    if (t0 + i >= static_cast<uint32_t>(p.count)) break;
    float x[8];
    bytes_to_f32(q[i], x);
    __stcs(out, pack8<T>(x, s[i]));
  }
}

constexpr int kCopy = 4;  // vectors of keys and of values that a thread has in flight

struct ReorderParams {
  KvView c;
  const int32_t *parents;
  uint32_t *done;    // per clip: CTAs that have copied
  int32_t beams, parts;
};

// The parent row of row r, r itself where the given one is out of range.
__device__ __forceinline__ int parent_row(const ReorderParams &p, int r) {
  const int q = p.parents[r];
  return q >= 0 && q < p.beams ? r / p.beams * p.beams + q : r;
}

// Grid: (part, row).  Each CTA copies its part of the row's open block (over
// layers, keys and values, heads) from the parent's to the row's spare one.
// The tables still show the old state meanwhile; the last CTA of a clip to
// finish then rewrites them.  The open blocks of 320 rows, 4 layers of 16 heads
// of 64, 10.4 us with two CTAs a row (one 11.6, three 12.0, eight 16.5).
__global__ void __launch_bounds__(kThreads) reorder_kernel(const ReorderParams p) {
  pdl_launch();
  pdl_wait();
  const int r = blockIdx.y;
  const int clip = r / p.beams;
  const int64_t width = p.c.width;
  const int len = max(p.c.lens[clip * p.beams], 0);
  const int col = len / p.c.block;
  const bool open = len % p.c.block != 0 && col < width;
  const int from_row = parent_row(p, r);
  if (open && from_row != r) {
    const int from = p.c.table[from_row * width + col], to = p.c.spare[r];
    if (from >= 0 && from < p.c.blocks && to >= 0 && to < p.c.blocks) {
      // The tokens that are held: a head's first `used` 16-byte vectors.
      const uint32_t head_vecs = p.c.block * p.c.head_dim / 16, used = len % p.c.block * p.c.head_dim / 16;
      const uint32_t vecs = p.c.heads * used, all = vecs * p.c.layers;
      for (uint32_t i0 = blockIdx.x * kThreads + threadIdx.x; i0 < all; i0 += kCopy * gridDim.x * kThreads) {
        uint4 x[kCopy][2];
        int64_t at[kCopy];
#pragma unroll
        for (int u = 0; u < kCopy; ++u) {
          const uint32_t i = i0 + u * gridDim.x * kThreads;
          at[u] = -1;
          if (i >= all) continue;
          const uint32_t tile = i / used, v = i - tile * used;  // (layer, head) and its vector
          const uint32_t layer = tile / p.c.heads, head = tile - layer * p.c.heads;
          const int64_t first = static_cast<int64_t>(layer) * p.c.blocks;
          const int64_t a = ((first + from) * p.c.heads + head) * head_vecs + v;
          at[u] = ((first + to) * p.c.heads + head) * head_vecs + v;
          x[u][0] = reinterpret_cast<const uint4 *>(p.c.k8)[a];
          x[u][1] = reinterpret_cast<const uint4 *>(p.c.v8)[a];
        }
#pragma unroll
        for (int u = 0; u < kCopy; ++u) {
          if (at[u] < 0) continue;
          reinterpret_cast<uint4 *>(p.c.k8)[at[u]] = x[u][0];
          reinterpret_cast<uint4 *>(p.c.v8)[at[u]] = x[u][1];
        }
      }
      const int scales = p.c.heads * p.c.layers;
      for (int i = blockIdx.x * kThreads + threadIdx.x; i < scales; i += gridDim.x * kThreads) {
        const int64_t layer = i / p.c.heads, h = i % p.c.heads;
        const int64_t a = (layer * p.c.blocks + from) * p.c.heads + h, b = (layer * p.c.blocks + to) * p.c.heads + h;
        p.c.k_scale[b] = p.c.k_scale[a];
        p.c.v_scale[b] = p.c.v_scale[a];
      }
    }
  }
  // Last CTA of the clip: every reader of the old tables has finished.
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(&p.done[clip], 1u) == static_cast<uint32_t>(p.beams * p.parts - 1);
  }
  __syncthreads();
  if (!last) return;
  if (threadIdx.x == 0) p.done[clip] = 0;
  // A thread per beam and column, whole columns at a time: all entries of a
  // column are read before one is written.
  const int row0 = clip * p.beams;
  const int cols = static_cast<int>(min(static_cast<int64_t>(col) + (open ? 1 : 0), width));
  const int step = kThreads / p.beams, i = threadIdx.x % p.beams, c0 = threadIdx.x / p.beams;
  const int parent = parent_row(p, row0 + i);
  const int mine = p.c.spare[row0 + i];
  for (int c1 = 0; c1 < cols; c1 += step) {
    const int c = c1 + c0;
    const bool moves = c0 < step && c < cols && parent != row0 + i;
    int next = 0, was = 0;
    bool copied = false;
    if (moves) {
      was = p.c.table[(row0 + i) * width + c];
      next = p.c.table[parent * width + c];
      copied = c == col && next >= 0 && next < p.c.blocks;  // (an absent block stays absent)
      if (copied) next = mine;
    }
    __syncthreads();
    if (moves) {
      p.c.table[(row0 + i) * width + c] = next;
      if (copied) p.c.spare[row0 + i] = was;
    }
  }
}

template <typename T, int D>
lm_status append_block(const AppendParams &p, int block, cudaStream_t s) {
  const int nt = block * D / 64;
  const int per = kThreads / nt;
  const dim3 grid((p.units + per - 1) / per, 2);
  switch (block) {
    case 16: return launch_dependent(append_kernel<T, D, 16>, grid, kThreads, 0, s, 1, p);
    case 32: return launch_dependent(append_kernel<T, D, 32>, grid, kThreads, 0, s, 1, p);
    case 64: return launch_dependent(append_kernel<T, D, 64>, grid, kThreads, 0, s, 1, p);
    default: return launch_dependent(append_kernel<T, D, 128>, grid, kThreads, 0, s, 1, p);
  }
}

template <typename T>
lm_status append_dim(const AppendParams &p, int dim, int block, cudaStream_t s) {
  switch (dim) {
    case 32: return append_block<T, 32>(p, block, s);
    case 64: return append_block<T, 64>(p, block, s);
    default: return append_block<T, 128>(p, block, s);
  }
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

lm_status kv_check(const lm_kv_cache *c) {
  if (!c) return LM_ERR_INVALID_ARG;
  if (c->rows != 0 && !c->lens) return LM_ERR_INVALID_ARG;
  if (c->rows != 0 && c->width != 0 && (!c->k8 || !c->v8 || !c->k_scale || !c->v_scale || !c->table))
    return LM_ERR_INVALID_ARG;
  if (c->blocks < 0 || c->layers < 1 || c->rows < 0 || c->width < 0 || c->heads < 1) return LM_ERR_INVALID_ARG;
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) return LM_ERR_UNSUPPORTED;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) return LM_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->width) * c->block > INT_MAX - 65536 || c->blocks > INT_MAX) return LM_ERR_UNSUPPORTED;
  if (!aligned(c->k8, 16) || !aligned(c->v8, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->table, 4) || !aligned(c->lens, 4))
    return LM_ERR_MISALIGNED;
  return LM_OK;
}

KvView kv_view(const lm_kv_cache *c, int32_t layer) {
  KvView v;
  v.k8 = c->k8;
  v.v8 = c->v8;
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.table = c->table;
  v.spare = c->spare;
  v.lens = c->lens;
  v.blocks = c->blocks;
  v.layer_tiles = static_cast<int64_t>(layer < 0 ? 0 : layer) * c->blocks * c->heads;
  v.layers = c->layers;
  v.rows = c->rows;
  v.width = c->width;
  v.heads = c->heads;
  v.head_dim = c->head_dim;
  v.block = c->block;
  return v;
}

}  // namespace lm

extern "C" lm_status lm_kv_append(const lm_kv_cache *cache, int32_t layer, const void *k, const void *v,
                                  const int64_t *k_strides, const int64_t *v_strides, int32_t tokens,
                                  const int32_t *counts, int32_t dtype, void *k_values, void *v_values,
                                  lm_stream_t stream) {
  using namespace lm;
  if (lm_status st = kv_check(cache); st != LM_OK) return st;
  if (layer < 0 || layer >= cache->layers || tokens < 0 || !k_strides || !v_strides) return LM_ERR_INVALID_ARG;
  if (dtype != LM_F16 && dtype != LM_BF16) return LM_ERR_UNSUPPORTED;
  if ((k_values == nullptr) != (v_values == nullptr)) return LM_ERR_INVALID_ARG;
  if (cache->rows == 0 || tokens == 0) return LM_OK;
  if (!k || !v) return LM_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (k_strides[i] < 0 || v_strides[i] < 0) return LM_ERR_INVALID_ARG;
  if (!aligned(k, 2) || !aligned(v, 2) || !aligned(k_values, 16) || !aligned(v_values, 16)) return LM_ERR_MISALIGNED;
  if (tokens > INT_MAX - 256) return LM_ERR_UNSUPPORTED;
  AppendParams p;
  p.c = kv_view(cache, layer);
  p.src[0] = k;
  p.src[1] = v;
  p.values[0] = k_values;
  p.values[1] = v_values;
  p.vec = aligned(k, 16) && aligned(v, 16);
  for (int w = 0; w < 2; ++w) {
    const int64_t *s = w ? v_strides : k_strides;
    p.row_s[w] = s[0];
    p.tok_s[w] = s[1];
    p.head_s[w] = s[2];
    for (int i = 0; i < 3; ++i) p.vec = p.vec && s[i] % 8 == 0;
  }
  p.counts = counts;
  p.tokens = tokens;
  p.spans = (tokens - 1 + cache->block - 1) / cache->block + 1;
  const int64_t units = static_cast<int64_t>(cache->rows) * p.spans * cache->heads;
  if (units > INT_MAX - kThreads) return LM_ERR_UNSUPPORTED;
  p.units = static_cast<uint32_t>(units);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == LM_F16 ? append_dim<__half>(p, cache->head_dim, cache->block, s)
                         : append_dim<__nv_bfloat16>(p, cache->head_dim, cache->block, s);
}

extern "C" lm_status lm_kv_read(const lm_kv_cache *cache, int32_t layer, int32_t start, int32_t count, int32_t dtype,
                                void *k_out, void *v_out, lm_stream_t stream) {
  using namespace lm;
  if (lm_status st = kv_check(cache); st != LM_OK) return st;
  if (layer < -1 || layer >= cache->layers || start < 0 || count < 0) return LM_ERR_INVALID_ARG;
  if (dtype != LM_F16 && dtype != LM_BF16) return LM_ERR_UNSUPPORTED;
  if (cache->rows == 0 || count == 0) return LM_OK;
  if (!k_out || !v_out) return LM_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return LM_ERR_MISALIGNED;
  ReadParams p;
  p.c = kv_view(cache, layer);
  p.out[0] = k_out;
  p.out[1] = v_out;
  p.start = start;
  p.count = count;
  const int layers = layer < 0 ? cache->layers : 1;
  p.dim_shift = cache->head_dim == 32 ? 2 : cache->head_dim == 64 ? 3 : 4;
  const int64_t per_token = static_cast<int64_t>(cache->heads) << p.dim_shift;
  const int64_t units = (static_cast<int64_t>(count) + kReadTokens - 1) / kReadTokens * per_token;
  if (per_token > INT_MAX || units > INT_MAX - kThreads || cache->rows > 65535 || layers > 32767)
    return LM_ERR_UNSUPPORTED;
  p.per_token = static_cast<uint32_t>(per_token);
  p.units = static_cast<uint32_t>(units);
  const dim3 grid((p.units + kThreads - 1) / kThreads, cache->rows, 2 * layers);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == LM_F16 ? launch_dependent(read_kernel<__half>, grid, kThreads, 0, s, 1, p)
                         : launch_dependent(read_kernel<__nv_bfloat16>, grid, kThreads, 0, s, 1, p);
}

extern "C" lm_status lm_kv_reorder(const lm_kv_cache *cache, const int32_t *parents, int32_t beams, void *workspace,
                                   size_t workspace_bytes, lm_stream_t stream) {
  using namespace lm;
  if (lm_status st = kv_check(cache); st != LM_OK) return st;
  if (beams < 1 || cache->rows % beams != 0) return LM_ERR_INVALID_ARG;
  if (beams > 32 || cache->rows > 65535) return LM_ERR_UNSUPPORTED;
  if (cache->rows == 0 || cache->width == 0) return LM_OK;
  if (!parents || !cache->spare) return LM_ERR_INVALID_ARG;
  const int clips = cache->rows / beams;
  if (!workspace || workspace_bytes < kWorkspaceHeaderBytes + 4 * static_cast<size_t>(clips)) return LM_ERR_WORKSPACE;
  if (!aligned(workspace, 16) || !aligned(parents, 4) || !aligned(cache->spare, 4)) return LM_ERR_MISALIGNED;
  ReorderParams p;
  p.c = kv_view(cache, 0);
  p.parents = parents;
  p.done = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + kWorkspaceHeaderBytes);
  p.beams = beams;
  // CTAs of a row: about four an SM over all rows, and no more than a vector per thread
  // needs.
  const int64_t vecs = static_cast<int64_t>(cache->layers) * cache->heads * cache->block * cache->head_dim / 16;
  if (vecs > INT_MAX / 2) return LM_ERR_UNSUPPORTED;
  const int64_t most = (vecs + kThreads - 1) / kThreads, round = (4 * 152 + cache->rows / 2) / cache->rows;
  p.parts = static_cast<int32_t>(round < 1 ? 1 : round < most ? round : most);
  return launch_dependent(reorder_kernel, dim3(p.parts, cache->rows), kThreads, 0, reinterpret_cast<cudaStream_t>(stream),
                          1, p);
}
