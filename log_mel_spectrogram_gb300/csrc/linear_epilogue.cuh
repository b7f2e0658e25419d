// linear_epilogue.cuh -- what linear.cu and linear4.cu share: a launch's parameters, its tiles, and their sums'
// way from tensor memory (or from a cluster's shared memories) to outputs.
#pragma once

#include "activate.cuh"
#include "f32x2.cuh"
#include "half.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace lm {
namespace {

constexpr int kBk = 64;      // elements of k per stage: one 128-byte swizzle row
constexpr int kLanes = 128;  // rows of W of a CTA's tile
constexpr int kMaxBn = 256;

struct LinearParams {
  const void *bias, *residual;
  void *out;
  int64_t out_row, res_row;
  int32_t rows, n;                       // rows of x per group; rows of W
  int32_t bn, stages, kblocks, tmem_cols;
  int32_t lane_tiles, col_tiles, tiles;  // of one group, and in all
  int32_t lane_step;                     // rows of W of a tile: 128, or a pair's 256
  int32_t lanes_inside;                  // consecutive tiles share x, not W
  int32_t splits;                        // CTAs that share a tile's k
  int32_t bias_f32, out_f32, act;
  uint32_t idesc;
  float scale;
  uint32_t *err;
  uint64_t wait_ns;                      // limit of a wait
  int32_t withheld;                      // CTA whose first stage never fills (tests), or -1
};

template <typename T>
__device__ __forceinline__ float bias_at(const LinearParams &p, int n) {
  if (!p.bias || n >= p.n) return 0.0f;
  return p.bias_f32 ? static_cast<const float *>(p.bias)[n] : to_f32(static_cast<const T *>(p.bias)[n]);
}

// One output element.
template <typename T, int ACT>
__device__ __forceinline__ void put(const LinearParams &p, float acc, float bias, int64_t row, int n) {
  float y = p.scale * activate<ACT>(acc + bias);
  if (p.residual) y += to_f32(static_cast<const T *>(p.residual)[row * p.res_row + n]);
  if (p.out_f32) {
    static_cast<float *>(p.out)[row * p.out_row + n] = y;
  } else {
    static_cast<T *>(p.out)[row * p.out_row + n] = from_f32<T>(y);
  }
}

// The residual of output n in `count` <= 16 rows from `row` on.
template <typename T>
__device__ __forceinline__ void residual_rows(const LinearParams &p, T (&v)[16], int64_t row, int count, int n) {
  if (n >= p.n) return;
  const T *x = static_cast<const T *>(p.residual) + row * p.res_row + n;
#pragma unroll
  for (int j = 0; j < 16; ++j, x += p.res_row)
    if (j < count) v[j] = *x;
}

// Output n of `count` <= 16 rows from `row` on, from the lane's sums r.
template <typename T, int ACT, bool RES>
__device__ __forceinline__ void put_rows(const LinearParams &p, const uint32_t (&r)[16], const T (&residual)[16],
                                         float bias, int64_t row, int count, int n) {
  float y[16];
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const f32x2 z = add2(pair(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), both(bias));
    const float2 f = unpair(mul2(both(p.scale), activate2<ACT>(z)));
    y[j] = f.x;
    y[j + 1] = f.y;
  }
  if (RES) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < count) y[j] += to_f32(residual[j]);
  }
  if (p.out_f32) {
    float *o = static_cast<float *>(p.out) + row * p.out_row + n;
#pragma unroll
    for (int j = 0; j < 16; ++j, o += p.out_row)
      if (j < count) *o = y[j];
  } else {
    T *o = static_cast<T *>(p.out) + row * p.out_row + n;
    if (count == 16) {
#pragma unroll
      for (int j = 0; j < 16; ++j, o += p.out_row) *o = from_f32<T>(y[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j, o += p.out_row)
        if (j < count) *o = from_f32<T>(y[j]);
    }
  }
}

struct Tile {
  int group, lane0, col0;
};

// Of a pair's 256 lanes CTA `rank` has 128.
__device__ __forceinline__ Tile tile_at(const LinearParams &p, int t, int rank) {
  Tile o;
  const int per = p.lane_tiles * p.col_tiles;
  o.group = t / per;
  const int u = t - o.group * per;
  const int inside = p.lanes_inside ? p.lane_tiles : p.col_tiles;
  const int outer = u / inside, inner = u - outer * inside;
  o.lane0 = (p.lanes_inside ? inner : outer) * p.lane_step + rank * kLanes;
  o.col0 = (p.lanes_inside ? outer : inner) * p.bn;
  return o;
}

// Turns tile `t` into outputs.  `acc` is the tile's tensor memory; warp e of WARPS
// has lanes 32 * (e % 4) .. + 31 and every (WARPS / 4)th 16 columns.
// RES: `residual` has that of the first 16 columns; the next ones' travels while they
// are worked on (2642 x 144 x 12143 66 -> 38 us, 24000 x 1024 x 1024 57 -> 42).
template <typename T, int ACT, bool RES, int WARPS>
__device__ __forceinline__ void epilogue(const LinearParams &p, const Tile &t, uint32_t acc, int e, T (&residual)[16]) {
  const int n = t.lane0 + 32 * (e % 4) + static_cast<int>(threadIdx.x % 32);
  const int64_t row = static_cast<int64_t>(t.group) * p.rows + t.col0;
  const int cols = min(p.bn, p.rows - t.col0);
  const uint32_t base = acc + (static_cast<uint32_t>(32 * (e % 4)) << 16);
  const float bias = bias_at<T>(p, n);
  for (int c = e / 4 * 16; c < cols; c += 4 * WARPS) {
    uint32_t r[16];
    tmem_ld16(base + c, r);
    tmem_wait_ld();
    if (p.kblocks == 0) {
#pragma unroll
      for (int j = 0; j < 16; ++j) r[j] = 0;
    }
    T now[16];
    if (RES) {
#pragma unroll
      for (int j = 0; j < 16; ++j) now[j] = residual[j];
      if (c + 4 * WARPS < cols) residual_rows<T>(p, residual, row + c + 4 * WARPS, min(16, cols - c - 4 * WARPS), n);
    }
    if (n < p.n) put_rows<T, ACT, RES>(p, r, now, bias, row + c, min(16, cols - c), n);
  }
}

// The split form's outputs: columns of the tile are shared out over the
// cluster's CTAs; every CTA's partial sums lie at the same place of its
// shared memory, [column][lane].
template <typename T, int ACT>
__device__ __forceinline__ void finish_split(const LinearParams &p, const Tile &t, uint32_t partial, int rank, int tid,
                                             int threads) {
  const int64_t row = static_cast<int64_t>(t.group) * p.rows + t.col0;
  const int cols = min(p.bn, p.rows - t.col0);
  for (int i = tid; i < kLanes * ((p.bn + p.splits - 1) / p.splits); i += threads) {
    const int c = i / kLanes * p.splits + rank, lane = i % kLanes;
    const int n = t.lane0 + lane;
    if (c >= cols || n >= p.n) continue;
    const uint32_t at = partial + static_cast<uint32_t>(c * kLanes + lane) * 4;
    uint32_t v[kMaxSplits];
#pragma unroll
    for (int r = 0; r < kMaxSplits; ++r)
      if (r < p.splits) v[r] = ld_dsmem_u32(at, static_cast<uint32_t>(r));
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < kMaxSplits; ++r)
      if (r < p.splits) s += __uint_as_float(v[r]);
    put<T, ACT>(p, s, bias_at<T>(p, n), row + c, n);
  }
}

template <typename T, bool RES, int WARPS>
__device__ __forceinline__ void epilogue_act(const LinearParams &p, const Tile &t, uint32_t acc, int e,
                                             T (&residual)[16]) {
  switch (p.act) {
    case LM_ACT_RELU: epilogue<T, LM_ACT_RELU, RES, WARPS>(p, t, acc, e, residual); break;
    case LM_ACT_GELU: epilogue<T, LM_ACT_GELU, RES, WARPS>(p, t, acc, e, residual); break;
    case LM_ACT_GELU_TANH: epilogue<T, LM_ACT_GELU_TANH, RES, WARPS>(p, t, acc, e, residual); break;
    case LM_ACT_SILU: epilogue<T, LM_ACT_SILU, RES, WARPS>(p, t, acc, e, residual); break;
    default: epilogue<T, LM_ACT_NONE, RES, WARPS>(p, t, acc, e, residual); break;
  }
}

template <typename T>
__device__ __forceinline__ void finish_split_act(const LinearParams &p, const Tile &t, uint32_t partial, int rank,
                                                 int tid, int threads) {
  switch (p.act) {
    case LM_ACT_RELU: finish_split<T, LM_ACT_RELU>(p, t, partial, rank, tid, threads); break;
    case LM_ACT_GELU: finish_split<T, LM_ACT_GELU>(p, t, partial, rank, tid, threads); break;
    case LM_ACT_GELU_TANH: finish_split<T, LM_ACT_GELU_TANH>(p, t, partial, rank, tid, threads); break;
    case LM_ACT_SILU: finish_split<T, LM_ACT_SILU>(p, t, partial, rank, tid, threads); break;
    default: finish_split<T, LM_ACT_NONE>(p, t, partial, rank, tid, threads); break;
  }
}

}  // namespace
}  // namespace lm
