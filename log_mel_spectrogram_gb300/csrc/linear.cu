// linear.cu -- y = residual + scale * act(x W^T + bias) on the tensor cores.
//
// A CTA computes tiles of 128 x bn outputs: one thread fetches 128 x 64 and
// bn x 64 operand tiles by TMA into a ring of shared-memory stages, one thread
// issues tcgen05.mma into tensor memory (32-bit sums), the other warps turn a
// finished tile into outputs while the next one is summed into the other half
// of the tensor memory.  CTAs are persistent: one per SM walks the tiles.
//
// The tile has two orientations.
//  - rows of x along the 128 lanes: a lane holds 16 consecutive outputs of a
//    row, i.e. whole 32-byte sectors per thread.  Taken where outputs (and the
//    residual) can be accessed in 16-byte vectors and there are enough rows.
//  - rows of W along the lanes: x fills the other side of the tile with
//    exactly the rows there are (bn = 16 .. 256), so few rows do not waste
//    products, and lanes are consecutive outputs, so odd row lengths still
//    store whole lines.
// Few tiles (decoding steps) split k over a cluster of CTAs, whose partial sums
// meet in distributed shared memory in rank order: one launch, and the same
// result on every call.
//
// Operands that TMA cannot address (rows off 16-byte boundaries) are first
// copied into padded rows in the workspace.
#include <climits>
#include <cuda.h>
#include <map>
#include <mutex>

#include "f32x2.cuh"
#include "half.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace lm {
namespace {

constexpr int kBk = 64;             // elements of k per stage: one 128-byte swizzle row
constexpr int kLanes = 128;         // rows of the tile's lane side
constexpr int kMaxBn = 256;
constexpr int kMaxStages = 8;

enum class Form {
  kOne,    // a CTA per tile of 128 lanes
  kPair,   // two CTAs per tile of 256 lanes
  kSplit,  // a cluster per tile, each CTA a part of k
};

// Warps: TMA, MMA, TMEM and an idle one, then the epilogue's: 16, or 8 for the
// split form's few columns.
constexpr int epi_warps(Form f) { return f == Form::kSplit ? 8 : 16; }
constexpr int threads_of(Form f) { return 128 + 32 * epi_warps(f); }
constexpr int kStageOut = 32 * 32 * 2;  // a warp's 32 rows x 32 columns of 16 bits

struct LinearParams {
  const void *bias, *residual;
  void *out;
  int64_t out_row, res_row;
  int64_t rows_total;         // rows of the output
  int32_t rows, k, n;         // rows per group
  int32_t bn, stages, kblocks, tmem_cols;
  int32_t lane_tiles, col_tiles, tiles;  // tiles along the lanes and columns of one group, and in all
  int32_t lane_step;          // rows along the lanes of a tile: 128, or a pair's 256
  int32_t splits;             // CTAs that share a tile's k
  int32_t bias_f32, out_f32, act, vec32;
  int32_t tma_out, stage_out; // outputs leave by TMA, through that many bytes of shared memory
  uint32_t idesc;
  float scale;
  uint32_t *err;
};

struct alignas(16) Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
};

// max(x, 0), NaN for NaN.
__device__ __forceinline__ float relu(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// z Phi(z) = max(z, 0) - |z| erfc(|z| / sqrt 2) / 2, with erfc by formula
// 7.1.26 of Abramowitz and Stegun, Handbook of Mathematical Functions
// (erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2), t = 1 / (1 + 0.3275911 x), off by
// at most 1.5e-7); the coefficients below are halved and negated.  Past
// |z| = 20 the second term is 0.
__device__ __forceinline__ f32x2 gelu2(f32x2 z) {
  const float2 zz = unpair(z);
  const f32x2 a = pair(fminf(fabsf(zz.x), 20.0f), fminf(fabsf(zz.y), 20.0f));
  const float2 den = unpair(fma2(both(0.3275911f * 0.70710678118654752f), a, both(1.0f)));
  const f32x2 t = pair(rcp(den.x), rcp(den.y));
  f32x2 q = fma2(both(-0.5f * 1.061405429f), t, both(0.5f * 1.453152027f));
  q = fma2(q, t, both(-0.5f * 1.421413741f));
  q = fma2(q, t, both(0.5f * 0.284496736f));
  q = fma2(q, t, both(-0.5f * 0.254829592f));
  const float2 arg = unpair(mul2(a, mul2(a, both(-0.5f * kLog2e))));
  const f32x2 e = pair(ex2(arg.x), ex2(arg.y));
  return fma2(mul2(a, t), mul2(q, e), pair(relu(zz.x), relu(zz.y)));
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if (ACT == LM_ACT_RELU) return relu(z);
  if (ACT == LM_ACT_GELU) return unpair(gelu2(both(z))).x;
  if (ACT == LM_ACT_GELU_TANH) {
    // (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
    const float u = fmaf(-2.0f * 0.79788456080286536f * kLog2e * 0.044715f * z * z, z,
                         -2.0f * 0.79788456080286536f * kLog2e * z);
    return z * rcp(1.0f + ex2(u));
  }
  if (ACT == LM_ACT_SILU) return z * rcp(1.0f + ex2(-kLog2e * z));
  return z;
}

template <int ACT>
__device__ __forceinline__ f32x2 activate2(f32x2 z) {
  if (ACT == LM_ACT_NONE) return z;
  if (ACT == LM_ACT_GELU) return gelu2(z);
  const float2 f = unpair(z);
  return pair(activate<ACT>(f.x), activate<ACT>(f.y));
}

__device__ __forceinline__ uint4 ldg_v4(const void *p) { return *reinterpret_cast<const uint4 *>(p); }

// 16 consecutive 16-bit values as f32, in 16-byte loads.
template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = ldg_v4(p + 8 * i);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack2<T>(u[j]);
      x[8 * i + 2 * j] = f.x;
      x[8 * i + 2 * j + 1] = f.y;
    }
  }
}

__device__ __forceinline__ void store_v8(void *p, const uint32_t (&w)[8], bool vec32) {
  if (vec32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <typename T>
__device__ __forceinline__ float bias_at(const LinearParams &p, int n) {
  if (!p.bias || n >= p.n) return 0.0f;
  return p.bias_f32 ? static_cast<const float *>(p.bias)[n] : to_f32(static_cast<const T *>(p.bias)[n]);
}

// One output element of the lane = W orientation.
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

// The 16 columns in `r` of a lane's tile row.
template <typename T, int ACT, bool SWAP>
__device__ __forceinline__ void finish16(const LinearParams &p, const uint32_t (&r)[16], const float *bias_s,
                                         float lane_bias, int64_t group_row, int lane_at, int col_at,
                                         uint32_t stage, uint32_t stage_at) {
  if (SWAP) {
    if (lane_at >= p.n) return;
    const int count = min(16, p.rows - col_at);
    const int64_t row = group_row + col_at;
    float y[16];
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const f32x2 z = add2(pair(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), both(lane_bias));
      const float2 f = unpair(mul2(both(p.scale), activate2<ACT>(z)));
      y[j] = f.x;
      y[j + 1] = f.y;
    }
    if (p.residual) {
      const T *x = static_cast<const T *>(p.residual) + row * p.res_row + lane_at;
#pragma unroll
      for (int j = 0; j < 16; ++j, x += p.res_row)
        if (j < count) y[j] += to_f32(*x);
    }
    if (p.out_f32) {
      float *o = static_cast<float *>(p.out) + row * p.out_row + lane_at;
#pragma unroll
      for (int j = 0; j < 16; ++j, o += p.out_row)
        if (j < count) *o = y[j];
    } else {
      T *o = static_cast<T *>(p.out) + row * p.out_row + lane_at;
      if (count == 16) {
#pragma unroll
        for (int j = 0; j < 16; ++j, o += p.out_row) *o = from_f32<T>(y[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j, o += p.out_row)
          if (j < count) *o = from_f32<T>(y[j]);
      }
    }
    return;
  }
  if (lane_at >= p.rows || col_at >= p.n) return;
  const int64_t row = group_row + lane_at;
  float y[16];
  const f32x2 scale = both(p.scale);
#pragma unroll
  for (int j = 0; j < 16; j += 4) {
    const float4 v = *reinterpret_cast<const float4 *>(bias_s + j);
    const f32x2 z0 = add2(pair(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), pair(v.x, v.y));
    const f32x2 z1 = add2(pair(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])), pair(v.z, v.w));
    const float2 y0 = unpair(mul2(scale, activate2<ACT>(z0))), y1 = unpair(mul2(scale, activate2<ACT>(z1)));
    y[j] = y0.x;
    y[j + 1] = y0.y;
    y[j + 2] = y1.x;
    y[j + 3] = y1.y;
  }
  if (p.tma_out) {
    if (p.residual) {
      if (col_at + 16 <= p.n) {
        float x[16];
        load16(static_cast<const T *>(p.residual) + row * p.res_row + col_at, x);
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] += x[j];
      } else {
        for (int j = 0; j < 16 && col_at + j < p.n; ++j)
          y[j] += to_f32(static_cast<const T *>(p.residual)[row * p.res_row + col_at + j]);
      }
    }
    // Two 16-byte parts of a 64-byte row, in the 64-byte swizzle.
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t off = stage_at + 16 * i, to = stage + (off ^ ((off >> 3) & 0x30u));
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(pack2<T>(y[8 * i], y[8 * i + 1])),
                   "r"(pack2<T>(y[8 * i + 2], y[8 * i + 3])), "r"(pack2<T>(y[8 * i + 4], y[8 * i + 5])),
                   "r"(pack2<T>(y[8 * i + 6], y[8 * i + 7]))
                   : "memory");
    }
    return;
  }
  if (col_at + 16 <= p.n) {
    if (p.residual) {
      float x[16];
      load16(static_cast<const T *>(p.residual) + row * p.res_row + col_at, x);
#pragma unroll
      for (int j = 0; j < 16; ++j) y[j] += x[j];
    }
    if (p.out_f32) {
      float *const o = static_cast<float *>(p.out) + row * p.out_row + col_at;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(y[8 * i + j]);
        store_v8(o + 8 * i, w, p.vec32);
      }
    } else {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = pack2<T>(y[2 * j], y[2 * j + 1]);
      store_v8(static_cast<T *>(p.out) + row * p.out_row + col_at, w, p.vec32);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (col_at + j >= p.n) break;
      float v = y[j];
      if (p.residual) v += to_f32(static_cast<const T *>(p.residual)[row * p.res_row + col_at + j]);
      if (p.out_f32) {
        static_cast<float *>(p.out)[row * p.out_row + col_at + j] = v;
      } else {
        static_cast<T *>(p.out)[row * p.out_row + col_at + j] = from_f32<T>(v);
      }
    }
  }
}

struct Tile {
  int group, lane0, col0;
};

// Consecutive tiles share their rows along the lanes; of a pair's 256 rows
// CTA `rank` has 128.
__device__ __forceinline__ Tile tile_at(const LinearParams &p, int t, int rank) {
  Tile o;
  const int per = p.lane_tiles * p.col_tiles;
  o.group = t / per;
  const int u = t % per;
  o.lane0 = u / p.col_tiles * p.lane_step + rank * kLanes;
  o.col0 = u % p.col_tiles * p.bn;
  return o;
}

// Turns tile `t` into outputs.  `acc` is the tile's tensor memory; warp e of
// the epilogue reads lanes 32 * (e % 4) .. + 31.  `stage`: the warp's shared
// memory for outputs that leave by TMA.
template <typename T, int ACT, bool SWAP>
__device__ __forceinline__ void epilogue(const LinearParams &p, const CUtensorMap *out_map, const Tile &t, uint32_t acc,
                                         const float *bias_s, int e, uint32_t stage) {
  const int64_t group_row = static_cast<int64_t>(t.group) * p.rows;
  const int lane = threadIdx.x % 32;
  const uint32_t base = acc + (static_cast<uint32_t>(32 * (e % 4)) << 16);
  const int at = t.lane0 + 32 * (e % 4) + lane;
  const int end = min(p.bn, (SWAP ? p.rows : p.n) - t.col0);
  uint32_t r[SWAP ? 1 : 2][16];
  if constexpr (SWAP) {
    // Every fourth 16 columns.
    const float lane_bias = bias_at<T>(p, at);
    for (int c = e / 4 * 16; c < end; c += 64) {
      tmem_ld16(base + c, r[0]);
      tmem_wait_ld();
      if (p.kblocks == 0) {
#pragma unroll
        for (int j = 0; j < 16; ++j) r[0][j] = 0;
      }
      finish16<T, ACT, SWAP>(p, r[0], bias_s, lane_bias, group_row, at, t.col0 + c, 0, 0);
    }
  } else {
    // Every fourth 32 columns.
    for (int c = e / 4 * 32; c < end; c += 128) {
      tmem_ld16(base + c, r[0]);
      tmem_ld16(base + c + 16, r[1]);
      if (p.tma_out) {  // the last outputs have left the stage
        if (lane == 0) tma_store_wait_read();
        __syncwarp();
      }
      tmem_wait_ld();
      if (p.kblocks == 0) {
#pragma unroll
        for (int j = 0; j < 16; ++j) r[0][j] = r[1][j] = 0;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        finish16<T, ACT, SWAP>(p, r[i], bias_s + c + 16 * i, 0.0f, group_row, at, t.col0 + c + 16 * i, stage,
                               static_cast<uint32_t>(lane * 64 + i * 32));
      if (p.tma_out) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && t.lane0 + 32 * (e % 4) < p.rows) {
          tma_store_3d(out_map, stage, t.col0 + c, t.lane0 + 32 * (e % 4), t.group);
          tma_store_commit();
        }
      }
    }
  }
}

template <typename T, bool SWAP>
__device__ __forceinline__ void epilogue_act(const LinearParams &p, const CUtensorMap *out_map, const Tile &t,
                                             uint32_t acc, const float *bias_s, int e, uint32_t stage) {
  switch (p.act) {
    case LM_ACT_RELU: epilogue<T, LM_ACT_RELU, SWAP>(p, out_map, t, acc, bias_s, e, stage); break;
    case LM_ACT_GELU: epilogue<T, LM_ACT_GELU, SWAP>(p, out_map, t, acc, bias_s, e, stage); break;
    case LM_ACT_GELU_TANH: epilogue<T, LM_ACT_GELU_TANH, SWAP>(p, out_map, t, acc, bias_s, e, stage); break;
    case LM_ACT_SILU: epilogue<T, LM_ACT_SILU, SWAP>(p, out_map, t, acc, bias_s, e, stage); break;
    default: epilogue<T, LM_ACT_NONE, SWAP>(p, out_map, t, acc, bias_s, e, stage); break;
  }
}

// The split form's outputs: columns of the tile are shared out over the
// cluster's CTAs; every CTA's partial sums lie at the same place of its
// shared memory, [column][lane].
template <typename T, int ACT>
__device__ __forceinline__ void finish_split(const LinearParams &p, const Tile &t, uint32_t partial, int rank, int tid,
                                             int threads) {
  const int64_t group_row = static_cast<int64_t>(t.group) * p.rows;
  const int cols = min(p.bn, p.rows - t.col0);
  for (int i = tid; i < kLanes * ((p.bn + p.splits - 1) / p.splits); i += threads) {
    const int c = i / kLanes * p.splits + rank, lane = i % kLanes;
    const int n = t.lane0 + lane;
    if (c >= cols || n >= p.n) continue;
    const uint32_t at = partial + static_cast<uint32_t>(c * kLanes + lane) * 4;
    float s = 0.0f;
    for (int r = 0; r < p.splits; ++r) s += __uint_as_float(ld_dsmem_u32(at, static_cast<uint32_t>(r)));
    put<T, ACT>(p, s, bias_at<T>(p, n), group_row + t.col0 + c, n);
  }
}

// Barrier of the epilogue's warps: whether `ok` holds for all their threads.
template <int THREADS>
__device__ __forceinline__ bool epilogue_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "n"(THREADS)
      : "memory");
  return r != 0;
}

template <typename T, bool SWAP, Form FORM>
__global__ void __launch_bounds__(threads_of(FORM), 1)
    linear_kernel(const __grid_constant__ CUtensorMap lane_map, const __grid_constant__ CUtensorMap col_map,
                  const __grid_constant__ CUtensorMap out_map, const LinearParams p) {
  constexpr bool PAIR = FORM == Form::kPair, SPLIT = FORM == Form::kSplit;
  constexpr int EPI = epi_warps(FORM);
  extern __shared__ __align__(1024) uint8_t ring[];  // stages on a boundary of the swizzle's period
  const int col_rows = PAIR ? p.bn / 2 : p.bn;  // rows of the column side that this CTA holds
  const int stage_bytes = kLanes * 128 + col_rows * 128;
  uint8_t *const stage_s = ring + p.stages * stage_bytes;  // outputs on their way
  Barriers &b = *reinterpret_cast<Barriers *>(stage_s + p.stage_out);
  float *const bias_s = reinterpret_cast<float *>(&b + 1);  // two tiles of bn
  // (The shuffle tells the compiler that the warp number is uniform.)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
  const int rank = FORM != Form::kOne ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = SPLIT ? static_cast<int>(blockIdx.x) / p.splits
                          : PAIR ? static_cast<int>(blockIdx.x) / 2 : static_cast<int>(blockIdx.x);
  const int step = SPLIT ? p.tiles : PAIR ? static_cast<int>(gridDim.x) / 2 : static_cast<int>(gridDim.x);
  const int lane_rank = PAIR ? rank : 0;
  // This CTA's part of k.
  const int k_begin = SPLIT ? static_cast<int>(static_cast<int64_t>(p.kblocks) * rank / p.splits) : 0;
  const int k_end = SPLIT ? static_cast<int>(static_cast<int64_t>(p.kblocks) * (rank + 1) / p.splits) : p.kblocks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&b.full[i], 1);
      mbar_init(&b.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.acc_full[i], 1);
      mbar_init(&b.acc_empty[i], PAIR ? 2 * EPI : EPI);
    }
    mbar_init(&b.drain, 1);
    b.abort = 0;
    fence_mbar_init();
    if (p.kblocks > 0) {
      tma_prefetch_map(&lane_map);
      tma_prefetch_map(&col_map);
    }
  }
  if (warp == 2) tmem_alloc<PAIR>(&b.tmem, static_cast<uint32_t>(p.tmem_cols));
  tcgen05_fence_before();
  __syncthreads();
  __syncwarp();
  if (PAIR) cluster_sync_all();  // both CTAs' barriers exist
  pdl_launch();
  pdl_wait();
  tcgen05_fence_after();
  const uint32_t tmem = b.tmem;
  volatile int *const abort = &b.abort;

  if (warp == 0) {
    int fills = 0, s = 0;
    uint32_t phase = 1;  // of the stage's last release; the first round waits for nothing
    bool ok = true;
    for (int t = first; t < p.tiles && ok; t += step) {
      const Tile tile = tile_at(p, t, lane_rank);
      const int col0 = tile.col0 + (PAIR ? rank * col_rows : 0);
      const int lane_z = SWAP ? 0 : tile.group, col_z = SWAP ? tile.group : 0;
      for (int kb = k_begin; kb < k_end; ++kb) {
        if (fills >= p.stages) ok = __all_sync(0xffffffffu, mbar_wait(&b.empty[s], phase, abort, p.err));
        if (!ok) break;
        if (elect_one()) {
          uint8_t *const dst = ring + s * stage_bytes;
          // A pair's copies all count on CTA 0's barrier, which expects both.
          // (CTA 1's may be first: the phase still lacks CTA 0's arrival.)
          uint32_t bar = smem_u32(&b.full[s]);
          if (PAIR) bar = cluster_addr(bar, 0);
          if (!PAIR || rank == 0)
            mbar_arrive_expect_tx(&b.full[s], static_cast<uint32_t>(PAIR ? 2 * stage_bytes : stage_bytes));
          tma_load_3d<PAIR>(dst, &lane_map, kb * kBk, tile.lane0, lane_z, bar);
          tma_load_3d<PAIR>(dst + kLanes * 128, &col_map, kb * kBk, col0, col_z, bar);
        }
        __syncwarp();
        ++fills;
        if (++s == p.stages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    // No copy outlives the CTA, whatever the other warps did.
    if (!ok) {
      if (!PAIR || rank == 0) {
        for (int f = fills > p.stages ? fills - p.stages : 0; f < fills; ++f)
          mbar_wait_drain(&b.full[f % p.stages], (f / p.stages) & 1, p.err);
      } else {  // counted on the other CTA's barriers: time enough for any copy
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 10000000ull) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    if (!PAIR || rank == 0) {
      int s = 0, tiles = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t ring_a = smem_u32(ring);
      for (int t = first; t < p.tiles && ok; t += step, ++tiles) {
        const int half = tiles & 1;
        if (tiles >= 2)
          ok = __all_sync(0xffffffffu, mbar_wait(&b.acc_empty[half], ((tiles >> 1) - 1) & 1, abort, p.err));
        tcgen05_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(half * (p.tmem_cols / 2));
        for (int kb = k_begin; kb < k_end && ok; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait(&b.full[s], phase, abort, p.err));
          if (!ok) break;
          tcgen05_fence_after();
          const uint64_t a = smem_desc_k128(ring_a + s * stage_bytes);
          const uint64_t c = smem_desc_k128(ring_a + s * stage_bytes + kLanes * 128);
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < kBk / 16; ++i)
              tcgen05_mma_f16<PAIR>(d, a + 2 * i, c + 2 * i, p.idesc, kb > k_begin || i > 0);
            tcgen05_commit<PAIR>(&b.empty[s]);
          }
          __syncwarp();
          if (++s == p.stages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (ok && elect_one()) tcgen05_commit<PAIR>(&b.acc_full[half]);
        __syncwarp();
      }
      if (!ok) {  // products in flight end before the tensor memory is given back
        if (elect_one()) tcgen05_commit<PAIR>(&b.drain);
        mbar_wait_drain(&b.drain, 0, p.err);
      }
    }
  } else if (warp >= 4) {
    const int e = warp - 4;
    const int et = threadIdx.x - 128;
    int tiles = 0;
    // A thread's column of the bias, fetched a tile ahead (bn <= threads).
    float next_bias = 0.0f;
    if (!SWAP && et < p.bn && first < p.tiles) next_bias = bias_at<T>(p, tile_at(p, first, lane_rank).col0 + et);
    for (int t = first; t < p.tiles; t += step, ++tiles) {
      const Tile tile = tile_at(p, t, lane_rank);
      const int half = tiles & 1;
      float *const bs = bias_s + half * p.bn;
      if (!SWAP) {
        // Every epilogue warp has left the tile that used this half before:
        // the barrier of the tile in between lies behind it.
        if (et < p.bn) {
          bs[et] = next_bias;
          if (t + step < p.tiles) next_bias = bias_at<T>(p, tile_at(p, t + step, lane_rank).col0 + et);
        }
      }
      bool ok = mbar_wait(&b.acc_full[half], (tiles >> 1) & 1, abort, p.err);
      // One decision for all warps that meet at the barrier, and per warp
      // elsewhere: tensor memory loads are executed by whole warps.
      ok = SWAP ? __all_sync(0xffffffffu, ok) : epilogue_all<32 * EPI>(ok);
      if (!ok) break;
      tcgen05_fence_after();
      const uint32_t acc = tmem + static_cast<uint32_t>(half * (p.tmem_cols / 2));
      if (SPLIT) {
        // Products are complete: the ring is free to hold the partial sums.
        float *const partial = reinterpret_cast<float *>(ring);
        const int lane = 32 * (e % 4) + static_cast<int>(threadIdx.x % 32);
        for (int c = e / 4 * 16; c < p.bn; c += EPI / 4 * 16) {
          uint32_t r[16];
          tmem_ld16(acc + (static_cast<uint32_t>(32 * (e % 4)) << 16) + c, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) partial[(c + j) * kLanes + lane] = __uint_as_float(r[j]);
        }
      } else {
        epilogue_act<T, SWAP>(p, &out_map, tile, acc, bs, e, smem_u32(stage_s) + e * kStageOut);
        tcgen05_fence_before();
        __syncwarp();
        if (threadIdx.x % 32 == 0) {
          if (PAIR && rank != 0) {
            mbar_arrive_cluster(cluster_addr(smem_u32(&b.acc_empty[half]), 0));
          } else {
            mbar_arrive(&b.acc_empty[half]);
          }
        }
      }
    }
  }

  if (warp >= 4 && threadIdx.x % 32 == 0) tma_store_wait_read();
  __syncwarp();
  if (SPLIT) {
    __syncthreads();
    cluster_sync_all();
    if (!*abort && first < p.tiles) {
      const Tile tile = tile_at(p, first, 0);
      const uint32_t partial = smem_u32(ring);
      const int tid = threadIdx.x;
      constexpr int N = threads_of(FORM);
      switch (p.act) {
        case LM_ACT_RELU: finish_split<T, LM_ACT_RELU>(p, tile, partial, rank, tid, N); break;
        case LM_ACT_GELU: finish_split<T, LM_ACT_GELU>(p, tile, partial, rank, tid, N); break;
        case LM_ACT_GELU_TANH: finish_split<T, LM_ACT_GELU_TANH>(p, tile, partial, rank, tid, N); break;
        case LM_ACT_SILU: finish_split<T, LM_ACT_SILU>(p, tile, partial, rank, tid, N); break;
        default: finish_split<T, LM_ACT_NONE>(p, tile, partial, rank, tid, N); break;
      }
    }
    cluster_sync_all();  // no CTA leaves while another reads its sums
  }
  tcgen05_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();  // ... or its barriers and tensor memory are in use
  if (warp == 2) {
    tcgen05_fence_after();
    tmem_dealloc<PAIR>(tmem, static_cast<uint32_t>(p.tmem_cols));
  }
}

// Copies rows off 16-byte boundaries into rows padded to 8 elements.
struct PackParams {
  const uint16_t *src;
  uint4 *dst;
  int64_t group_stride, row_stride, rows, k, vecs, total;  // vecs: 16-byte vectors a row
};

__global__ void __launch_bounds__(256) pack_kernel(const PackParams p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  pdl_launch();
  pdl_wait();
  if (i >= p.total) return;
  const int64_t row = i / p.vecs, v = i % p.vecs;
  const uint16_t *const s = p.src + row / p.rows * p.group_stride + row % p.rows * p.row_stride + v * 8;
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = v * 8 + j < p.k ? s[j] : 0u;
  p.dst[i] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

lm_status check(const lm_linear_args *a) {
  if (!a || a->groups < 0 || a->rows < 0 || a->k < 0 || a->n < 0) return LM_ERR_INVALID_ARG;
  if (a->x_group_stride < 0 || a->x_row_stride < 0 || a->weight_row_stride < 0 || a->residual_row_stride < 0 ||
      a->out_row_stride < 0)
    return LM_ERR_INVALID_ARG;
  if (a->activation < LM_ACT_NONE || a->activation > LM_ACT_SILU) return LM_ERR_INVALID_ARG;
  if (a->dtype != LM_F16 && a->dtype != LM_BF16) return LM_ERR_UNSUPPORTED;
  if ((a->bias && a->bias_dtype != LM_F32 && a->bias_dtype != a->dtype) ||
      (a->out_dtype != LM_F32 && a->out_dtype != a->dtype))
    return LM_ERR_UNSUPPORTED;
  const int64_t most = INT_MAX - 512;
  if (a->k > most || a->n > most || a->groups > most || a->rows > most ||
      (a->rows > 0 && a->groups > most / a->rows))
    return LM_ERR_UNSUPPORTED;
  return LM_OK;
}

// An operand as TMA sees it: [groups][rows][k], strides in elements.
struct Operand {
  const void *p;
  int64_t groups, rows, group_stride, row_stride;
  bool pack;       // copied into the workspace first
  size_t bytes;    // of that copy
};

Operand operand(const void *p, int64_t groups, int64_t rows, int64_t k, int64_t group_stride, int64_t row_stride) {
  Operand o{p, groups, rows, group_stride, row_stride, false, 0};
  if (o.rows == 1 && o.groups > 1) {  // one row per group: the groups are the rows
    o.rows = o.groups;
    o.groups = 1;
    o.row_stride = group_stride;
  }
  if (o.rows <= 1) o.row_stride = k;  // never used
  if (o.groups <= 1) o.group_stride = o.rows * o.row_stride;
  if (o.groups > 1 && o.group_stride == o.rows * o.row_stride) {
    o.rows *= o.groups;
    o.groups = 1;
  }
  // Strides that are in use must be multiples of 16 bytes, and not zero.
  const bool rows_ok = o.rows <= 1 || (o.row_stride > 0 && o.row_stride % 8 == 0);
  const bool groups_ok = o.groups <= 1 || (o.group_stride > 0 && o.group_stride % 8 == 0);
  o.pack = k > 0 && !(aligned(p, 16) && rows_ok && groups_ok && o.row_stride < (1ll << 38) &&
                      o.group_stride < (1ll << 38));
  if (o.pack) o.bytes = static_cast<size_t>(o.groups) * o.rows * ((k + 7) / 8) * 16;
  return o;
}

struct Plan {
  Operand x, w;
  size_t bytes;
};

Plan plan(const lm_linear_args &a) {
  Plan p;
  p.x = operand(a.x, a.groups, a.rows, a.k, a.x_group_stride, a.x_row_stride);
  p.w = operand(a.weight, 1, a.n, a.k, 0, a.weight_row_stride);
  p.bytes = 256 + (p.x.bytes + 255) / 256 * 256 + (p.w.bytes + 255) / 256 * 256;
  return p;
}

lm_status pack(Operand *o, int64_t k, void *dst, cudaStream_t s) {
  PackParams p;
  p.src = static_cast<const uint16_t *>(o->p);
  p.dst = static_cast<uint4 *>(dst);
  p.group_stride = o->group_stride;
  p.row_stride = o->row_stride;
  p.rows = o->rows;
  p.k = k;
  p.vecs = (k + 7) / 8;
  p.total = o->groups * o->rows * p.vecs;
  const int64_t ctas = (p.total + 255) / 256;
  if (ctas > INT_MAX) return LM_ERR_UNSUPPORTED;
  if (lm_status st = launch_dependent(pack_kernel, dim3(static_cast<unsigned>(ctas)), 256, 0, s, 1, p); st != LM_OK)
    return st;
  o->p = dst;
  o->row_stride = p.vecs * 8;
  o->group_stride = o->rows * o->row_stride;
  return LM_OK;
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// Boxes of `box_rows` rows x `box_k` (64 or 32) elements in a swizzle of as
// many bytes, zeros outside.
lm_status make_map(CUtensorMap *map, const Operand &o, int64_t k, int box_rows, bool bf16, int box_k = kBk) {
  const EncodeFn fn = encode_fn();
  if (!fn) return cuda_fail(cudaErrorNotSupported);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(o.rows),
                              static_cast<cuuint64_t>(o.groups)};
  // A stride that is not used still has to be a valid one.
  const int64_t pad = (k + 7) / 8 * 8;
  // (A row that is alone may have any stride.)
  const int64_t rs = o.rows > 1 ? o.row_stride : pad;
  const int64_t gs = o.groups > 1 ? o.group_stride : pad;
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(rs) * 2, static_cast<cuuint64_t>(gs) * 2};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_k), static_cast<cuuint32_t>(box_rows), 1}, one[3] = {1, 1, 1};
  const CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                        const_cast<void *>(o.p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        box_k == kBk ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? LM_OK : cuda_fail(cudaErrorInvalidValue);
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const LinearParams);

// Pairs of CTAs that the device holds at once (SMs that have no partner in
// their group stay out), asked once per device.
int resident_pairs(Kernel kernel, int threads, int smem, const DeviceInfo &dev) {
  static std::mutex mu;
  static std::map<int, int> known;
  std::lock_guard<std::mutex> lk(mu);
  const auto it = known.find(dev.device);
  if (it != known.end()) return it->second;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(dev.sm_count / 2 * 2));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    n = dev.sm_count / 2;
  }
  return known[dev.device] = n < dev.sm_count / 2 ? n : dev.sm_count / 2;
}

template <typename T>
Kernel kernel_of(bool swap, Form form) {
  if (form == Form::kSplit) return linear_kernel<T, true, Form::kSplit>;
  if (form == Form::kPair) return swap ? linear_kernel<T, true, Form::kPair> : linear_kernel<T, false, Form::kPair>;
  return swap ? linear_kernel<T, true, Form::kOne> : linear_kernel<T, false, Form::kOne>;
}

}  // namespace
}  // namespace lm

extern "C" lm_status lm_linear_workspace_size(const lm_linear_args *args, size_t *bytes) {
  if (!bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::check(args); st != LM_OK) return st;
  *bytes = lm::plan(*args).bytes;
  return LM_OK;
}

extern "C" lm_status lm_linear(const lm_linear_args *args, void *workspace, size_t workspace_bytes,
                               lm_stream_t stream) {
  using namespace lm;
  if (lm_status st = check(args); st != LM_OK) return st;
  const lm_linear_args &a = *args;
  if (a.groups * a.rows == 0 || a.n == 0) return LM_OK;
  if (!a.out || (a.k > 0 && (!a.x || !a.weight))) return LM_ERR_INVALID_ARG;
  const size_t out_size = a.out_dtype == LM_F32 ? 4 : 2;
  if (!aligned(a.x, 2) || !aligned(a.weight, 2) || !aligned(a.bias, a.bias_dtype == LM_F32 ? 4 : 2) ||
      !aligned(a.residual, 2) || !aligned(a.out, out_size) || !aligned(workspace, 16))
    return LM_ERR_MISALIGNED;
  Plan pl = plan(a);
  if (!workspace || workspace_bytes < pl.bytes) return LM_ERR_WORKSPACE;
  DeviceInfo dev;
  if (lm_status st = current_device_info(&dev); st != LM_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char *const scratch = static_cast<char *>(workspace) + 256;
  const size_t x_bytes = pl.x.bytes;
  if (pl.x.pack)
    if (lm_status st = pack(&pl.x, a.k, scratch, s); st != LM_OK) return st;
  if (pl.w.pack)
    if (lm_status st = pack(&pl.w, a.k, scratch + (x_bytes + 255) / 256 * 256, s); st != LM_OK) return st;

  LinearParams p = {};
  p.bias = a.bias;
  p.residual = a.residual;
  p.out = a.out;
  p.rows_total = a.groups * a.rows;
  p.out_row = a.out_row_stride;
  p.res_row = a.residual_row_stride;
  p.rows = static_cast<int32_t>(pl.x.rows);
  p.k = static_cast<int32_t>(a.k);
  p.n = static_cast<int32_t>(a.n);
  p.kblocks = (p.k + kBk - 1) / kBk;
  p.bias_f32 = a.bias_dtype == LM_F32;
  p.out_f32 = a.out_dtype == LM_F32;
  p.act = a.activation;
  p.scale = a.scale;
  p.err = static_cast<uint32_t *>(workspace);
  const bool bf16 = a.dtype == LM_BF16;

  // Outputs in 16-byte vectors, 16 of a row at a time.
  const int64_t ov = 16 / static_cast<int64_t>(out_size);
  const bool one_row = p.rows_total == 1;
  const bool vec = aligned(a.out, 16) && (one_row || a.out_row_stride % ov == 0) &&
                   (!a.residual || (aligned(a.residual, 16) && (one_row || a.residual_row_stride % 8 == 0)));
  p.vec32 = aligned(a.out, 32) && (one_row || a.out_row_stride % (2 * ov) == 0);
  // Up to 512 rows, tiles that hold exactly the rows there are beat 128 or 256
  // lanes of them (320 x 1024 onto 50048: 38 us against 42).
  const bool swap = !vec || p.rows <= 512;
  const int64_t lane_rows = swap ? p.n : p.rows, col_rows = swap ? p.rows : p.n;
  const int64_t groups = pl.x.groups;
  // Columns in equal tiles of at most 256, a multiple of 16 each.
  auto columns = [&](int most, int unit) {
    const int64_t n = (col_rows + most - 1) / most;
    return static_cast<int32_t>(((col_rows + n - 1) / n + unit - 1) / unit * unit);
  };
  auto count = [&](int lanes, int bn) {
    return (lane_rows + lanes - 1) / lanes * ((col_rows + bn - 1) / bn) * groups;
  };
  Form form = Form::kOne;
  const int unit = swap ? 16 : 32;
  p.bn = columns(kMaxBn, unit);
  const int32_t pair_bn = columns(kMaxBn, 32);
  // Pairs fetch a third less per product; their tiles are longer to fill and
  // to empty, which shows where k is short (k = 240: 20.5 us against 18.5).
  if (pair_bn >= 128 && p.kblocks >= 8 && count(2 * kLanes, pair_bn) >= dev.sm_count / 2) {
    form = Form::kPair;
    p.bn = pair_bn;
  } else if (!swap && count(kLanes, p.bn) < dev.sm_count && p.bn > 128) {
    p.bn = columns(128, unit);
  }
  p.lane_step = form == Form::kPair ? 2 * kLanes : kLanes;
  p.lane_tiles = static_cast<int32_t>((lane_rows + p.lane_step - 1) / p.lane_step);
  p.col_tiles = static_cast<int32_t>((col_rows + p.bn - 1) / p.bn);
  const int64_t tiles = count(p.lane_step, p.bn);
  if (tiles > INT_MAX / 16) return LM_ERR_UNSUPPORTED;
  p.tiles = static_cast<int32_t>(tiles);
  p.splits = 1;
  if (swap && form == Form::kOne && p.bn <= 64) {
    while (p.splits < 8 && tiles * p.splits * 2 <= dev.sm_count && p.kblocks >= p.splits * 2) p.splits *= 2;
    if (p.splits > 1) form = Form::kSplit;
  }
  p.tmem_cols = 32;
  while (p.tmem_cols < 2 * p.bn) p.tmem_cols *= 2;
  const int held_cols = form == Form::kPair ? p.bn / 2 : p.bn;
  const int stage_bytes = kLanes * 128 + held_cols * 128;
  p.tma_out = !swap && !p.out_f32;
  p.stage_out = p.tma_out ? epi_warps(form) * kStageOut : 0;
  const int rest = p.stage_out + static_cast<int>(sizeof(Barriers)) + 2 * p.bn * 4;
  p.stages = (227 * 1024 - rest) / stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.idesc = idesc_f16(bf16, static_cast<uint32_t>(p.lane_step), static_cast<uint32_t>(p.bn));
  const int smem = p.stages * stage_bytes + rest;

  CUtensorMap lanes = {}, cols = {}, outs = {};
  if (p.kblocks > 0) {
    if (lm_status st = make_map(&lanes, swap ? pl.w : pl.x, a.k, kLanes, bf16); st != LM_OK) return st;
    if (lm_status st = make_map(&cols, swap ? pl.x : pl.w, a.k, held_cols, bf16); st != LM_OK) return st;
  }
  if (p.tma_out) {
    const Operand o{a.out, groups, p.rows, static_cast<int64_t>(p.rows) * a.out_row_stride, a.out_row_stride, false, 0};
    if (lm_status st = make_map(&outs, o, a.n, 32, bf16, 32); st != LM_OK) return st;
  }
  const Kernel kernel = bf16 ? kernel_of<__nv_bfloat16>(swap, form) : kernel_of<__half>(swap, form);
  if (lm_status st = ensure_smem_attribute(reinterpret_cast<const void *>(kernel), smem); st != LM_OK) return st;
  int cluster = 1, grid = p.tiles < dev.sm_count ? p.tiles : dev.sm_count;
  if (form == Form::kSplit) {
    cluster = p.splits;
    grid = p.tiles * p.splits;
  } else if (form == Form::kPair) {
    cluster = 2;
    const int pairs = resident_pairs(kernel, threads_of(form), smem, dev);
    grid = 2 * (p.tiles < pairs ? p.tiles : pairs);
  }
  return launch_dependent(kernel, dim3(static_cast<unsigned>(grid)), threads_of(form), static_cast<size_t>(smem), s,
                          cluster, lanes, cols, outs, p);
}
