// gated.cu -- act(x Wg^T + bg) * (x Wu^T + bu), and its gradients, on the tensor cores.
//
// Backward, with a = x Wg^T + bg and b = x Wu^T + bu computed anew:
//   da = grad b act'(a), db = grad act(a)
//   dx = da Wg + db Wu, dWg = da^T x, dWu = db^T x, dbg and dbu the sums of da and db over rows.
//
// One kernel, built as linear.cu's is (TMA into a ring of stages, tcgen05.mma into
// tensor memory, sixteen warps that turn a finished tile into outputs while the next
// one is summed; a CTA, a pair of CTAs or a cluster that shares out the sum per tile),
// computes four products, all with 128 lanes a CTA and bn columns:
//   forward   lanes are outputs n, columns rows of x; a stage holds a tile of Wg and of Wu
//             and one of x, the tensor memory both sums, which meet in registers
//   grads     the same, with da and db for outputs; for a layer with biases (grad sums) also
//             their sums over columns, from products that are added up in registers every 256 of k
//   input     dx: lanes are k, columns rows; W is summed over n, along its rows (an
//             operand whose contiguous index is not summed over, "MN-major")
//   weight    dWg and dWu: lanes are k, columns n; x and da or db are both summed over rows
// So no operand is transposed in memory, and consecutive lanes are consecutive outputs.
//
// Measured, in a graph: 24000 x 1024 -> 4096 bf16 forward 215 to 222 us (1.8 to 1.87 PFLOP/s; 258 in a long row of calls, at the
// clock that the power limit allows: 1.56, 91% of the sustained rate); 12000 rows with all gradients 455 to 465 us
// (540 in a long row: 1.49 PFLOP/s with the second a and b), with biases 567.  5 x 1024 -> 4096 5.8 us for
// 16.8 MB of weights (k over clusters).  777 x 504 -> 1008 f16 with biases and gradients 31 us, five launches of
// about 5; 777 x 500 -> 1001 38 to 48, with copies of all operands to 16-byte boundaries in both directions.
//
// a and b are computed twice instead of kept: a training step keeps nothing but its inputs.  In 32 bits they would be
// 8 bytes of memory an element, and 16 of traffic (written and read; the gradient, da and db pass either way), as much
// time as computing them anew takes products at a k of about 1000 to 1100 (4 k operations an element, at 1710 to 1911
// TFLOP/s): above that it is the slower way, taken for the memory.  In 16 bits the biases' gradients would lose their 32.
#include <climits>

#include "activate.cuh"
#include "half.cuh"
#include "internal.h"
#include "operand.cuh"
#include "pdl.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "waits.cuh"

namespace lm {
namespace {

constexpr int kBk = 64;  // of the summed index, per stage
constexpr int kLanes = 128;
constexpr int kTileBytes = kLanes * kBk * 2;
constexpr int kBoxBytes = 64 * kBk * 2;  // 64 elements of a contiguous index by 64 of the summed one
constexpr int kMaxStages = 8;

enum class Form { kOne, kPair, kSplit };
enum class Kind { kForward, kGrads, kGradSums, kInput, kWeight };

constexpr bool dual(Kind k) { return k == Kind::kForward || k == Kind::kGrads || k == Kind::kGradSums; }
constexpr int epi_warps(Form f) { return f == Form::kSplit ? 8 : 16; }
constexpr int threads_of(Form f) { return 128 + 32 * epi_warps(f); }
// Blocks of k after which sums that have to be right to 32 bits go from tensor memory into registers: it loses a
// little towards zero with each of its additions (measured at k = 912: 7e-7 of the result, systematically, where
// additions that round are 2e-7 off), which a sum of thousands of da keeps.  All other sums stay in tensor memory and end
// in 16 bits, to half a step of 2^-11 or 2^-8 of them: of products of one sign they lose 7e-10 a product (linear with f32
// outputs 1.1e-5 at k = 16384, 1.9e-4 at 262144), of random signs a fifth of that, which a weight's gradient does not show
// (512 x 256 in f16, over 4096 rows 2.94e-4 off in the norm, over 200000 2.95e-4).
constexpr int kSumBlocks = 4;
// Parts of a tile's columns whose sums of da and db are kept apart.
constexpr int kColumnParts = epi_warps(Form::kOne) / 4;

struct GatedParams {
  const void *bg, *bu, *grad;
  void *out[2];       // forward: y; grads: da, db; input: dx; weight: dWg, dWu
  float *columns;     // [column tiles * kColumnParts][2][n], sums of da and db (Kind::kGradSums)
  int64_t out_row, grad_row;
  int32_t rows, n;    // columns and lanes of a group's outputs
  int32_t bn, stages, blocks, half_blocks, tmem_cols;
  int32_t lane_tiles, col_tiles, tiles, lane_step, lanes_inside, splits, first_group;
  int32_t bias_f32, act;
  uint32_t idesc;
  uint32_t *err;
  uint64_t wait_ns;
  int32_t withheld;
};

__device__ uint32_t g_gated_error;

struct alignas(16) Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
};

struct Tile {
  int group, lane0, col0, col_tile;
};

__device__ __forceinline__ Tile tile_at(const GatedParams &p, int t, int rank) {
  Tile o;
  const int per = p.lane_tiles * p.col_tiles;
  const int g = t / per;
  o.group = p.first_group + g;
  const int u = t - g * per;
  const int inside = p.lanes_inside ? p.lane_tiles : p.col_tiles;
  const int outer = u / inside, inner = u - outer * inside;
  o.lane0 = (p.lanes_inside ? inner : outer) * p.lane_step + rank * kLanes;
  o.col_tile = p.lanes_inside ? outer : inner;
  o.col0 = o.col_tile * p.bn;
  return o;
}

template <typename T>
__device__ __forceinline__ float bias_of(const void *b, int f32, int i) {
  if (!b) return 0.0f;
  return f32 ? static_cast<const float *>(b)[i] : to_f32(static_cast<const T *>(b)[i]);
}

// Values of activations for two elements; those of linear.cu work on pairs.
template <int ACT>
__device__ __forceinline__ float2 gate2(float a, float b) {
  if (ACT == LM_ACT_SIGMOID) return make_float2(sigmoid(a), sigmoid(b));
  return unpair(activate2<ACT>(pair(a, b)));
}

// The gradient at `count` <= 8 rows from `row` on.
template <typename T>
__device__ __forceinline__ void grad_rows(const GatedParams &p, T (&v)[8], int64_t row, int count, int n) {
  if (n >= p.n) return;
  const T *x = static_cast<const T *>(p.grad) + row * p.grad_row + n;
#pragma unroll
  for (int j = 0; j < 8; ++j, x += p.grad_row)
    if (j < count) v[j] = *x;
}

// Both sums of eight columns of a lane into outputs.
template <typename T, Kind KIND, int ACT>
__device__ __forceinline__ void put_dual(const GatedParams &p, const uint32_t (&ra)[8], const uint32_t (&rb)[8],
                                         const T (&grad)[8], float bg, float bu, float2 &sums, int64_t row, int count,
                                         int n) {
  T *o = static_cast<T *>(p.out[0]) + row * p.out_row + n;
  if constexpr (KIND == Kind::kForward) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 y = gate2<ACT>(__uint_as_float(ra[j]) + bg, __uint_as_float(ra[j + 1]) + bg);
      if (j < count) *o = from_f32<T>(y.x * (__uint_as_float(rb[j]) + bu));
      o += p.out_row;
      if (j + 1 < count) *o = from_f32<T>(y.y * (__uint_as_float(rb[j + 1]) + bu));
      o += p.out_row;
    }
  } else {
    T *o2 = static_cast<T *>(p.out[1]) + row * p.out_row + n;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float slope;
      const float y = activate_slope<ACT>(__uint_as_float(ra[j]) + bg, slope);
      const float g = to_f32(grad[j]);
      const float da = g * (__uint_as_float(rb[j]) + bu) * slope, db = g * y;
      if (j < count) {
        *o = from_f32<T>(da);
        *o2 = from_f32<T>(db);
        sums.x += da;
        sums.y += db;
      }
      o += p.out_row;
      o2 += p.out_row;
    }
  }
}

// The sums of da and db of a warp's columns in a tile.
__device__ __forceinline__ void put_columns(const GatedParams &p, const Tile &t, int e, int n, float2 sums) {
  float *const to = p.columns + (static_cast<int64_t>(t.col_tile) * kColumnParts + e / 4) * 2 * p.n + n;
  to[0] = sums.x;
  to[p.n] = sums.y;
}

// Turns a tile of both sums into outputs: warp e has lanes 32 * (e % 4) .. + 31 and every fourth 8 columns.
template <typename T, Kind KIND, int ACT>
__device__ __forceinline__ void dual_epilogue(const GatedParams &p, const Tile &t, uint32_t acc, int e, T (&grad)[8]) {
  const int n = t.lane0 + 32 * (e % 4) + static_cast<int>(threadIdx.x % 32);
  const int64_t row = t.col0;
  const int cols = min(p.bn, p.rows - t.col0);
  const uint32_t base = acc + (static_cast<uint32_t>(32 * (e % 4)) << 16);
  const bool in = n < p.n;
  const float bg = in ? bias_of<T>(p.bg, p.bias_f32, n) : 0.0f, bu = in ? bias_of<T>(p.bu, p.bias_f32, n) : 0.0f;
  float2 sums = make_float2(0.0f, 0.0f);
  for (int c = e / 4 * 8; c < cols; c += 32) {
    uint32_t ra[8], rb[8];
    tmem_ld8(base + c, ra);
    tmem_ld8(base + p.tmem_cols / 4 + c, rb);
    tmem_wait_ld();
    if (p.blocks == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) ra[j] = rb[j] = 0;
    }
    T now[8];
    if constexpr (KIND == Kind::kGrads) {
#pragma unroll
      for (int j = 0; j < 8; ++j) now[j] = grad[j];
      if (c + 32 < cols) grad_rows<T>(p, grad, row + c + 32, min(8, cols - c - 32), n);
    }
    if (in) put_dual<T, KIND, ACT>(p, ra, rb, now, bg, bu, sums, row + c, min(8, cols - c), n);
  }
}

// ... from a lane's sums of 16 columns in registers, from column 16 * (e / 4) on (Kind::kGradSums).
template <typename T, int ACT>
__device__ __forceinline__ void held_epilogue(const GatedParams &p, const Tile &t, int e, const float (&a)[16],
                                              const float (&b)[16], const T (&grad)[2][8]) {
  const int n = t.lane0 + 32 * (e % 4) + static_cast<int>(threadIdx.x % 32), c = e / 4 * 16;
  const int cols = min(p.bn, p.rows - t.col0) - c;
  if (n >= p.n) return;
  const float bg = bias_of<T>(p.bg, p.bias_f32, n), bu = bias_of<T>(p.bu, p.bias_f32, n);
  float2 sums = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t ra[8], rb[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ra[j] = __float_as_uint(a[8 * h + j]);
      rb[j] = __float_as_uint(b[8 * h + j]);
    }
    if (8 * h < cols)
      put_dual<T, Kind::kGradSums, ACT>(p, ra, rb, grad[h], bg, bu, sums, static_cast<int64_t>(t.col0) + c + 8 * h,
                                        min(8, cols - 8 * h), n);
  }
  if (p.columns) put_columns(p, t, e, n, sums);
}

template <typename T, Kind KIND>
__device__ __forceinline__ void dual_epilogue_act(const GatedParams &p, const Tile &t, uint32_t acc, int e, T (&grad)[8]) {
  switch (p.act) {
    case LM_ACT_RELU: dual_epilogue<T, KIND, LM_ACT_RELU>(p, t, acc, e, grad); break;
    case LM_ACT_GELU: dual_epilogue<T, KIND, LM_ACT_GELU>(p, t, acc, e, grad); break;
    case LM_ACT_GELU_TANH: dual_epilogue<T, KIND, LM_ACT_GELU_TANH>(p, t, acc, e, grad); break;
    case LM_ACT_SILU: dual_epilogue<T, KIND, LM_ACT_SILU>(p, t, acc, e, grad); break;
    case LM_ACT_SIGMOID: dual_epilogue<T, KIND, LM_ACT_SIGMOID>(p, t, acc, e, grad); break;
    default: dual_epilogue<T, KIND, LM_ACT_NONE>(p, t, acc, e, grad); break;
  }
}

template <typename T>
__device__ __forceinline__ void held_epilogue_act(const GatedParams &p, const Tile &t, int e, const float (&a)[16],
                                                  const float (&b)[16], const T (&grad)[2][8]) {
  switch (p.act) {
    case LM_ACT_RELU: held_epilogue<T, LM_ACT_RELU>(p, t, e, a, b, grad); break;
    case LM_ACT_GELU: held_epilogue<T, LM_ACT_GELU>(p, t, e, a, b, grad); break;
    case LM_ACT_GELU_TANH: held_epilogue<T, LM_ACT_GELU_TANH>(p, t, e, a, b, grad); break;
    case LM_ACT_SILU: held_epilogue<T, LM_ACT_SILU>(p, t, e, a, b, grad); break;
    case LM_ACT_SIGMOID: held_epilogue<T, LM_ACT_SIGMOID>(p, t, e, a, b, grad); break;
    default: held_epilogue<T, LM_ACT_NONE>(p, t, e, a, b, grad); break;
  }
}

// ... and one of a single sum.
template <typename T, Kind KIND>
__device__ __forceinline__ void plain_epilogue(const GatedParams &p, const Tile &t, uint32_t acc, int e) {
  const int n = t.lane0 + 32 * (e % 4) + static_cast<int>(threadIdx.x % 32);
  const int cols = min(p.bn, p.rows - t.col0);
  const uint32_t base = acc + (static_cast<uint32_t>(32 * (e % 4)) << 16);
  T *const out = static_cast<T *>(p.out[KIND == Kind::kWeight ? t.group : 0]) + t.col0 * p.out_row + n;
  for (int c = e / 4 * 16; c < cols; c += 64) {
    uint32_t r[16];
    tmem_ld16(base + c, r);
    tmem_wait_ld();
    if (n >= p.n) continue;
    T *o = out + c * p.out_row;
    const int count = cols - c;
#pragma unroll
    for (int j = 0; j < 16; ++j, o += p.out_row)
      if (j < count) *o = from_f32<T>(p.blocks ? __uint_as_float(r[j]) : 0.0f);
  }
}

// The split form's outputs: columns of the tile are shared out over the cluster's CTAs; every CTA's partial
// sums lie at the same place of its shared memory, [column][lane].
template <typename T, Kind KIND>
__device__ __forceinline__ void finish_split(const GatedParams &p, const Tile &t, uint32_t partial, int rank, int tid,
                                             int threads) {
  const int cols = min(p.bn, p.rows - t.col0);
  for (int i = tid; i < kLanes * ((p.bn + p.splits - 1) / p.splits); i += threads) {
    const int c = i / kLanes * p.splits + rank, lane = i % kLanes;
    const int n = t.lane0 + lane;
    if (c >= cols || n >= p.n) continue;
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < (dual(KIND) ? 2 : 1); ++h) {
      const uint32_t at = partial + static_cast<uint32_t>((c + h * p.bn) * kLanes + lane) * 4;
      uint32_t v[kMaxSplits];
#pragma unroll
      for (int r = 0; r < kMaxSplits; ++r)
        if (r < p.splits) v[r] = ld_dsmem_u32(at, static_cast<uint32_t>(r));
#pragma unroll
      for (int r = 0; r < kMaxSplits; ++r)
        if (r < p.splits) s[h] += __uint_as_float(v[r]);
    }
    const int64_t at = (static_cast<int64_t>(t.col0) + c) * p.out_row + n;
    if constexpr (KIND == Kind::kForward) {
      const float a = s[0] + bias_of<T>(p.bg, p.bias_f32, n), b = s[1] + bias_of<T>(p.bu, p.bias_f32, n);
      static_cast<T *>(p.out[0])[at] = from_f32<T>(activate_any(a, p.act) * b);
    } else {
      static_cast<T *>(p.out[KIND == Kind::kWeight ? t.group : 0])[at] = from_f32<T>(s[0]);
    }
  }
}

template <typename T, Form FORM, Kind KIND>
__global__ void __launch_bounds__(threads_of(FORM), 1)
    gated_kernel(const __grid_constant__ CUtensorMap gate_map, const __grid_constant__ CUtensorMap up_map,
                 const __grid_constant__ CUtensorMap col_map, const GatedParams p) {
  constexpr bool PAIR = FORM == Form::kPair, SPLIT = FORM == Form::kSplit, DUAL = dual(KIND);
  constexpr bool CHUNKED = KIND == Kind::kGradSums;
  constexpr int EPI = epi_warps(FORM);
  constexpr int LANE_BYTES = DUAL ? 2 * kTileBytes : kTileBytes;
  extern __shared__ __align__(1024) uint8_t ring[];
  const int col_rows = PAIR ? p.bn / 2 : p.bn;
  const int stage_bytes = LANE_BYTES + col_rows * 128;
  Barriers &b = *reinterpret_cast<Barriers *>(ring + p.stages * stage_bytes);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
  const int rank = FORM != Form::kOne ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = SPLIT ? static_cast<int>(blockIdx.x) / p.splits
                          : PAIR ? static_cast<int>(blockIdx.x) / 2 : static_cast<int>(blockIdx.x);
  const int step = SPLIT ? p.tiles : PAIR ? static_cast<int>(gridDim.x) / 2 : static_cast<int>(gridDim.x);
  const int lane_rank = PAIR ? rank : 0;
  const int k_begin = SPLIT ? static_cast<int>(static_cast<int64_t>(p.blocks) * rank / p.splits) : 0;
  const int k_end = SPLIT ? static_cast<int>(static_cast<int64_t>(p.blocks) * (rank + 1) / p.splits) : p.blocks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&b.full[i], i == 0 && static_cast<int>(blockIdx.x) == p.withheld ? 2 : 1);
      mbar_init(&b.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.acc_full[i], 1);
      mbar_init(&b.acc_empty[i], PAIR ? 2 * EPI : EPI);
    }
    mbar_init(&b.drain, 1);
    b.abort = 0;
    fence_mbar_init();
    if (p.blocks > 0) {
      tma_prefetch_map(&gate_map);
      if (KIND != Kind::kWeight) tma_prefetch_map(&up_map);
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
      for (int kb = k_begin; kb < k_end; ++kb) {
        if (fills >= p.stages) ok = mbar_wait_warp(&b.empty[s], phase, p.wait_ns, abort, p.err);
        if (!ok) break;
        if (elect_one()) {
          uint8_t *const dst = ring + s * stage_bytes;
          // A pair's copies all count on CTA 0's barrier, which expects both.
          // (CTA 1's may be first: the phase still lacks CTA 0's arrival.)
          uint32_t bar = smem_u32(&b.full[s]);
          if (PAIR) bar = cluster_addr(bar, 0);
          if (!PAIR || rank == 0)
            mbar_arrive_expect_tx(&b.full[s], static_cast<uint32_t>(PAIR ? 2 * stage_bytes : stage_bytes));
          if constexpr (DUAL) {
            tma_load_3d<PAIR>(dst, &gate_map, kb * kBk, tile.lane0, 0, bar);
            tma_load_3d<PAIR>(dst + kTileBytes, &up_map, kb * kBk, tile.lane0, 0, bar);
            tma_load_3d<PAIR>(dst + LANE_BYTES, &col_map, kb * kBk, col0, 0, bar);
          } else if constexpr (KIND == Kind::kInput) {
            // The sum runs over n of the gate, then over n of the other projection.
            const int half = kb >= p.half_blocks ? 1 : 0, at = (kb - half * p.half_blocks) * kBk;
            const CUtensorMap *const map = half ? &up_map : &gate_map;
            tma_load_3d<PAIR>(dst, map, tile.lane0, at, 0, bar);
            tma_load_3d<PAIR>(dst + kBoxBytes, map, tile.lane0 + 64, at, 0, bar);
            tma_load_3d<PAIR>(dst + LANE_BYTES, &col_map, at, col0, half, bar);
          } else {
            tma_load_3d<PAIR>(dst, &gate_map, tile.lane0, kb * kBk, 0, bar);
            tma_load_3d<PAIR>(dst + kBoxBytes, &gate_map, tile.lane0 + 64, kb * kBk, 0, bar);
            for (int j = 0; j < col_rows; j += 64)
              tma_load_3d<PAIR>(dst + LANE_BYTES + j * 128, &col_map, col0 + j, kb * kBk, tile.group, bar);
          }
        }
        __syncwarp();
        ++fills;
        if (++s == p.stages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    // No copy outlives the CTA, whatever the other warps did: also where all of them are issued
    // and the products give up.  (Of a pair, CTA 0's barriers count both CTAs' copies, and CTA 1
    // stays until CTA 0 leaves.)
    if (!PAIR || rank == 0) {
      for (int f = fills > p.stages ? fills - p.stages : 0; f < fills; ++f)
        if (!mbar_drain(&b.full[f % p.stages], (f / p.stages) & 1, p.wait_ns, p.err)) break;
    } else if (!ok) {  // CTA 0 may not have come as far: time enough for any copy
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 10000000ull) __nanosleep(1000);
    }
  } else if (warp == 1) {
    if (!PAIR || rank == 0) {
      int s = 0, turns = 0;  // stages; halves of the tensor memory, filled in turn
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t ring_a = smem_u32(ring);
      for (int t = first; t < p.tiles && ok; t += step) {
        int kb = k_begin;
        do {  // a tile, or (CHUNKED) kSumBlocks of its blocks
          const int half = turns & 1, begin = kb, end = CHUNKED ? min(kb + kSumBlocks, k_end) : k_end;
          if (turns >= 2) ok = mbar_wait_warp(&b.acc_empty[half], ((turns >> 1) - 1) & 1, p.wait_ns, abort, p.err);
          tcgen05_fence_after();
          const uint32_t d = tmem + static_cast<uint32_t>(half * (p.tmem_cols / 2));
          for (; kb < end && ok; ++kb) {
            ok = mbar_wait_warp(&b.full[s], phase, p.wait_ns, abort, p.err);
            if (!ok) break;
            tcgen05_fence_after();
            const uint32_t at = ring_a + s * stage_bytes;
            const uint64_t a = DUAL ? smem_desc_k128(at) : smem_desc_mn128(at);
            const uint64_t c = KIND == Kind::kWeight ? smem_desc_mn128(at + LANE_BYTES) : smem_desc_k128(at + LANE_BYTES);
            constexpr int A_STEP = DUAL ? 2 : 128, C_STEP = KIND == Kind::kWeight ? 128 : 2;  // 16 further in the sum
            if (elect_one()) {
#pragma unroll
              for (int i = 0; i < kBk / 16; ++i) {
                tcgen05_mma_f16<PAIR>(d, a + A_STEP * i, c + C_STEP * i, p.idesc, kb > begin || i > 0);
                if (DUAL)
                  tcgen05_mma_f16<PAIR>(d + p.tmem_cols / 4, a + (kTileBytes >> 4) + A_STEP * i, c + C_STEP * i, p.idesc,
                                        kb > begin || i > 0);
              }
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
          ++turns;
        } while (kb < k_end && ok);
      }
      if (!ok) {  // products in flight end before the tensor memory is given back
        if (elect_one()) tcgen05_commit<PAIR>(&b.drain);
        mbar_drain(&b.drain, 0, p.wait_ns, p.err);
      }
    }
  } else if (CHUNKED && warp >= 4) {
    const int e = warp - 4, c = e / 4 * 16;
    int turns = 0;
    bool ok = true;
    for (int t = first; t < p.tiles && ok; t += step) {
      const Tile tile = tile_at(p, t, lane_rank);
      float sa[16], sb[16];
      T grad[2][8];
      const int cols = min(p.bn, p.rows - tile.col0) - c;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sa[8 * h + j] = sb[8 * h + j] = 0.0f;
          grad[h][j] = from_f32<T>(0.0f);
        }
        if (8 * h < cols)
          grad_rows<T>(p, grad[h], static_cast<int64_t>(tile.col0) + c + 8 * h, min(8, cols - 8 * h),
                       tile.lane0 + 32 * (e % 4) + static_cast<int>(threadIdx.x % 32));
      }
      int kb = k_begin;
      do {
        const int half = turns & 1;
        // One decision per warp: tensor memory loads are executed by whole warps.
        ok = mbar_wait_warp(&b.acc_full[half], (turns >> 1) & 1, p.wait_ns, abort, p.err);
        if (!ok) break;
        tcgen05_fence_after();
        const uint32_t acc = tmem + static_cast<uint32_t>(half * (p.tmem_cols / 2) + c) + (static_cast<uint32_t>(32 * (e % 4)) << 16);
        if (c < p.bn && p.blocks > 0) {
          uint32_t r[16];
          tmem_ld16(acc, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) sa[j] += __uint_as_float(r[j]);
          tmem_ld16(acc + p.tmem_cols / 4, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) sb[j] += __uint_as_float(r[j]);
        }
        tcgen05_fence_before();
        __syncwarp();
        if (threadIdx.x % 32 == 0) {
          if (PAIR && rank != 0) {
            mbar_arrive_cluster(cluster_addr(smem_u32(&b.acc_empty[half]), 0));
          } else {
            mbar_arrive(&b.acc_empty[half]);
          }
        }
        ++turns;
        kb += kSumBlocks;
      } while (kb < k_end);
      if (ok) held_epilogue_act<T>(p, tile, e, sa, sb, grad);
    }
  } else if (warp >= 4) {
    const int e = warp - 4;
    int tiles = 0;
    for (int t = first; t < p.tiles; t += step, ++tiles) {
      const Tile tile = tile_at(p, t, lane_rank);
      const int half = tiles & 1;
      T grad[8];
      if constexpr (KIND == Kind::kGrads) {
#pragma unroll
        for (int j = 0; j < 8; ++j) grad[j] = from_f32<T>(0.0f);
        const int c = e / 4 * 8, cols = min(p.bn, p.rows - tile.col0);
        if (c < cols)
          grad_rows<T>(p, grad, static_cast<int64_t>(tile.col0) + c, min(8, cols - c),
                       tile.lane0 + 32 * (e % 4) + static_cast<int>(threadIdx.x % 32));
      }
      // One decision per warp: tensor memory loads are executed by whole warps.
      if (!mbar_wait_warp(&b.acc_full[half], (tiles >> 1) & 1, p.wait_ns, abort, p.err)) break;
      tcgen05_fence_after();
      const uint32_t acc = tmem + static_cast<uint32_t>(half * (p.tmem_cols / 2));
      if (SPLIT) {
        // Products are complete: the ring is free to hold the partial sums.
        float *const partial = reinterpret_cast<float *>(ring);
        const int lane = 32 * (e % 4) + static_cast<int>(threadIdx.x % 32);
        for (int c = e / 4 * 16; c < (DUAL ? 2 : 1) * p.bn; c += EPI / 4 * 16) {
          uint32_t r[16];
          const int at = c < p.bn ? c : p.tmem_cols / 4 + c - p.bn;  // the other projection's sums
          tmem_ld16(acc + (static_cast<uint32_t>(32 * (e % 4)) << 16) + at, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) partial[(c + j) * kLanes + lane] = __uint_as_float(r[j]);
        }
      } else {
        if constexpr (CHUNKED) {
        } else if constexpr (DUAL) {
          dual_epilogue_act<T, KIND>(p, tile, acc, e, grad);
        } else {
          plain_epilogue<T, KIND>(p, tile, acc, e);
        }
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

  __syncwarp();
  if (SPLIT) {
    __syncthreads();
    cluster_sync_all();
    if (!*abort && first < p.tiles)
      finish_split<T, KIND>(p, tile_at(p, first, 0), smem_u32(ring), rank, threadIdx.x, threads_of(FORM));
    cluster_sync_all();  // no CTA leaves while another reads its sums
  }
  tcgen05_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort) atomicOr(&g_gated_error, kErrMbarTimeout);
  if (PAIR) cluster_sync_all();  // ... or its barriers and tensor memory are in use
  if (warp == 2) {
    tcgen05_fence_after();
    tmem_dealloc<PAIR>(tmem, static_cast<uint32_t>(p.tmem_cols));
  }
}

// Joins the tiles' sums of da and db: a CTA has 32 columns, its warps every eighth part; then the warps in their order.
template <typename T>
__global__ void __launch_bounds__(256) columns_kernel(const float *columns, int parts, int64_t n, void *dbg, void *dbu,
                                                      int f32) {
  __shared__ float sums[8][32];
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (i < 2 * n) {
#pragma unroll 8
    for (int c = warp; c < parts; c += 8) s += columns[static_cast<int64_t>(c) * 2 * n + i];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || i >= 2 * n) return;
  void *const to = i < n ? dbg : dbu;
  if (!to) return;
  s = 0.0f;
#pragma unroll
  for (int c = 0; c < 8; ++c) s += sums[c][lane];
  const int64_t at = i < n ? i : i - n;
  if (f32) {
    static_cast<float *>(to)[at] = s;
  } else {
    static_cast<T *>(to)[at] = from_f32<T>(s);
  }
}

inline int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

lm_status check(const lm_gated_args *a) {
  if (!a || a->rows < 0 || a->k < 0 || a->n < 0 || a->x_row_stride < 0 || a->gate_row_stride < 0 ||
      a->up_row_stride < 0 || a->out_row_stride < 0)
    return LM_ERR_INVALID_ARG;
  if (a->activation < LM_ACT_NONE || a->activation > LM_ACT_SIGMOID) return LM_ERR_INVALID_ARG;
  if (a->dtype != LM_F16 && a->dtype != LM_BF16) return LM_ERR_UNSUPPORTED;
  if ((a->b_gate || a->b_up) && a->bias_dtype != LM_F32 && a->bias_dtype != a->dtype) return LM_ERR_UNSUPPORTED;
  const int64_t most = INT_MAX - 512;
  if (a->rows > most || a->n > most / 2 || a->k > most) return LM_ERR_UNSUPPORTED;
  for (const int64_t s : {a->x_row_stride, a->gate_row_stride, a->up_row_stride, a->out_row_stride})
    if (s > (1ll << 38)) return LM_ERR_UNSUPPORTED;
  return LM_OK;
}

lm_status check_pointers(const lm_gated_args &a, const void *workspace) {
  if (a.k > 0 && (!a.x || !a.w_gate || !a.w_up)) return LM_ERR_INVALID_ARG;
  const size_t bias = a.bias_dtype == LM_F32 ? 4 : 2;
  if (!aligned(a.x, 2) || !aligned(a.w_gate, 2) || !aligned(a.w_up, 2) || !aligned(a.b_gate, bias) ||
      !aligned(a.b_up, bias) || !aligned(workspace, 16))
    return LM_ERR_MISALIGNED;
  return LM_OK;
}

bool meets_inputs(const lm_gated_args &a, ByteRows out) {
  const int64_t bias = a.bias_dtype == LM_F32 ? 4 : 2;
  return (a.k > 0 && (rows_meet(out, {a.x, a.rows, a.x_row_stride * 2, a.k * 2}) ||
                      rows_meet(out, {a.w_gate, a.n, a.gate_row_stride * 2, a.k * 2}) ||
                      rows_meet(out, {a.w_up, a.n, a.up_row_stride * 2, a.k * 2}))) ||
         (a.b_gate && rows_meet(out, {a.b_gate, 1, 0, a.n * bias})) ||
         (a.b_up && rows_meet(out, {a.b_up, 1, 0, a.n * bias}));
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const GatedParams);

template <typename T, Kind KIND>
Kernel kernel_of(Form form) {
  if constexpr (KIND == Kind::kGrads || KIND == Kind::kGradSums) {  // (a tile's sums over rows stay with one CTA)
    return form == Form::kPair ? gated_kernel<T, Form::kPair, KIND> : gated_kernel<T, Form::kOne, KIND>;
  } else {
    return form == Form::kSplit ? gated_kernel<T, Form::kSplit, KIND>
           : form == Form::kPair ? gated_kernel<T, Form::kPair, KIND> : gated_kernel<T, Form::kOne, KIND>;
  }
}

struct Cut {
  Form form;
  int bn, splits;
  int64_t tiles;
};

// Columns of a tile, at least: sums over rows take space by the tile.
int narrowest(Kind kind, int64_t rows) { return kind == Kind::kGradSums && rows > 1024 ? 64 : 16; }

// The cut with the least estimated time, in microseconds: linear.cu's model, with the tile of the second
// projection where there is one, and this kernel's epilogues.  Of 120 problems (5 to 1000 rows, k and n of 512 to 8192,
// all kinds) its choice is within 10% of the best of all cuts, of nine in ten within 5%.
Cut best_cut(Kind kind, int64_t n, int64_t rows, int64_t groups, int64_t blocks, int sms, const Resident &held) {
  Cut best = {Form::kOne, kind == Kind::kWeight ? 64 : 16, 1, 0};
  float least = 3.0e38f;
  const bool grads = kind == Kind::kGrads || kind == Kind::kGradSums, forward = kind == Kind::kForward;
  const float column = grads ? 0.035f : forward ? 0.02f : 0.0085f;
  const float sums = dual(kind) ? 2.0f : 1.0f;
  auto consider = [&](Form form, int bn, int splits) {
    const bool two = form == Form::kPair;
    const int64_t lanes = two ? 2 * kLanes : kLanes;
    const int64_t tiles = up(n, lanes) * up(rows, bn) * groups;
    const int64_t at_once = two ? held.pairs : splits > 1 ? held.split[splits] : sms;
    if (splits > 1 && tiles > at_once) return;
    const int64_t rounds = up(tiles, at_once);
    const int64_t each = up(blocks, splits);
    const float kb = 16.0f * sums + static_cast<float>(bn) / (two ? 16.0f : 8.0f);  // KB of a stage
    const float bytes = kb / (forward && !two ? 150.0f : 185.0f), stage = bytes > 0.13f ? bytes : 0.13f;
    float t = (forward ? (two ? 3.4f : 2.7f) : two ? 4.2f : 3.0f) + static_cast<float>(each) * stage;
    if (splits > 1) {
      t += (forward ? 0.9f + 0.15f * static_cast<float>(splits) : 0.9f) + sums * (0.03f * static_cast<float>(bn) / static_cast<float>(splits) +
                                             (forward ? 0.016f : 0.008f) * static_cast<float>(bn));
    } else {
      t += (forward && two ? 0.03f : column) * static_cast<float>(bn);
    }
    if (rounds > 1) {
      const float products = 0.0011f * sums * static_cast<float>(bn), feed = kb / 140.0f;
      const float main = static_cast<float>(each) * (products > feed ? products : feed);
      const float epi = 0.5f + column * static_cast<float>(bn);
      t += static_cast<float>(rounds - 1) * (main > epi ? main : epi);
    }
    if (t < least) {
      least = t;
      best = {form, bn, splits, tiles};
    }
  };
  auto forms = [&](int bn, int unit) {
    consider(Form::kOne, bn, 1);
    if (bn % (2 * unit) == 0) consider(Form::kPair, bn, 1);
    if (grads) return;
    for (int s = 2; s <= kMaxSplits && s <= blocks; s *= 2) consider(Form::kSplit, bn, s);
  };
  if (kind == Kind::kWeight) {  // whole boxes of 64 columns a CTA
    for (int bn = 64; bn <= 256; bn += 64)
      if (bn == 64 || bn - 64 < rows) forms(bn, 64);
    return best;
  }
  // Both sums twice, or one twice, in 512 columns of tensor memory; or 16 columns a warp's lanes hold in registers.
  const int widest = kind == Kind::kGradSums ? 64 : dual(kind) ? 128 : 256;
  const int most = rows < widest ? static_cast<int>(up(rows, 16) * 16) : widest;
  for (int bn = narrowest(kind, rows); bn <= most; bn += bn < 64 ? 16 : 32) forms(bn, 16);
  const int64_t shares = up(rows, widest);
  forms(static_cast<int>(up(up(rows, shares), 16) * 16), 16);
  return best;
}

// What the four products share.
struct Launch {
  DeviceInfo dev;
  Resident held;
  uint32_t *err;
  const WaitFault *fault;
  cudaStream_t stream;
  bool bf16;
};

// One product: `lanes`, and for two projections `lanes2`, against `cols`; `sum` elements of the
// summed index in each operand, twice of it for Kind::kInput.
template <typename T, Kind KIND>
lm_status run(const Launch &l, GatedParams p, int64_t groups, const Operand &lanes, const Operand &lanes2,
              const Operand &cols, int64_t sum) {
  const int64_t half = up(sum, kBk), blocks = KIND == Kind::kInput ? 2 * half : half;
  if (blocks > INT_MAX / 2) return LM_ERR_UNSUPPORTED;
  p.half_blocks = static_cast<int32_t>(half);
  p.blocks = static_cast<int32_t>(blocks);
  const Cut cut = best_cut(KIND, p.n, p.rows, groups, blocks, l.dev.sm_count, l.held);
  if (cut.tiles > INT_MAX / 16) return LM_ERR_UNSUPPORTED;
  p.bn = cut.bn;
  p.splits = cut.splits;
  p.tiles = static_cast<int32_t>(cut.tiles);
  p.lane_step = cut.form == Form::kPair ? 2 * kLanes : kLanes;
  p.lane_tiles = static_cast<int32_t>(up(p.n, p.lane_step));
  p.col_tiles = static_cast<int32_t>(up(p.rows, p.bn));
  p.lanes_inside = p.n <= p.rows;
  p.tmem_cols = 32;
  while (p.tmem_cols < (dual(KIND) ? 4 : 2) * p.bn) p.tmem_cols *= 2;
  const int held_cols = cut.form == Form::kPair ? p.bn / 2 : p.bn;
  const int stage_bytes = (dual(KIND) ? 2 : 1) * kTileBytes + held_cols * 128;
  p.stages = (227 * 1024 - static_cast<int>(sizeof(Barriers))) / stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.idesc = idesc_f16(l.bf16, static_cast<uint32_t>(p.lane_step), static_cast<uint32_t>(p.bn)) |
            (dual(KIND) ? 0 : kIdescMnA) | (KIND == Kind::kWeight ? kIdescMnB : 0);
  p.err = l.err;
  p.wait_ns = l.fault ? l.fault->wait_ns : kWaitTimeoutNs;
  p.withheld = l.fault ? static_cast<int32_t>(l.fault->withheld_cta) : -1;
  const int smem = p.stages * stage_bytes + static_cast<int>(sizeof(Barriers));
  CUtensorMap a = {}, b = {}, c = {};
  if (blocks > 0) {
    // Tiles of the lanes: 128 rows by 64 of the sum, or boxes of 64 lanes by 64 of the sum.
    const int64_t wide = dual(KIND) ? sum : p.n;
    const int box = dual(KIND) ? kLanes : kBk;
    if (lm_status st = make_map(&a, lanes, wide, box, l.bf16); st != LM_OK) return st;
    if (KIND != Kind::kWeight)
      if (lm_status st = make_map(&b, lanes2, wide, box, l.bf16); st != LM_OK) return st;
    if (lm_status st = KIND == Kind::kWeight ? make_map(&c, cols, p.rows, kBk, l.bf16)
                                             : make_map(&c, cols, sum, held_cols, l.bf16);
        st != LM_OK)
      return st;
  }
  const Kernel kernel = kernel_of<T, KIND>(cut.form);
  if (lm_status st = ensure_smem_attribute(reinterpret_cast<const void *>(kernel), smem); st != LM_OK) return st;
  int cluster = 1, grid = p.tiles < l.dev.sm_count ? p.tiles : l.dev.sm_count;
  if (cut.form == Form::kSplit) {
    cluster = p.splits;
    grid = p.tiles * p.splits;
  } else if (cut.form == Form::kPair) {
    cluster = 2;
    grid = 2 * (p.tiles < l.held.pairs ? p.tiles : l.held.pairs);
  }
  return launch_dependent(kernel, dim3(static_cast<unsigned>(grid)), threads_of(cut.form), static_cast<size_t>(smem),
                          l.stream, cluster, a, b, c, p);
}

// The inputs as the kernels fetch them, and where copies of them, the gradients and (columns) the tiles' sums of
// them lie in the workspace.
struct Plan {
  Operand x, gate, up_;
  size_t pitch;          // elements a row of da and db
  size_t copies, grads, bytes;
};

size_t padded(size_t n) { return (n + 255) / 256 * 256; }

Plan plan(const lm_gated_args &a, bool backward = false, bool columns = false) {
  Plan p = {};
  p.x = operand(a.x, 1, a.rows, a.k, 0, a.x_row_stride);
  p.gate = operand(a.w_gate, 1, a.n, a.k, 0, a.gate_row_stride);
  p.up_ = operand(a.w_up, 1, a.n, a.k, 0, a.up_row_stride);
  p.copies = 256;
  p.grads = p.copies + padded(p.x.bytes) + padded(p.gate.bytes) + padded(p.up_.bytes);
  p.bytes = p.grads;
  if (backward) {
    p.pitch = static_cast<size_t>(up(a.n, 8) * 8);
    p.bytes += padded(static_cast<size_t>(a.rows) * p.pitch * 4);
  }
  if (columns)
    p.bytes += static_cast<size_t>(up(a.rows, narrowest(Kind::kGradSums, a.rows)) * kColumnParts) * 8 *
               static_cast<size_t>(a.n);
  return p;
}

Plan plan(const lm_gated_backward_args &a) { return plan(a.forward, true, a.db_gate || a.db_up); }

template <typename T>
GatedParams params(const lm_gated_args &a) {
  GatedParams p = {};
  p.bg = a.b_gate;
  p.bu = a.b_up;
  p.rows = static_cast<int32_t>(a.rows);
  p.n = static_cast<int32_t>(a.n);
  p.bias_f32 = a.bias_dtype == LM_F32;
  p.act = a.activation;
  return p;
}

lm_status start(const lm_gated_args &a, Plan *pl, void *workspace, const WaitFault *fault, cudaStream_t s, Launch *l) {
  if (lm_status st = current_device_info(&l->dev); st != LM_OK) return st;
  if (lm_status st = resident_clusters(l->dev, &l->held); st != LM_OK) return st;
  l->err = static_cast<uint32_t *>(workspace);
  l->fault = fault;
  l->stream = s;
  l->bf16 = a.dtype == LM_BF16;
  Operand *const operands[3] = {&pl->x, &pl->gate, &pl->up_};
  return pack_three(operands, a.k, static_cast<char *>(workspace) + pl->copies, s);
}

template <typename T>
lm_status forward(const lm_gated_args &a, Plan pl, void *workspace, const WaitFault *fault, cudaStream_t s) {
  Launch l;
  if (lm_status st = start(a, &pl, workspace, fault, s, &l); st != LM_OK) return st;
  GatedParams p = params<T>(a);
  p.out[0] = a.out;
  p.out_row = a.out_row_stride;
  return run<T, Kind::kForward>(l, p, 1, pl.gate, pl.up_, pl.x, a.k);
}

template <typename T>
lm_status backward(const lm_gated_backward_args &a, Plan pl, void *workspace, const WaitFault *fault, cudaStream_t s) {
  const lm_gated_args &f = a.forward;
  const int64_t size = f.bias_dtype == LM_F32 ? 4 : 2;
  if (f.rows == 0 || f.n == 0) {  // sums of nothing
    if (a.dx && f.rows > 0) LM_CUDA_TRY(cudaMemsetAsync(a.dx, 0, static_cast<size_t>(f.rows * f.k) * 2, s));
    for (void *const w : {a.dw_gate, a.dw_up})
      if (w && f.n > 0) LM_CUDA_TRY(cudaMemsetAsync(w, 0, static_cast<size_t>(f.n * f.k) * 2, s));
    for (void *const b : {a.db_gate, a.db_up})
      if (b && f.n > 0) LM_CUDA_TRY(cudaMemsetAsync(b, 0, static_cast<size_t>(f.n * size), s));
    return LM_OK;
  }
  Launch l;
  if (lm_status st = start(f, &pl, workspace, fault, s, &l); st != LM_OK) return st;
  T *const da = reinterpret_cast<T *>(static_cast<char *>(workspace) + pl.grads);
  const int64_t plane = f.rows * static_cast<int64_t>(pl.pitch);
  float *const columns = reinterpret_cast<float *>(static_cast<char *>(workspace) + pl.grads +
                                                   padded(static_cast<size_t>(plane) * 4));
  GatedParams p = params<T>(f);
  p.out[0] = da;
  p.out[1] = da + plane;
  p.out_row = static_cast<int64_t>(pl.pitch);
  p.grad = a.grad;
  p.grad_row = a.grad_row_stride;
  p.columns = a.db_gate || a.db_up ? columns : nullptr;
  // (A layer with biases takes it whichever gradients are wanted: each has the same bits then.)
  if (lm_status st = p.columns || f.b_gate || f.b_up
                         ? run<T, Kind::kGradSums>(l, p, 1, pl.gate, pl.up_, pl.x, f.k)
                         : run<T, Kind::kGrads>(l, p, 1, pl.gate, pl.up_, pl.x, f.k);
      st != LM_OK)
    return st;
  const Operand both{da, 2, f.rows, plane, static_cast<int64_t>(pl.pitch), false, 0};
  if (a.dx && f.k > 0) {
    GatedParams q = {};
    q.rows = static_cast<int32_t>(f.rows);
    q.n = static_cast<int32_t>(f.k);
    q.out[0] = a.dx;
    q.out_row = f.k;
    if (lm_status st = run<T, Kind::kInput>(l, q, 1, pl.gate, pl.up_, both, f.n); st != LM_OK) return st;
  }
  if ((a.dw_gate || a.dw_up) && f.k > 0) {
    GatedParams q = {};
    q.rows = static_cast<int32_t>(f.n);
    q.n = static_cast<int32_t>(f.k);
    q.out[0] = a.dw_gate;
    q.out[1] = a.dw_up;
    q.out_row = f.k;
    q.first_group = a.dw_gate ? 0 : 1;
    const int64_t groups = a.dw_gate && a.dw_up ? 2 : 1;
    if (lm_status st = run<T, Kind::kWeight>(l, q, groups, pl.x, pl.x, both, f.rows); st != LM_OK) return st;
  }
  if (p.columns) {
    const Cut cut = best_cut(Kind::kGradSums, f.n, f.rows, 1, up(f.k, kBk), l.dev.sm_count, l.held);
    const int parts = static_cast<int>(up(f.rows, cut.bn)) * kColumnParts;
    return launch_dependent(columns_kernel<T>, dim3(static_cast<unsigned>(up(2 * f.n, 32))), 256, 0, s, 1,
                            static_cast<const float *>(columns), parts, f.n, a.db_gate, a.db_up, p.bias_f32);
  }
  return LM_OK;
}

lm_status run_forward(const lm_gated_args *args, void *workspace, size_t workspace_bytes, cudaStream_t s,
                      const WaitFault *fault) {
  if (lm_status st = check(args); st != LM_OK) return st;
  const lm_gated_args &a = *args;
  if (a.rows == 0 || a.n == 0) return LM_OK;
  if (!a.out) return LM_ERR_INVALID_ARG;
  if (lm_status st = check_pointers(a, workspace); st != LM_OK) return st;
  if (!aligned(a.out, 2)) return LM_ERR_MISALIGNED;
  const Plan pl = plan(a);
  if (!workspace || workspace_bytes < pl.bytes) return LM_ERR_WORKSPACE;
  if ((a.rows > 1 && a.out_row_stride < a.n) || meets_inputs(a, {a.out, a.rows, a.out_row_stride * 2, a.n * 2}))
    return LM_ERR_INVALID_ARG;
  return a.dtype == LM_F16 ? forward<__half>(a, pl, workspace, fault, s)
                           : forward<__nv_bfloat16>(a, pl, workspace, fault, s);
}

lm_status run_backward(const lm_gated_backward_args *args, void *workspace, size_t workspace_bytes, cudaStream_t s,
                       const WaitFault *fault) {
  size_t need = 0;
  if (lm_status st = lm_gated_linear_backward_workspace_size(args, &need); st != LM_OK) return st;
  const lm_gated_backward_args &a = *args;
  const lm_gated_args &f = a.forward;
  void *const outs[] = {a.dx, a.dw_gate, a.dw_up, a.db_gate, a.db_up};
  const int64_t bias = f.bias_dtype == LM_F32 ? 4 : 2;
  const int64_t sizes[] = {f.rows * f.k * 2, f.n * f.k * 2, f.n * f.k * 2, f.n * bias, f.n * bias};
  bool any = false;
  for (int i = 0; i < 5; ++i) any = any || (outs[i] && sizes[i] > 0);
  if (!any) return LM_OK;
  if (f.rows > 0 && f.n > 0) {
    if (!a.grad) return LM_ERR_INVALID_ARG;
    if (lm_status st = check_pointers(f, workspace); st != LM_OK) return st;
  }
  if ((a.db_gate || a.db_up) && f.bias_dtype != LM_F32 && f.bias_dtype != f.dtype) return LM_ERR_UNSUPPORTED;
  for (int i = 0; i < 5; ++i)
    if (!aligned(outs[i], i < 3 ? 2 : static_cast<size_t>(bias))) return LM_ERR_MISALIGNED;
  if (!aligned(a.grad, 2) || !aligned(workspace, 16)) return LM_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < need) return LM_ERR_WORKSPACE;
  for (int i = 0; i < 5; ++i) {
    if (!outs[i]) continue;
    const ByteRows out{outs[i], 1, 0, sizes[i]};
    if (meets_inputs(f, out) || rows_meet(out, {a.grad, f.rows, a.grad_row_stride * 2, f.n * 2})) return LM_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (outs[j] && rows_meet(out, {outs[j], 1, 0, sizes[j]})) return LM_ERR_INVALID_ARG;
  }
  const Plan pl = plan(a);
  return f.dtype == LM_F16 ? backward<__half>(a, pl, workspace, fault, s)
                           : backward<__nv_bfloat16>(a, pl, workspace, fault, s);
}

}  // namespace

lm_status gated_error(uint32_t *value, bool clear, cudaStream_t s) { return read_sticky(g_gated_error, value, clear, s); }

}  // namespace lm

extern "C" lm_status lm_gated_linear_workspace_size(const lm_gated_args *args, size_t *bytes) {
  if (!bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::check(args); st != LM_OK) return st;
  *bytes = lm::plan(*args).bytes;
  return LM_OK;
}

extern "C" lm_status lm_gated_linear(const lm_gated_args *args, void *workspace, size_t workspace_bytes,
                                     lm_stream_t stream) {
  return lm::run_forward(args, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream), nullptr);
}

extern "C" lm_status lm_gated_linear_backward_workspace_size(const lm_gated_backward_args *args, size_t *bytes) {
  if (!args || !bytes || args->grad_row_stride < 0) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::check(&args->forward); st != LM_OK) return st;
  if (args->grad_row_stride > (1ll << 38)) return LM_ERR_UNSUPPORTED;
  *bytes = lm::plan(*args).bytes;
  return LM_OK;
}

extern "C" lm_status lm_gated_linear_backward(const lm_gated_backward_args *args, void *workspace,
                                              size_t workspace_bytes, lm_stream_t stream) {
  return lm::run_backward(args, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream), nullptr);
}

extern "C" lm_status lm_debug_gated_linear_withhold(const lm_gated_args *args, void *workspace, size_t workspace_bytes,
                                                    int64_t withheld_cta, uint64_t wait_ns, lm_stream_t stream) {
  if (withheld_cta < 0 || withheld_cta > INT_MAX || wait_ns < 100000ull || wait_ns > lm::kWaitTimeoutNs)
    return LM_ERR_INVALID_ARG;
  const lm::WaitFault fault{withheld_cta, wait_ns};
  return lm::run_forward(args, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream), &fault);
}

extern "C" lm_status lm_debug_gated_linear_backward_withhold(const lm_gated_backward_args *args, void *workspace,
                                                             size_t workspace_bytes, int64_t withheld_cta,
                                                             uint64_t wait_ns, lm_stream_t stream) {
  if (withheld_cta < 0 || withheld_cta > INT_MAX || wait_ns < 100000ull || wait_ns > lm::kWaitTimeoutNs)
    return LM_ERR_INVALID_ARG;
  const lm::WaitFault fault{withheld_cta, wait_ns};
  return lm::run_backward(args, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream), &fault);
}
