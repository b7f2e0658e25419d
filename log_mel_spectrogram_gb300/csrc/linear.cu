// linear.cu -- y = residual + scale * act(x W^T + bias) on the tensor cores.
//
// A CTA computes tiles of 128 outputs (rows of W, along the lanes of tensor
// memory) by bn rows of x: one warp fetches 128 x 64 and bn x 64 operand tiles
// by TMA into a ring of shared-memory stages, one warp issues tcgen05.mma into
// tensor memory (32-bit sums), sixteen turn a finished tile into outputs while
// the next one is summed into the other half of the tensor memory.  CTAs are
// persistent: one per SM walks the tiles.
//
// With W along the lanes, bn is any multiple of 16 up to 256, so that few rows
// of x waste no products and the tiles of a medium problem can be cut to fill the
// SMs once; and the lanes of a warp are consecutive outputs of a row, so that
// stores are whole, whatever the row length's alignment.  (The other way round,
// with outputs leaving by TMA, was equal at 24000 x 1024 x 4096 and up to 45%
// slower between 100 and 6000 rows.)
//
// Three forms, chosen with bn by the estimate in best_cut():
//  - a CTA per tile;
//  - a pair of CTAs per tile of 256 lanes (cta_group::2): each fetches half of
//    the rows of x and both use them, a third less traffic from L2, which is
//    what bounds large problems (8192^3, calls in a row: 1.48 -> 1.65 PFLOP/s);
//  - a cluster of 2 to 8 CTAs per tile, each with a part of k, for the few tiles
//    of a decoding step: the partial sums meet in distributed shared memory in
//    rank order, in the same launch and with the same result on every call (5 x
//    1024 x 1024 in a graph: a CTA a tile 4.8 us, clusters of two 4.6, of eight 4.0).
//
// The issuing warps stay converged up to one elected lane: addresses and
// descriptors then live in uniform registers, which the tensor instructions
// take.  Issued from one divergent thread, a product of 128 x 256 x 16 took 172
// to 237 cycles, in competition with the epilogue; now 130.
//
// Measured, calls in a row: 24000 x 1024 -> 4096 bf16 with bias and gelu 127 to 134
// us (1.50 to 1.58 PFLOP/s; the tensor pipe is active 92% of the time, at the clock that the
// power limit allows).
// 320 x 1024 -> 50001 34 to 35 us against 20 us of memory traffic; no unit is near its
// rate (tensor pipe 53%, L2 41%, DRAM half), and best_cut()'s model gives 23.  Off 16-byte
// boundaries (k = 1023) 74 us, most of it the copy of W.
// Windows of 8 x 3000 frames, 240 -> 512 with gelu, 13.3 us, without 10.9: four stages of
// k a tile, each tile fetching its part of W anew.  24000 x 1024 -> 1024 with a residual 42 us,
// without 37.  5 x 1024 -> 1024 4.6 to 5.9 us from the host, 4.0 in a graph: a launch, one load's
// latency and the cluster's exchange.
//
// Operands that TMA cannot address (rows off 16-byte boundaries) are first
// copied into padded rows in the workspace.
#include <atomic>
#include <climits>
#include <cuda.h>

#include "activate.cuh"
#include "f32x2.cuh"
#include "half.cuh"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "operand.cuh"
#include "pdl.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "waits.cuh"

namespace lm {
namespace {

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

__device__ uint32_t g_linear_error;  // bits of every call on the device, whatever its workspace

struct alignas(16) Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
};

template <typename T, Form FORM>
__global__ void __launch_bounds__(threads_of(FORM), 1)
    linear_kernel(const __grid_constant__ CUtensorMap lane_map, const __grid_constant__ CUtensorMap col_map,
                  const LinearParams p) {
  constexpr bool PAIR = FORM == Form::kPair, SPLIT = FORM == Form::kSplit;
  constexpr int EPI = epi_warps(FORM);
  extern __shared__ __align__(1024) uint8_t ring[];  // stages on a boundary of the swizzle's period
  const int col_rows = PAIR ? p.bn / 2 : p.bn;  // rows of the column side that this CTA holds
  const int stage_bytes = kLanes * 128 + col_rows * 128;
  Barriers &b = *reinterpret_cast<Barriers *>(ring + p.stages * stage_bytes);
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
          tma_load_3d<PAIR>(dst, &lane_map, kb * kBk, tile.lane0, 0, bar);
          tma_load_3d<PAIR>(dst + kLanes * 128, &col_map, kb * kBk, col0, tile.group, bar);
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
      int s = 0, tiles = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t ring_a = smem_u32(ring);
      for (int t = first; t < p.tiles && ok; t += step, ++tiles) {
        const int half = tiles & 1;
        if (tiles >= 2) ok = mbar_wait_warp(&b.acc_empty[half], ((tiles >> 1) - 1) & 1, p.wait_ns, abort, p.err);
        tcgen05_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(half * (p.tmem_cols / 2));
        for (int kb = k_begin; kb < k_end && ok; ++kb) {
          ok = mbar_wait_warp(&b.full[s], phase, p.wait_ns, abort, p.err);
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
        mbar_drain(&b.drain, 0, p.wait_ns, p.err);
      }
    }
  } else if (warp >= 4) {
    const int e = warp - 4;
    int tiles = 0;
    for (int t = first; t < p.tiles; t += step, ++tiles) {
      const Tile tile = tile_at(p, t, lane_rank);
      const int half = tiles & 1;
      T residual[16];
      if (!SPLIT && p.residual) {
#pragma unroll
        for (int j = 0; j < 16; ++j) residual[j] = from_f32<T>(0.0f);
        const int c = e / 4 * 16, cols = min(p.bn, p.rows - tile.col0);
        if (c < cols)
          residual_rows<T>(p, residual, static_cast<int64_t>(tile.group) * p.rows + tile.col0 + c, min(16, cols - c),
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
        for (int c = e / 4 * 16; c < p.bn; c += EPI / 4 * 16) {
          uint32_t r[16];
          tmem_ld16(acc + (static_cast<uint32_t>(32 * (e % 4)) << 16) + c, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) partial[(c + j) * kLanes + lane] = __uint_as_float(r[j]);
        }
      } else {
        if (p.residual) {
          epilogue_act<T, true, EPI>(p, tile, acc, e, residual);
        } else {
          epilogue_act<T, false, EPI>(p, tile, acc, e, residual);
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
    if (!*abort && first < p.tiles) {
      const Tile tile = tile_at(p, first, 0);
      finish_split_act<T>(p, tile, smem_u32(ring), rank, threadIdx.x, threads_of(FORM));
    }
    cluster_sync_all();  // no CTA leaves while another reads its sums
  }
  tcgen05_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort) atomicOr(&g_linear_error, kErrMbarTimeout);
  if (PAIR) cluster_sync_all();  // ... or its barriers and tensor memory are in use
  if (warp == 2) {
    tcgen05_fence_after();
    tmem_dealloc<PAIR>(tmem, static_cast<uint32_t>(p.tmem_cols));
  }
}

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

// Whether the output's rows run into one another or into an input.  (Equal to
// the residual it may be: an element is read before it is written.)
bool out_meets_inputs(const lm_linear_args &a, const Plan &p, int64_t out_size) {
  const int64_t rows = a.groups * a.rows;
  if (rows > 1 && a.out_row_stride < a.n) return true;
  const ByteRows out{a.out, rows, a.out_row_stride * out_size, a.n * out_size};
  auto input = [&](const Operand &o) {
    const ByteRows r{o.p, o.rows, o.row_stride * 2, a.k * 2};
    if (o.groups == 1) return r;
    return ByteRows{o.p, o.groups, o.group_stride * 2, (o.rows - 1) * r.step + r.size};
  };
  if (a.k > 0 && (rows_meet(out, input(p.x)) || rows_meet(out, input(p.w)))) return true;
  if (a.bias && rows_meet(out, {a.bias, 1, 0, a.n * (a.bias_dtype == LM_F32 ? 4 : 2)})) return true;
  const bool same = a.residual == a.out && out_size == 2 && (rows == 1 || a.residual_row_stride == a.out_row_stride);
  return a.residual && !same && rows_meet(out, {a.residual, rows, a.residual_row_stride * 2, a.n * 2});
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const LinearParams);

template <typename T>
Kernel kernel_of(Form form) {
  return form == Form::kSplit ? linear_kernel<T, Form::kSplit>
         : form == Form::kPair ? linear_kernel<T, Form::kPair> : linear_kernel<T, Form::kOne>;
}

// Asked once per device.  Two threads that ask together get the same answer.
constexpr int kKnownDevices = 64;
Resident g_resident[kKnownDevices];
std::atomic<int> g_resident_state[kKnownDevices];  // 0: not known, 1: being written, 2: known

lm_status ask_resident_clusters(const DeviceInfo &dev, Resident *r) {
  if (dev.device < kKnownDevices && g_resident_state[dev.device].load(std::memory_order_acquire) == 2) {
    *r = g_resident[dev.device];
    return LM_OK;
  }
  auto ask = [&](Kernel kernel, Form form, int size) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(dev.sm_count / size * size));
    cfg.blockDim = dim3(static_cast<unsigned>(threads_of(form)));
    cfg.dynamicSmemBytes = 128 * 1024;  // more than half an SM's
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(size);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      n = dev.sm_count / (2 * size);
    }
    return n < dev.sm_count / size ? n : dev.sm_count / size;
  };
  Resident a = {};
  const Kernel pair = kernel_of<__half>(Form::kPair), split = kernel_of<__half>(Form::kSplit);
  for (const Kernel k : {pair, split})
    if (lm_status st = ensure_smem_attribute(reinterpret_cast<const void *>(k), 128 * 1024); st != LM_OK) return st;
  a.pairs = ask(pair, Form::kPair, 2);
  for (int size = 2; size <= kMaxSplits; size *= 2) a.split[size] = ask(split, Form::kSplit, size);
  *r = a;
  int none = 0;
  if (dev.device < kKnownDevices && g_resident_state[dev.device].compare_exchange_strong(none, 1)) {
    g_resident[dev.device] = a;
    g_resident_state[dev.device].store(2, std::memory_order_release);
  }
  return LM_OK;
}

// How a problem is cut into tiles.
struct Cut {
  Form form;
  int bn, splits;
  int64_t tiles;
};

// The cut with the least estimated time, in microseconds.  The constants are
// fitted to 256 problems of 5 to 24000 rows, k of 256 to 4096 and 256 to 10000
// outputs; the estimate's choice was 0.6% slower than the best of all cuts in the
// geometric mean, and within 7% of it for 96 in 100.
//   first tile: 3, a stage's latency or its traffic at 185 KB/us for each block
//     of k, and the epilogue's 0.008 a column;
//   each further round of tiles: the most of traffic (140 KB/us per SM with all
//     of them fetching), products (0.0011 a column and block) and epilogue.
Cut best_cut(int64_t n, int64_t rows, int64_t groups, int kblocks, bool activation, int sms, const Resident &held) {
  Cut best = {Form::kOne, 16, 1, 0};
  float least = 3.0e38f;
  const float column = activation ? 0.0125f : 0.0085f;
  auto consider = [&](Form form, int bn, int splits) {
    const bool two = form == Form::kPair;
    const int64_t lanes = two ? 2 * kLanes : kLanes;
    const int64_t tiles = (n + lanes - 1) / lanes * ((rows + bn - 1) / bn) * groups;
    const int64_t at_once = two ? held.pairs : splits > 1 ? held.split[splits] : sms;
    if (splits > 1 && tiles > at_once) return;
    const int64_t rounds = (tiles + at_once - 1) / at_once;
    const int blocks = (kblocks + splits - 1) / splits;
    const float kb = 16.0f + static_cast<float>(bn) / (two ? 16.0f : 8.0f);  // KB of a stage
    const float stage = kb / 185.0f > 0.13f ? kb / 185.0f : 0.13f;
    float t = (two ? 4.2f : 3.0f) + static_cast<float>(blocks) * stage;
    if (splits > 1) {
      t += 0.9f + 0.03f * static_cast<float>(bn) / static_cast<float>(splits) + 0.008f * static_cast<float>(bn);
    } else {
      t += column * static_cast<float>(bn);
    }
    if (rounds > 1) {
      const float products = 0.0011f * static_cast<float>(bn), feed = kb / 140.0f;
      const float main = static_cast<float>(blocks) * (products > feed ? products : feed);
      const float epi = 0.5f + column * static_cast<float>(bn);
      t += static_cast<float>(rounds - 1) * (main > epi ? main : epi);
    }
    if (t < least) {
      least = t;
      best = {form, bn, splits, tiles};
    }
  };
  const int most = rows < kMaxBn ? static_cast<int>((rows + 15) / 16 * 16) : kMaxBn;
  for (int bn = 16; bn <= most; bn += bn < 64 ? 16 : 32) {
    consider(Form::kOne, bn, 1);
    if (bn % 32 == 0) consider(Form::kPair, bn, 1);
    for (int s = 2; s <= kMaxSplits && s <= kblocks; s *= 2) consider(Form::kSplit, bn, s);
  }
  // Exactly the rows there are, or equal shares of them.
  const int64_t shares = (rows + kMaxBn - 1) / kMaxBn;
  const int even = static_cast<int>(((rows + shares - 1) / shares + 15) / 16 * 16);
  consider(Form::kOne, even, 1);
  if (even % 32 == 0) consider(Form::kPair, even, 1);
  return best;
}

// lm_linear; `fault` is null outside tests.
lm_status run(const lm_linear_args *args, void *workspace, size_t workspace_bytes, cudaStream_t s,
              const WaitFault *fault) {
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
  if (out_meets_inputs(a, pl, static_cast<int64_t>(out_size))) return LM_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (lm_status st = current_device_info(&dev); st != LM_OK) return st;
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
  p.out_row = a.out_row_stride;
  p.res_row = a.residual_row_stride;
  p.rows = static_cast<int32_t>(pl.x.rows);
  p.n = static_cast<int32_t>(a.n);
  p.kblocks = static_cast<int32_t>((a.k + kBk - 1) / kBk);
  p.bias_f32 = a.bias_dtype == LM_F32;
  p.out_f32 = a.out_dtype == LM_F32;
  p.act = a.activation;
  p.scale = a.scale;
  p.err = static_cast<uint32_t *>(workspace);
  p.wait_ns = fault ? fault->wait_ns : kWaitTimeoutNs;
  p.withheld = fault ? static_cast<int32_t>(fault->withheld_cta) : -1;
  const bool bf16 = a.dtype == LM_BF16;

  Resident held;
  if (lm_status st = ask_resident_clusters(dev, &held); st != LM_OK) return st;
  const Cut cut = best_cut(p.n, p.rows, pl.x.groups, p.kblocks, p.act > LM_ACT_RELU, dev.sm_count, held);
  if (cut.tiles > INT_MAX / 16) return LM_ERR_UNSUPPORTED;
  p.bn = cut.bn;
  p.splits = cut.splits;
  p.tiles = static_cast<int32_t>(cut.tiles);
  p.lane_step = cut.form == Form::kPair ? 2 * kLanes : kLanes;
  p.lane_tiles = (p.n + p.lane_step - 1) / p.lane_step;
  p.col_tiles = (p.rows + p.bn - 1) / p.bn;
  // The smaller operand goes round inside, out of L2, the larger passes once.
  p.lanes_inside = p.n <= p.rows;
  p.tmem_cols = 32;
  while (p.tmem_cols < 2 * p.bn) p.tmem_cols *= 2;
  const int held_cols = cut.form == Form::kPair ? p.bn / 2 : p.bn;
  const int stage_bytes = kLanes * 128 + held_cols * 128;
  p.stages = (227 * 1024 - static_cast<int>(sizeof(Barriers))) / stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.idesc = idesc_f16(bf16, static_cast<uint32_t>(p.lane_step), static_cast<uint32_t>(p.bn));
  const int smem = p.stages * stage_bytes + static_cast<int>(sizeof(Barriers));

  CUtensorMap lanes = {}, cols = {};
  if (p.kblocks > 0) {
    if (lm_status st = make_map(&lanes, pl.w, a.k, kLanes, bf16); st != LM_OK) return st;
    if (lm_status st = make_map(&cols, pl.x, a.k, held_cols, bf16); st != LM_OK) return st;
  }
  const Kernel kernel = bf16 ? kernel_of<__nv_bfloat16>(cut.form) : kernel_of<__half>(cut.form);
  if (lm_status st = ensure_smem_attribute(reinterpret_cast<const void *>(kernel), smem); st != LM_OK) return st;
  int cluster = 1, grid = p.tiles < dev.sm_count ? p.tiles : dev.sm_count;
  if (cut.form == Form::kSplit) {
    cluster = p.splits;
    grid = p.tiles * p.splits;
  } else if (cut.form == Form::kPair) {
    cluster = 2;
    grid = 2 * (p.tiles < held.pairs ? p.tiles : held.pairs);
  }
  return launch_dependent(kernel, dim3(static_cast<unsigned>(grid)), threads_of(cut.form), static_cast<size_t>(smem), s,
                          cluster, lanes, cols, p);
}

}  // namespace

lm_status linear_check(const lm_linear_args *args) { return check(args); }

lm_status resident_clusters(const DeviceInfo &dev, Resident *r) { return ask_resident_clusters(dev, r); }

lm_status linear_error(uint32_t *value, bool clear, cudaStream_t s) { return read_sticky(g_linear_error, value, clear, s); }

}  // namespace lm

extern "C" lm_status lm_linear_workspace_size(const lm_linear_args *args, size_t *bytes) {
  if (!bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::check(args); st != LM_OK) return st;
  *bytes = lm::plan(*args).bytes;
  return LM_OK;
}

extern "C" lm_status lm_linear(const lm_linear_args *args, void *workspace, size_t workspace_bytes,
                               lm_stream_t stream) {
  return lm::run(args, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream), nullptr);
}

extern "C" lm_status lm_debug_linear_withhold(const lm_linear_args *args, void *workspace, size_t workspace_bytes,
                                              int64_t withheld_cta, uint64_t wait_ns, lm_stream_t stream) {
  if (withheld_cta < 0 || withheld_cta > INT_MAX || wait_ns < 100000ull || wait_ns > lm::kWaitTimeoutNs)
    return LM_ERR_INVALID_ARG;
  const lm::WaitFault fault{withheld_cta, wait_ns};
  return lm::run(args, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream), &fault);
}
