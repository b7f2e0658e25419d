// tcgen05.cuh -- inline PTX for the 5th-generation tensor cores and tiled TMA
// loads (sm_103a): tensor memory, matrix products issued by one thread, and
// the descriptors that they take.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace lm {

// One lane of a converged warp, the same one each time.  Code that issues
// products or copies runs on whole warps up to this point: addresses and
// descriptors then stay in the warp's uniform registers, which the
// instructions take their operands from.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// PAIR: the two CTAs of a cluster work on one tile (cta_group::2): tensor memory
// is taken and given back by both, products are issued by CTA 0 alone and read
// both shared memories, and each CTA holds its 128 rows of the result.

// Tensor memory: `columns` (a power of two, 32..512) of 128 lanes x 32 bits.
// All three are executed by one whole warp, the same one.
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t *smem_addr, uint32_t columns) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_addr)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_addr)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}

template <bool PAIR>
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t columns) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
  } else {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
  }
}

__device__ __forceinline__ void tcgen05_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tcgen05_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Arrives on `bar` (PAIR: on that of both CTAs) once the thread's earlier
// matrix products are complete.
template <bool PAIR>
__device__ __forceinline__ void tcgen05_commit(uint64_t *bar) {
  if constexpr (PAIR) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  } else {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
  }
}

// D[M x N] (+)= A[M x 16] B[N x 16]^T, operands by descriptor; M = 128, or 256
// of which each CTA of a pair holds 128, and half of B.
template <bool PAIR>
__device__ __forceinline__ void tcgen05_mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
  }
}

// Shared-memory operand: rows of 64 16-bit elements (128 bytes), K contiguous,
// in the 128-byte swizzle that a tiled TMA load writes; 1024-byte aligned.
// Eight rows are 1024 bytes apart from the next eight.  16 elements further
// along K is 32 bytes, i.e. +2 in the address field.
__device__ __forceinline__ uint64_t smem_desc_k128(uint32_t addr) {
  return (static_cast<uint64_t>(addr & 0x3ffffu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// ... whose contraction index K runs along the rows instead: rows of 64 elements of M or N, one for each k, 1024 bytes
// to the next eight; the next 64 elements of M or N are 8192 bytes away.  16 further along K is 2048 bytes: +128.
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t addr) {
  return (static_cast<uint64_t>(addr & 0x3ffffu) >> 4) | (512ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// Bits of the instruction descriptor: A and B have K along the rows.
constexpr uint32_t kIdescMnA = 1u << 15, kIdescMnB = 1u << 16;

// Instruction descriptor of kind::f16 with f32 sums: bf16 operands or f16,
// both K-major, m = 128 or (pair) 256 rows of A, n rows of B (a multiple of 16,
// of 32 for a pair; at most 256).
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, uint32_t m, uint32_t n) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// 16 consecutive columns of the warp's 32 lanes (the quarter of the 128 lanes
// that warp number % 4 names): register i is column i.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}

// ... and of 8.
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}

// The registers of earlier tmem_ld16 and tmem_ld8 calls hold their values.
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// The address that `local` has in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}

// Arrives on the mbarrier at cluster address `bar`.  Relaxed: it tells that this
// warp's tensor memory loads are complete (tmem_wait_ld), not of anything it wrote;
// a release at cluster scope would first wait for its stores to global memory
// (24000 x 1024 x 4096 with gelu 122 -> 118 us).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A tile into this CTA's shared memory; its bytes count on the mbarrier at
// cluster address `bar` (PAIR: CTA 0's).
template <bool PAIR>
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  if constexpr (PAIR) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
        "%3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  }
}

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

}  // namespace lm
