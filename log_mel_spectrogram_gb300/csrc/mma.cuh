// mma.cuh -- warp-level matrix products (m16n8k16, f16 operands, f32 sums) and
// the exact conversion of signed bytes to f16.
//
// Fragments, with r = lane / 4 and c = lane % 4:
//   A (16 x 16, rows x k): a[0] = (r; 2c, 2c+1), a[1] = (r+8; 2c, 2c+1),
//                          a[2] = (r; 2c+8, 2c+9), a[3] = (r+8; 2c+8, 2c+9)
//   B (16 x 8, k x cols):  b[0] = (2c, 2c+1; r), b[1] = (2c+8, 2c+9; r)
//   C (16 x 8):            c[0], c[1] = (r; 2c, 2c+1), c[2], c[3] = (r+8; ...)
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace lm {

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ... of either type.
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  mma16816(d, a, b0, b1);
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8 x 8 matrices of 16-bit elements from shared memory: lane l gives the
// address of row l % 8 of matrix l / 8; r[m] holds, of matrix m, row lane / 4,
// columns 2 (lane % 4) and the next (TRANS: column lane / 4, those rows).
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if constexpr (TRANS) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  } else {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  }
}

// The bytes in the lower byte of each half of `u` as two f16: with the sign bit
// flipped a byte is b + 128, and 0x6400 | that is 1024 + 128 + b; subtracting
// 1152 is exact.
__device__ __forceinline__ uint32_t bytes_to_f16(uint32_t u) {
  const uint32_t x = (u & 0x00ff00ffu) ^ 0x64806480u;
  const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&x), __floats2half2_rn(1152.0f, 1152.0f));
  return *reinterpret_cast<const uint32_t *>(&d);
}

// The four bytes of `w` as two pairs of f16, by the same arithmetic.  (Through two words of
// every other byte, by shift and mask, the long rows of kv_attend.cu take 100.8 us, so 96.9.)
__device__ __forceinline__ void word_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const uint32_t x = w ^ 0x80808080u;
  const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
  const __half2 offset = __floats2half2_rn(1152.0f, 1152.0f);
  const __half2 l = __hsub2(*reinterpret_cast<const __half2 *>(&a), offset);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&b), offset);
  lo = *reinterpret_cast<const uint32_t *>(&l);
  hi = *reinterpret_cast<const uint32_t *>(&h);
}

}  // namespace lm
