// operand.cuh -- matrices of 16-bit elements as the tensor cores' kernels fetch them: tensor maps, and copies of
// those whose rows are off 16-byte boundaries.
#pragma once

#include <climits>
#include <cuda.h>

#include "internal.h"
#include "pdl.cuh"

namespace lm {
namespace {

// Copies rows off 16-byte boundaries into rows padded to 8 elements.
struct PackParams {
  const uint16_t *src;
  uint4 *dst;
  int64_t group_stride, row_stride, rows, k, vecs, total;  // vecs: 16-byte vectors a row
};

// Vector i of the copy.
__device__ __forceinline__ void pack_vector(const PackParams &p, int64_t i) {
  const int64_t row = i / p.vecs, v = i % p.vecs;
  const uint16_t *const s = p.src + row / p.rows * p.group_stride + row % p.rows * p.row_stride + v * 8;
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = v * 8 + j < p.k ? s[j] : 0u;
  p.dst[i] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
}

__global__ void __launch_bounds__(256) pack_kernel(const PackParams p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  pdl_launch();
  pdl_wait();
  if (i < p.total) pack_vector(p, i);
}

// Three of them in one launch; one that is not wanted has no vectors.
struct PackThree {
  PackParams p[3];
};

__global__ void __launch_bounds__(256) pack_three_kernel(const PackThree a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  pdl_launch();
  pdl_wait();
  const int64_t second = i - a.p[0].total, third = second - a.p[1].total;
  if (second < 0) {
    pack_vector(a.p[0], i);
  } else if (third < 0) {
    pack_vector(a.p[1], second);
  } else if (third < a.p[2].total) {
    pack_vector(a.p[2], third);
  }
}

inline bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// An operand as TMA sees it: [groups][rows][k], strides in elements.
struct Operand {
  const void *p;
  int64_t groups, rows, group_stride, row_stride;
  bool pack;       // copied into the workspace first
  size_t bytes;    // of that copy
};

inline Operand operand(const void *p, int64_t groups, int64_t rows, int64_t k, int64_t group_stride, int64_t row_stride) {
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

// The copy of an operand, which it stands for from then on.
inline PackParams pack_params(Operand *o, int64_t k, void *dst) {
  PackParams p;
  p.src = static_cast<const uint16_t *>(o->p);
  p.dst = static_cast<uint4 *>(dst);
  p.group_stride = o->group_stride;
  p.row_stride = o->row_stride;
  p.rows = o->rows;
  p.k = k;
  p.vecs = (k + 7) / 8;
  p.total = o->groups * o->rows * p.vecs;
  o->p = dst;
  o->row_stride = p.vecs * 8;
  o->group_stride = o->rows * o->row_stride;
  return p;
}

inline lm_status pack(Operand *o, int64_t k, void *dst, cudaStream_t s) {
  const PackParams p = pack_params(o, k, dst);
  const int64_t ctas = (p.total + 255) / 256;
  if (ctas > INT_MAX) return LM_ERR_UNSUPPORTED;
  return launch_dependent(pack_kernel, dim3(static_cast<unsigned>(ctas)), 256, 0, s, 1, p);
}

// Those of three operands that have to be copied, into dst one after the other, on boundaries of 256 bytes.
inline lm_status pack_three(Operand *const (&o)[3], int64_t k, char *dst, cudaStream_t s) {
  PackThree a = {};
  int64_t total = 0;
  for (int i = 0; i < 3; ++i) {
    const size_t bytes = o[i]->bytes;
    if (o[i]->pack) a.p[i] = pack_params(o[i], k, dst);
    total += a.p[i].total;
    dst += (bytes + 255) / 256 * 256;
  }
  const int64_t ctas = (total + 255) / 256;
  if (ctas > INT_MAX) return LM_ERR_UNSUPPORTED;
  if (ctas == 0) return LM_OK;
  return launch_dependent(pack_three_kernel, dim3(static_cast<unsigned>(ctas)), 256, 0, s, 1, a);
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
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

// Tiles of `box_rows` rows x 64 of the `k` contiguous elements, zeros outside.
inline lm_status make_map(CUtensorMap *map, const Operand &o, int64_t k, int box_rows, bool bf16) {
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
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1}, one[3] = {1, 1, 1};
  auto encode = [&] {
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(o.p),
              dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {  // the thread's first call to CUDA, which is the driver's: it has no context yet
    int dev = 0;
    LM_CUDA_TRY(cudaGetDevice(&dev));
    LM_CUDA_TRY(cudaSetDevice(dev));
    r = encode();
  }
  return r == CUDA_SUCCESS ? LM_OK : cuda_fail(cudaErrorInvalidValue);
}

}  // namespace
}  // namespace lm
