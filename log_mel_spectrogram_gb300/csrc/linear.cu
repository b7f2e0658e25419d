// linear.cu -- y = residual + scale * act(x W^T + bias).
//
// One thread per output element, operands through 16 x 16 tiles of shared
// memory, sums in 32 bits.
#include <climits>

#include "half.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lm {
namespace {

constexpr int kTile = 16;

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case LM_ACT_RELU: return fmaxf(z, 0.0f);
    case LM_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case LM_ACT_GELU_TANH: return 0.5f * z * (1.0f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
    case LM_ACT_SILU: return z / (1.0f + expf(-z));
    default: return z;
  }
}

template <typename T>
__global__ void linear_kernel(const lm_linear_args a) {
  __shared__ float xs[kTile][kTile + 1], ws[kTile][kTile + 1];
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kTile + threadIdx.x;
  const int64_t m = static_cast<int64_t>(blockIdx.y) * kTile + threadIdx.y;
  const int64_t rows = a.groups * a.rows;
  const int64_t nl = static_cast<int64_t>(blockIdx.x) * kTile + threadIdx.y;
  const T *const x = static_cast<const T *>(a.x) + m / a.rows * a.x_group_stride + m % a.rows * a.x_row_stride;
  const T *const w = static_cast<const T *>(a.weight) + nl * a.weight_row_stride;
  float s = 0.0f;
  for (int64_t k0 = 0; k0 < a.k; k0 += kTile) {
    const int64_t k = k0 + threadIdx.x;
    xs[threadIdx.y][threadIdx.x] = m < rows && k < a.k ? to_f32(x[k]) : 0.0f;
    ws[threadIdx.y][threadIdx.x] = nl < a.n && k < a.k ? to_f32(w[k]) : 0.0f;
    __syncthreads();
    for (int j = 0; j < kTile; ++j) s += xs[threadIdx.y][j] * ws[threadIdx.x][j];
    __syncthreads();
  }
  if (m >= rows || n >= a.n) return;
  if (a.bias)
    s += a.bias_dtype == LM_F32 ? static_cast<const float *>(a.bias)[n] : to_f32(static_cast<const T *>(a.bias)[n]);
  s = a.scale * activate(s, a.activation);
  if (a.residual) s += to_f32(static_cast<const T *>(a.residual)[m * a.residual_row_stride + n]);
  if (a.out_dtype == LM_F32) {
    static_cast<float *>(a.out)[m * a.out_row_stride + n] = s;
  } else {
    static_cast<T *>(a.out)[m * a.out_row_stride + n] = from_f32<T>(s);
  }
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
  if (a->k > INT_MAX || a->n > INT_MAX || a->groups > INT_MAX || a->rows > INT_MAX ||
      a->groups * a->rows > INT_MAX)
    return LM_ERR_UNSUPPORTED;
  return LM_OK;
}

}  // namespace
}  // namespace lm

extern "C" lm_status lm_linear_workspace_size(const lm_linear_args *args, size_t *bytes) {
  if (!bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::check(args); st != LM_OK) return st;
  *bytes = lm::kWorkspaceHeaderBytes;
  return LM_OK;
}

extern "C" lm_status lm_linear(const lm_linear_args *args, void *workspace, size_t workspace_bytes,
                               lm_stream_t stream) {
  using namespace lm;
  size_t need = 0;
  if (lm_status st = lm_linear_workspace_size(args, &need); st != LM_OK) return st;
  const lm_linear_args &a = *args;
  if (a.groups * a.rows == 0 || a.n == 0) return LM_OK;
  if (!a.out || (a.k > 0 && (!a.x || !a.weight))) return LM_ERR_INVALID_ARG;
  const size_t out_size = a.out_dtype == LM_F32 ? 4 : 2;
  if (!aligned(a.x, 2) || !aligned(a.weight, 2) || !aligned(a.bias, a.bias_dtype == LM_F32 ? 4 : 2) ||
      !aligned(a.residual, 2) || !aligned(a.out, out_size) || !aligned(workspace, 16))
    return LM_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < need) return LM_ERR_WORKSPACE;
  const int64_t gx = (a.n + kTile - 1) / kTile, gy = (a.groups * a.rows + kTile - 1) / kTile;
  if (gy > 65535) return LM_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), block(kTile, kTile);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a.dtype == LM_F16) {
    linear_kernel<__half><<<grid, block, 0, s>>>(a);
  } else {
    linear_kernel<__nv_bfloat16><<<grid, block, 0, s>>>(a);
  }
  LM_CUDA_TRY(cudaGetLastError());
  return LM_OK;
}
