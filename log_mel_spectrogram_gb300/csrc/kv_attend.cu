// kv_attend.cu -- attention over the 8-bit key/value cache.
//
// One warp per query row and head walks the row's tokens with a running
// maximum and sum; lanes hold head_dim / 32 elements each.
#include <climits>

#include "half.cuh"
#include "internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace lm {
namespace {

constexpr int kThreads = 128;

struct AttendParams {
  KvView c;
  const void *q;
  void *out;
  int64_t row_s, tok_s, head_s;
  const int32_t *counts;
  int32_t tokens, q_heads, new_tokens, causal;
  float scale;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attend_kernel(const AttendParams p) {
  const int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (u >= static_cast<int64_t>(p.c.rows) * p.tokens * p.q_heads) return;
  const int hq = static_cast<int>(u % p.q_heads), i = static_cast<int>(u / p.q_heads % p.tokens);
  const int r = static_cast<int>(u / p.q_heads / p.tokens);
  const int h = hq / (p.q_heads / p.c.heads);
  const int64_t cap = static_cast<int64_t>(p.c.width) * p.c.block;
  const int64_t held = max(p.c.lens[r], 0);
  const int fresh = min(max(p.counts ? p.counts[r] : p.new_tokens, 0), p.causal ? p.tokens : INT_MAX);
  int64_t end = min(held + fresh, cap);
  if (p.causal) end = i < fresh ? min(end, held + i + 1) : 0;
  constexpr int N = D / 32;
  float q[N], acc[N] = {}, m = -INFINITY, l = 0.0f;
  const T *const qp = static_cast<const T *>(p.q) + r * p.row_s + i * p.tok_s + hq * p.head_s;
  for (int j = 0; j < N; ++j) q[j] = to_f32(qp[lane * N + j]) * p.scale;
  for (int64_t t = 0; t < end; ++t) {
    const int blk = p.c.table[r * static_cast<int64_t>(p.c.width) + t / p.c.block];
    if (blk < 0 || blk >= p.c.blocks) continue;
    const int64_t tile = p.c.layer_tiles + static_cast<int64_t>(blk) * p.c.heads + h;
    const int64_t at = (tile * p.c.block + t % p.c.block) * D + lane * N;
    float s = 0.0f;
    for (int j = 0; j < N; ++j) s += q[j] * p.c.k8[at + j];
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= p.c.k_scale[tile];
    const float mn = fmaxf(m, s), a = m == mn ? 1.0f : expf(m - mn), w = expf(s - mn);
    m = mn;
    l = l * a + w;
    for (int j = 0; j < N; ++j) acc[j] = acc[j] * a + w * (p.c.v8[at + j] * p.c.v_scale[tile]);
  }
  T *const o = static_cast<T *>(p.out) + u * D + lane * N;
  for (int j = 0; j < N; ++j) o[j] = from_f32<T>(l == 0.0f ? 0.0f : acc[j] / l);
}

template <typename T>
lm_status launch(const AttendParams &p, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.c.rows) * p.tokens * p.q_heads;
  const int64_t ctas = (rows + kThreads / 32 - 1) / (kThreads / 32);
  if (ctas > INT_MAX) return LM_ERR_UNSUPPORTED;
  const unsigned n = static_cast<unsigned>(ctas);
  switch (p.c.head_dim) {
    case 32: attend_kernel<T, 32><<<n, kThreads, 0, s>>>(p); break;
    case 64: attend_kernel<T, 64><<<n, kThreads, 0, s>>>(p); break;
    default: attend_kernel<T, 128><<<n, kThreads, 0, s>>>(p); break;
  }
  LM_CUDA_TRY(cudaGetLastError());
  return LM_OK;
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

lm_status check(const lm_kv_cache *cache, int32_t tokens, int32_t q_heads) {
  if (lm_status st = kv_check(cache); st != LM_OK) return st;
  if (tokens < 0 || q_heads < 1 || q_heads % cache->heads != 0) return LM_ERR_INVALID_ARG;
  return LM_OK;
}

}  // namespace
}  // namespace lm

extern "C" lm_status lm_kv_attend_workspace_size(const lm_kv_cache *cache, int32_t tokens, int32_t q_heads,
                                                 size_t *bytes) {
  if (!bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::check(cache, tokens, q_heads); st != LM_OK) return st;
  *bytes = lm::kWorkspaceHeaderBytes;
  return LM_OK;
}

extern "C" lm_status lm_kv_attend(const lm_kv_cache *cache, int32_t layer, const void *q, const int64_t *q_strides,
                                  int32_t tokens, int32_t q_heads, const int32_t *counts, int32_t new_tokens,
                                  int32_t causal, float scale, int32_t dtype, void *out, void *workspace,
                                  size_t workspace_bytes, lm_stream_t stream) {
  using namespace lm;
  if (lm_status st = check(cache, tokens, q_heads); st != LM_OK) return st;
  if (layer < 0 || layer >= cache->layers || !q_strides || new_tokens < 0) return LM_ERR_INVALID_ARG;
  if (dtype != LM_F16 && dtype != LM_BF16) return LM_ERR_UNSUPPORTED;
  if (cache->rows == 0 || tokens == 0) return LM_OK;
  if (!q || !out) return LM_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (q_strides[i] < 0) return LM_ERR_INVALID_ARG;
  if (!aligned(q, 2) || !aligned(out, 16) || !aligned(workspace, 16)) return LM_ERR_MISALIGNED;
  size_t need = 0;
  lm_kv_attend_workspace_size(cache, tokens, q_heads, &need);
  if (!workspace || workspace_bytes < need) return LM_ERR_WORKSPACE;
  AttendParams p;
  p.c = kv_view(cache, layer);
  p.q = q;
  p.out = out;
  p.row_s = q_strides[0];
  p.tok_s = q_strides[1];
  p.head_s = q_strides[2];
  p.counts = counts;
  p.tokens = tokens;
  p.q_heads = q_heads;
  p.new_tokens = new_tokens;
  p.causal = causal != 0;
  p.scale = scale;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == LM_F16 ? launch<__half>(p, s) : launch<__nv_bfloat16>(p, s);
}
