// beam.cu -- one step of beam search: log-softmax, selection over beams and
// vocabulary, and the token history that follows it.
//
// One CTA per beam finds its log normaliser and its best continuations, one
// warp per clip then merges the beams' lists.
#include <climits>

#include "half.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBeams = 32;

// A continuation's order: larger first.  Logits are compared as f32, -0 as 0;
// among equals the lower token is the larger.
__device__ __forceinline__ uint64_t order_key(float x, int token) {
  return static_cast<uint64_t>(float_to_ordered(x + 0.0f)) << 32 | (0xffffffffu - static_cast<uint32_t>(token));
}

__device__ __forceinline__ uint64_t block_max(uint64_t v, uint64_t *part) {
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
    v = w > v ? w : v;
  }
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  for (int i = 0; i < kThreads / 32; ++i) v = part[i] > v ? part[i] : v;
  return v;
}

// A beam's best continuations, at [row][beams].
struct Offer {
  float total;
  int32_t token;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) offer_kernel(const lm_beam_args a, Offer *offers) {
  __shared__ uint64_t part[kThreads / 32];
  __shared__ float sums[kThreads / 32];
  const int64_t row = blockIdx.x;
  const T *const x = static_cast<const T *>(a.logits) + row * a.row_stride;
  const int vocab = static_cast<int>(a.vocab);
  const bool done = a.finished && a.finished[row];
  const float score = a.scores[row];
  uint64_t best = 0;
  bool bad = false;
  for (int i = threadIdx.x; i < vocab; i += kThreads) {
    const float v = to_f32(x[i]);
    bad = bad || !(v < INFINITY);
    const uint64_t k = order_key(v, i);
    best = k > best ? k : best;
  }
  bad = __syncthreads_or(bad);
  const float m = ordered_to_float(static_cast<uint32_t>(block_max(best, part) >> 32));
  const bool dead = bad || m == -INFINITY;
  float z = 0.0f;
  for (int i = threadIdx.x; i < vocab && !dead; i += kThreads) z += expf(to_f32(x[i]) - m);
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = z;
  __syncthreads();
  z = 0.0f;
  for (int i = 0; i < kThreads / 32; ++i) z += sums[i];
  const float logz = logf(z);
  uint64_t limit = ~0ull;
  for (int n = 0; n < a.beams; ++n) {
    Offer o{-INFINITY, 0};
    if (n < vocab) {
      uint64_t next = 0;
      for (int i = threadIdx.x; i < vocab; i += kThreads) {
        const uint64_t k = order_key(dead ? -INFINITY : to_f32(x[i]), i);
        if (k < limit && k > next) next = k;
      }
      limit = block_max(next, part);
      o.token = static_cast<int>(0xffffffffu - static_cast<uint32_t>(limit));
      const float t = score + ((ordered_to_float(static_cast<uint32_t>(limit >> 32)) - m) - logz);
      if (!dead && t == t) o.total = t;
    }
    if (done) o = Offer{n == 0 ? score : -INFINITY, static_cast<int32_t>(a.eos)};
    if (threadIdx.x == 0) offers[row * a.beams + n] = o;
  }
}

__global__ void __launch_bounds__(kThreads) select_kernel(const lm_beam_args a, const Offer *offers) {
  __shared__ float tot[kMaxBeams * kMaxBeams];
  __shared__ int parents[kMaxBeams], tokens[kMaxBeams];
  const int64_t clip = blockIdx.x;
  const int beams = a.beams, places = static_cast<int>(a.vocab < beams ? a.vocab : beams);
  const Offer *const o = offers + clip * beams * beams;
  for (int i = threadIdx.x; i < beams * beams; i += kThreads) tot[i] = o[i].total;
  __syncthreads();
  // An offer's place is the number of offers in front of it.
  for (int i = threadIdx.x; i < beams * beams; i += kThreads) {
    if (i % beams >= places) continue;
    const float t = tot[i] == tot[i] ? tot[i] : -INFINITY;
    int place = 0;
    for (int j = 0; j < beams * beams; ++j) {
      const float u = tot[j] == tot[j] ? tot[j] : -INFINITY;
      place += j % beams < places && (u > t || (u == t && j < i));
    }
    if (place < beams) {
      const int64_t at = clip * beams + place;
      const int parent = i / beams;
      const bool ended = (a.finished && a.finished[clip * beams + parent]) || o[i].token == a.eos;
      a.out_scores[at] = t;
      a.out_tokens[at] = o[i].token;
      a.out_parents[at] = parent;
      a.out_finished[at] = ended;
      parents[place] = parent;
      tokens[place] = o[i].token;
    }
  }
  __syncthreads();
  if (!a.history) return;
  for (int b = 0; b < beams; ++b) {
    const int32_t *const from = a.history + (clip * beams + parents[b]) * a.width;
    int32_t *const to = a.out_history + (clip * beams + b) * a.width;
    for (int64_t i = threadIdx.x; i < a.width; i += kThreads) to[i] = i == a.length ? tokens[b] : from[i];
  }
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

lm_status check(const lm_beam_args *a) {
  if (!a || a->clips < 0 || a->vocab < 1 || a->beams < 1 || a->row_stride < 0) return LM_ERR_INVALID_ARG;
  if (a->eos < -1 || a->eos >= a->vocab) return LM_ERR_INVALID_ARG;
  if (a->finished && a->eos < 0) return LM_ERR_INVALID_ARG;
  if (a->dtype != LM_F32 && a->dtype != LM_F16 && a->dtype != LM_BF16) return LM_ERR_UNSUPPORTED;
  if (a->beams > kMaxBeams || a->vocab > INT_MAX || a->clips > INT_MAX / kMaxBeams) return LM_ERR_UNSUPPORTED;
  if ((a->history == nullptr) != (a->out_history == nullptr)) return LM_ERR_INVALID_ARG;
  if (a->history && (a->length < 0 || a->length >= a->width)) return LM_ERR_INVALID_ARG;
  return LM_OK;
}

}  // namespace
}  // namespace lm

extern "C" lm_status lm_beam_step_workspace_size(const lm_beam_args *args, size_t *bytes) {
  using namespace lm;
  if (!bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st = check(args); st != LM_OK) return st;
  *bytes = kWorkspaceHeaderBytes + sizeof(Offer) * args->clips * args->beams * args->beams;
  return LM_OK;
}

extern "C" lm_status lm_beam_step(const lm_beam_args *args, void *workspace, size_t workspace_bytes,
                                  lm_stream_t stream) {
  using namespace lm;
  size_t need = 0;
  if (lm_status st = lm_beam_step_workspace_size(args, &need); st != LM_OK) return st;
  const lm_beam_args &a = *args;
  if (a.clips == 0) return LM_OK;
  if (!a.logits || !a.scores || !a.out_scores || !a.out_tokens || !a.out_parents || !a.out_finished)
    return LM_ERR_INVALID_ARG;
  if (!aligned(a.logits, a.dtype == LM_F32 ? 4 : 2) || !aligned(a.scores, 4) || !aligned(a.history, 4) ||
      !aligned(a.out_scores, 4) || !aligned(a.out_tokens, 4) || !aligned(a.out_parents, 4) ||
      !aligned(a.out_history, 4) || !aligned(workspace, 16))
    return LM_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < need) return LM_ERR_WORKSPACE;
  Offer *const offers = reinterpret_cast<Offer *>(static_cast<char *>(workspace) + kWorkspaceHeaderBytes);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned rows = static_cast<unsigned>(a.clips * a.beams);
  switch (a.dtype) {
    case LM_F32: offer_kernel<float><<<rows, kThreads, 0, s>>>(a, offers); break;
    case LM_F16: offer_kernel<__half><<<rows, kThreads, 0, s>>>(a, offers); break;
    default: offer_kernel<__nv_bfloat16><<<rows, kThreads, 0, s>>>(a, offers); break;
  }
  LM_CUDA_TRY(cudaGetLastError());
  select_kernel<<<static_cast<unsigned>(a.clips), kThreads, 0, s>>>(a, offers);
  LM_CUDA_TRY(cudaGetLastError());
  return LM_OK;
}
