// beam.cu -- one step of beam search: log-softmax, selection over beams and
// vocabulary, and the token history that follows it, in one launch.
//
// A warp holds a tile of a beam's logits in registers (32 lanes x 8 vectors of
// 16 bytes, all in flight together: the pass is bound by reading the logits
// once) and takes three things from it: the maximum, the sum of exponentials,
// and its best `beams` continuations, a sorted list with one entry per lane.
// The n-th largest of the lanes' maxima bounds the list from below, so that
// only a few values ever reach the insertion.  A CTA joins its eight tiles; the
// last CTA of a clip joins the parts of its beams, in order, and selects.
//
// A continuation inside a beam is ordered by its key: the logit as an ordered
// integer, then the lower token.  Keys are distinct, so that an entry's place
// is the number of larger ones, whatever order it is found in.
#include <climits>

#include "half.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lm {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxBeams = 32;
constexpr int64_t kMaxVocab = 1 << 24;
constexpr int kVecs = 8;              // 16-byte vectors of a lane
constexpr int kTileVecs = 32 * kVecs;
constexpr int kClips = 16384;         // clips of a launch: counters at the workspace's start
constexpr size_t kCounterBytes = 4 * kClips;

struct BeamParams {
  lm_beam_args a;
  uint32_t *done;       // per clip: parts that are ready
  float2 *part_ms;      // [row][part]: maximum, sum of exponentials against it
  uint64_t *part_keys;  // [row][part][beams], largest first, 0 = none
  int32_t parts;
};

// Logits are compared as f32, -0 as 0; among equals the lower token is larger.
__device__ __forceinline__ uint64_t order_key(float x, int token) {
  return static_cast<uint64_t>(float_to_ordered(x + 0.0f)) << 32 | (0xffffffffu - static_cast<uint32_t>(token));
}
__device__ __forceinline__ float key_logit(uint64_t k) { return ordered_to_float(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ int key_token(uint64_t k) {
  return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// Value e of a 16-byte vector of T.
template <typename T>
__device__ __forceinline__ float value_of(const uint32_t (&w)[4], int e) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(w[e]);
  } else {
    const float2 f = unpack2<T>(w[e / 2]);
    return e & 1 ? f.y : f.x;
  }
}

template <typename T>
__device__ __forceinline__ uint32_t bits_of(T x);
template <>
__device__ __forceinline__ uint32_t bits_of<float>(float x) {
  return __float_as_uint(x);
}
template <>
__device__ __forceinline__ uint32_t bits_of<__half>(__half x) {
  return __half_as_ushort(x);
}
template <>
__device__ __forceinline__ uint32_t bits_of<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat16_as_ushort(x);
}

// The 16 bytes that start Q words (and half a word, with HALF) into the eight
// words w, x.
template <int Q, bool HALF>
__device__ __forceinline__ void shift_words(uint32_t (&w)[4], const uint32_t (&x)[4]) {
  uint32_t c[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    c[j] = w[j];
    c[4 + j] = x[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = HALF ? __funnelshift_r(c[j + Q], c[j + Q + 1], 16) : c[j + Q];
}

// Loads the aligned 16-byte vector `v` of a row that starts `skew` values into
// its vector 0; values outside the row read as -infinity.
template <typename T>
__device__ __forceinline__ void load_vec(const T *x, int64_t v, int skew, int vocab, uint32_t (&w)[4]) {
  constexpr int N = 16 / static_cast<int>(sizeof(T));
  const int64_t t0 = v * N - skew;
  if (t0 >= 0 && t0 + N <= vocab) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(x + t0));
    w[0] = u.x;
    w[1] = u.y;
    w[2] = u.z;
    w[3] = u.w;
    return;
  }
  const uint32_t none = bits_of<T>(from_f32<T>(-INFINITY));
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = sizeof(T) == 4 ? none : none | none << 16;
  if (t0 >= vocab) return;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (t0 + e >= 0 && t0 + e < vocab) {
      const uint32_t b = bits_of<T>(x[t0 + e]);
      if constexpr (sizeof(T) == 4) {
        w[e] = b;
      } else {
        w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | b << 16 : (w[e / 2] & 0xffff0000u) | b;
      }
    }
  }
}

// The largest `n` of the distinct nonzero keys in[0 .. count), largest first,
// into out[0 .. n) (0 where there are fewer); by `threads` threads.
__device__ __forceinline__ void largest(const uint64_t *in, int count, int n, uint64_t *out, int tid, int threads) {
  for (int i = tid; i < count; i += threads) {
    const uint64_t k = in[i];
    if (k == 0) continue;
    int place = 0;
    for (int j = 0; j < count; ++j) place += in[j] > k;
    if (place < n) out[place] = k;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_kernel(const BeamParams p) {
  constexpr int N = 16 / static_cast<int>(sizeof(T));  // values of a vector
  __shared__ uint64_t keys[kWarps * kMaxBeams];
  __shared__ float2 ms[kWarps];
  __shared__ uint64_t best[kMaxBeams];
  __shared__ bool last;
  const lm_beam_args &a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int part = blockIdx.x % p.parts;
  const int64_t row = blockIdx.x / p.parts;
  const int n = a.beams, vocab = static_cast<int>(a.vocab);

  // This lane's tokens: vectors v0 + 32 i of the row.  A row that starts off
  // a 16-byte boundary is read in the aligned vectors that hold it and moved
  // into place between the lanes, so that results do not depend on where a row
  // lies.
  const T *const x = static_cast<const T *>(a.logits) + row * a.row_stride;
  const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
  const int64_t v0 = (static_cast<int64_t>(part) * kWarps + warp) * kTileVecs + lane;
  uint32_t w[kVecs][4];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) load_vec(x, v0 + 32 * i, skew, vocab, w[i]);
  if (skew != 0) {
    uint32_t over[4];
    load_vec(x, v0 + 32 * kVecs - lane, skew, vocab, over);  // one address: the vector past the tile
    const int words = skew * static_cast<int>(sizeof(T)) / 4;
    const bool odd = sizeof(T) == 2 && (skew & 1);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      uint32_t next[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t first = i + 1 < kVecs ? __shfl_sync(0xffffffffu, w[(i + 1) % kVecs][j], 0) : over[j];
        next[j] = __shfl_down_sync(0xffffffffu, w[i][j], 1);
        if (lane == 31) next[j] = first;
      }
      switch (words * 2 + odd) {
        case 0: break;
        case 1: shift_words<0, true>(w[i], next); break;
        case 2: shift_words<1, false>(w[i], next); break;
        case 3: shift_words<1, true>(w[i], next); break;
        case 4: shift_words<2, false>(w[i], next); break;
        case 5: shift_words<2, true>(w[i], next); break;
        case 6: shift_words<3, false>(w[i], next); break;
        default: shift_words<3, true>(w[i], next); break;
      }
    }
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) top = fmaxf(top, value_of<T>(w[i], e));
  const float m = warp_max(top);
  // A NaN or +infinity makes the sum NaN, which marks the beam.
  const float base = m == -INFINITY ? 0.0f : m;
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) z += ex2((value_of<T>(w[i], e) - base) * kLog2e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);

  // The n-th largest of the lanes' maxima.
  uint32_t mine = float_to_ordered(top), kth = 0;
  for (int i = 0; i < n; ++i) {
    kth = __reduce_max_sync(0xffffffffu, mine);
    const uint32_t who = __ballot_sync(0xffffffffu, mine == kth);
    if (lane == __ffs(who) - 1) mine = 0;
  }
  float bound = kth == 0 ? -INFINITY : ordered_to_float(kth);
  uint64_t list = 0, floor = 0;  // lane i: the i-th best so far; the n-th
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float vt = value_of<T>(w[i], 0);
#pragma unroll
    for (int e = 1; e < N; ++e) vt = fmaxf(vt, value_of<T>(w[i], e));
    if (!__any_sync(0xffffffffu, vt >= bound)) continue;
    const int64_t t0 = (v0 + 32 * i) * N;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float v = value_of<T>(w[i], e);
      const int64_t t = t0 + e;
      uint64_t key = v >= bound && t < vocab ? order_key(v, static_cast<int>(t)) : 0;
      for (;;) {
        const uint32_t who = __ballot_sync(0xffffffffu, key > floor);
        if (who == 0) break;
        const int from = __ffs(who) - 1;
        const uint64_t k = __shfl_sync(0xffffffffu, key, from);
        if (lane == from) key = 0;
        const int place = __popc(__ballot_sync(0xffffffffu, list > k));
        const uint64_t up = __shfl_up_sync(0xffffffffu, list, 1);
        list = lane < place ? list : lane == place ? k : up;
        floor = __shfl_sync(0xffffffffu, list, n - 1);
      }
    }
  }
  if (lane < n) keys[warp * n + lane] = list;
  if (lane == 0) ms[warp] = make_float2(m, z);
  __syncthreads();

  // The CTA's eight tiles as one part.
  if (threadIdx.x < n) best[threadIdx.x] = 0;
  __syncthreads();
  largest(keys, kWarps * n, n, best, threadIdx.x, kThreads);
  __syncthreads();
  if (threadIdx.x < n) p.part_keys[(row * p.parts + part) * n + threadIdx.x] = best[threadIdx.x];
  if (threadIdx.x == 0) {
    float mm = -INFINITY, zz = 0.0f;
    for (int i = 0; i < kWarps; ++i) mm = fmaxf(mm, ms[i].x);
    const float bb = mm == -INFINITY ? 0.0f : mm;
    for (int i = 0; i < kWarps; ++i)
      zz += ms[i].x == -INFINITY ? ms[i].y : ms[i].y * ex2((ms[i].x - bb) * kLog2e);
    p.part_ms[row * p.parts + part] = make_float2(mm, zz);
  }
  __syncthreads();
  const int clip = static_cast<int>(row / n);
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(&p.done[clip], 1u) == static_cast<uint32_t>(p.parts * n - 1);
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (threadIdx.x == 0) p.done[clip] = 0;

  // The clip's last CTA.  A warp joins a beam's parts ...
  __shared__ float tot[kMaxBeams * kMaxBeams];
  __shared__ int tok[kMaxBeams * kMaxBeams];
  __shared__ int parents[kMaxBeams], tokens[kMaxBeams];
  const int places = vocab < n ? vocab : n;
  const int64_t row0 = static_cast<int64_t>(clip) * n;
  for (int b = warp; b < n; b += kWarps) {
    const int64_t r = row0 + b;
    const float2 *const pm = p.part_ms + r * p.parts;
    float mm = -INFINITY;
    for (int i = lane; i < p.parts; i += 32) mm = fmaxf(mm, __ldcg(pm + i).x);
    mm = warp_max(mm);
    const float bb = mm == -INFINITY ? 0.0f : mm;
    float zz = 0.0f;
    for (int i = lane; i < p.parts; i += 32) {
      const float2 v = __ldcg(pm + i);
      zz += v.x == -INFINITY ? v.y : v.y * ex2((v.x - bb) * kLog2e);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) zz += __shfl_xor_sync(0xffffffffu, zz, o);
    const bool dead = mm == -INFINITY || zz != zz;
    const float logz = logf(zz), score = a.scores[r];
    const bool ended = a.finished && a.finished[r];
    // ... its lists, one part after the other: n-way insertion of sorted lists.
    const uint64_t *const pk = p.part_keys + r * p.parts * n;
    uint64_t l = 0;
    for (int i0 = 0; i0 < p.parts; i0 += 4) {
      uint64_t next[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        next[i] = lane < n && i0 + i < p.parts
                      ? __ldcg(reinterpret_cast<const unsigned long long *>(pk + (i0 + i) * n + lane))
                      : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t k = next[i];
        if (i0 + i >= p.parts) break;
        // Both sorted, one per lane: an entry's place is its own index plus
        // the number of larger entries of the other list.
        int pl = lane, pn = lane;
        for (int j = 0; j < n; ++j) {
          pl += __shfl_sync(0xffffffffu, k, j) > l;
          pn += __shfl_sync(0xffffffffu, l, j) > k;
        }
        uint64_t *const mine_s = keys + warp * n;
        const int have = __popc(__ballot_sync(0xffffffffu, l != 0)) + __popc(__ballot_sync(0xffffffffu, k != 0));
        __syncwarp();
        if (lane < n && l != 0 && pl < n) mine_s[pl] = l;
        if (lane < n && k != 0 && pn < n) mine_s[pn] = k;
        __syncwarp();
        l = lane < n && lane < have ? mine_s[lane] : 0;
      }
    }
    if (lane < n) {
      float t = -INFINITY;
      int token = lane;
      if (ended) {
        t = lane == 0 ? score : -INFINITY;
        token = static_cast<int>(a.eos);
      } else if (!dead) {
        t = score + ((key_logit(l) - mm) - logz);
        token = key_token(l);
      }
      if (!(t == t)) t = -INFINITY;
      tot[b * n + lane] = t;
      tok[b * n + lane] = token;
    }
  }
  __syncthreads();
  // ... and all threads find each offer's place among the clip's.
  for (int i = threadIdx.x; i < n * n; i += kThreads) {
    const int b = i / n, c = i % n;
    if (c >= places) continue;
    const float t = tot[i];
    int place = 0;
    for (int j = 0; j < n && place < n; ++j) {
      // Beam j's list is sorted: count what goes in front.
      for (int k = 0; k < places; ++k) {
        const float u = tot[j * n + k];
        if (!(u > t || (u == t && j * n + k < i))) break;
        ++place;
      }
    }
    if (place < n) {
      const int64_t at = row0 + place;
      const bool was = a.finished && a.finished[row0 + b];
      a.out_scores[at] = t;
      a.out_tokens[at] = tok[i];
      a.out_parents[at] = b;
      a.out_finished[at] = was || tok[i] == a.eos;
      parents[place] = b;
      tokens[place] = tok[i];
    }
  }
  if (!a.history) return;
  __syncthreads();
  const uint32_t width = static_cast<uint32_t>(a.width), all = n * width;
  const int32_t *const from = a.history + row0 * a.width;
  int32_t *const to = a.out_history + row0 * a.width;
  for (uint32_t i0 = threadIdx.x; i0 < all; i0 += 8 * kThreads) {
    int32_t t[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t i = i0 + u * kThreads;
      if (i >= all) continue;
      const uint32_t b = i / width, c = i - b * width;
      t[u] = c == a.length ? tokens[b] : __ldg(from + parents[b] * static_cast<int64_t>(width) + c);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t i = i0 + u * kThreads;
      if (i < all) to[i] = t[u];
    }
  }
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

lm_status check(const lm_beam_args *a) {
  if (!a || a->clips < 0 || a->vocab < 1 || a->beams < 1 || a->row_stride < 0) return LM_ERR_INVALID_ARG;
  if (a->eos < -1 || a->eos >= a->vocab) return LM_ERR_INVALID_ARG;
  if (a->finished && a->eos < 0) return LM_ERR_INVALID_ARG;
  if (a->dtype != LM_F32 && a->dtype != LM_F16 && a->dtype != LM_BF16) return LM_ERR_UNSUPPORTED;
  if (a->beams > kMaxBeams || a->vocab > kMaxVocab || a->clips > INT_MAX / kMaxBeams) return LM_ERR_UNSUPPORTED;
  if ((a->history == nullptr) != (a->out_history == nullptr)) return LM_ERR_INVALID_ARG;
  if (a->history && (a->length < 0 || a->length >= a->width)) return LM_ERR_INVALID_ARG;
  if (a->width > (1 << 24)) return LM_ERR_UNSUPPORTED;
  return LM_OK;
}

// Parts of a row: eight warp tiles each.
int64_t parts_of(const lm_beam_args &a) {
  const int64_t n = kWarps * kTileVecs * (a.dtype == LM_F32 ? 4 : 8);
  return (a.vocab + n - 1) / n;
}

template <typename T>
lm_status launch(const BeamParams &p, cudaStream_t s) {
  const int64_t ctas = p.a.clips * p.a.beams * p.parts;
  if (ctas > INT_MAX) return LM_ERR_UNSUPPORTED;
  beam_kernel<T><<<static_cast<unsigned>(ctas), kThreads, 0, s>>>(p);
  LM_CUDA_TRY(cudaGetLastError());
  return LM_OK;
}

}  // namespace
}  // namespace lm

extern "C" lm_status lm_beam_step_workspace_size(const lm_beam_args *args, size_t *bytes) {
  using namespace lm;
  if (!bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st = check(args); st != LM_OK) return st;
  const size_t clips = static_cast<size_t>(args->clips < kClips ? args->clips : kClips);
  *bytes = 256 + kCounterBytes + clips * args->beams * parts_of(*args) * (sizeof(float2) + 8 * args->beams);
  return LM_OK;
}

extern "C" lm_status lm_beam_step(const lm_beam_args *args, void *workspace, size_t workspace_bytes,
                                  lm_stream_t stream) {
  using namespace lm;
  size_t need = 0;
  if (lm_status st = lm_beam_step_workspace_size(args, &need); st != LM_OK) return st;
  if (args->clips == 0) return LM_OK;
  BeamParams p;
  p.a = *args;
  lm_beam_args &a = p.a;
  if (!a.logits || !a.scores || !a.out_scores || !a.out_tokens || !a.out_parents || !a.out_finished)
    return LM_ERR_INVALID_ARG;
  if (!aligned(a.logits, a.dtype == LM_F32 ? 4 : 2) || !aligned(a.scores, 4) || !aligned(a.history, 4) ||
      !aligned(a.out_scores, 4) || !aligned(a.out_tokens, 4) || !aligned(a.out_parents, 4) ||
      !aligned(a.out_history, 4) || !aligned(workspace, 16))
    return LM_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < need) return LM_ERR_WORKSPACE;
  p.parts = static_cast<int32_t>(parts_of(a));
  char *const w = static_cast<char *>(workspace);
  p.done = reinterpret_cast<uint32_t *>(w + 256);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t size = a.dtype == LM_F32 ? 4 : 2;
  for (int64_t first = 0; first < args->clips; first += kClips) {
    a.clips = args->clips - first < kClips ? args->clips - first : kClips;
    const int64_t rows = a.clips * a.beams, skip = first * a.beams;
    p.part_ms = reinterpret_cast<float2 *>(w + 256 + kCounterBytes);
    p.part_keys = reinterpret_cast<uint64_t *>(p.part_ms + rows * p.parts);
    a.logits = static_cast<const char *>(args->logits) + skip * a.row_stride * size;
    a.scores = args->scores + skip;
    a.finished = args->finished ? args->finished + skip : nullptr;
    a.history = args->history ? args->history + skip * a.width : nullptr;
    a.out_scores = args->out_scores + skip;
    a.out_tokens = args->out_tokens + skip;
    a.out_parents = args->out_parents + skip;
    a.out_finished = args->out_finished + skip;
    a.out_history = args->out_history ? args->out_history + skip * a.width : nullptr;
    lm_status st;
    switch (a.dtype) {
      case LM_F32: st = launch<float>(p, s); break;
      case LM_F16: st = launch<__half>(p, s); break;
      default: st = launch<__nv_bfloat16>(p, s); break;
    }
    if (st != LM_OK) return st;
  }
  return LM_OK;
}
