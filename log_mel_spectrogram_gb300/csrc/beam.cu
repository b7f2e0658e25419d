// beam.cu -- one step of beam search: log-softmax, selection over beams and
// vocabulary, and the token history that follows it, in one launch.
//
// A warp holds a tile of a beam's logits in registers (32 lanes x 8 vectors of
// 16 bytes, all in flight together: the pass is bound by reading the logits
// once) and takes three things from it: the maximum, the sum of exponentials,
// and its best `beams` continuations.  The n-th largest of the lanes' maxima
// bounds those from below, so that hardly more than n values are ever gathered
// and ranked.  A CTA joins its eight tiles; the last CTA of a clip joins the
// parts of its beams, in order, and selects.  A few rows alone take tiles of 2
// vectors, for the sake of latency.
//
// A continuation inside a beam is ordered by its key: the logit as an ordered
// integer, then the lower token.  Keys are distinct, so that an entry's place
// is the number of larger ones, whatever order it is found in.
//
// Measured: 64 clips of 5 beams over 50001 f32 logits 25.5 us where the linear
// layer left them in L2, 32 from memory (fetching a warp's next tiles ahead into L2
// only cost time): seven tiles a warp, each with one load's latency and a chain
// of warp reductions, then 8 us for the joins.  One clip, bf16, 9.3 us without a history.
#include <climits>

#include "f32x2.cuh"
#include "half.cuh"
#include "internal.h"
#include "pdl.cuh"
#include "ptx.cuh"

namespace lm {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxBeams = 32;
constexpr int64_t kMaxVocab = 1 << 24;
constexpr int kHistory = 4096;         // entries of a clip's histories that are fetched ahead
constexpr int kGather = 64;           // keys that a warp gathers before it ranks them
constexpr int kClips = 16384;         // clips of a launch: counters at the workspace's start
constexpr size_t kCounterBytes = 4 * kClips;

struct BeamParams {
  lm_beam_args a;
  uint32_t *done;       // per clip: parts that are ready
  float2 *part_ms;      // [row][part]: maximum, sum of exponentials against it
  uint64_t *part_keys;  // [row][part][beams], largest first, 0 = none
  int32_t parts, tiles;  // CTAs of a row; tiles that each of their warps goes over
};

// Logits are compared as f32, -0 as 0; among equals the lower token is larger.
__device__ __forceinline__ uint64_t order_key(float x, int token) {
  return static_cast<uint64_t>(float_to_ordered(x + 0.0f)) << 32 | (0xffffffffu - static_cast<uint32_t>(token));
}
__device__ __forceinline__ float key_logit(uint64_t k) { return ordered_to_float(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ int key_token(uint64_t k) {
  return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k));
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

// Moves what a warp's lanes hold (vector i of lane l: the 16 bytes at 512 i + 16 l)
// down by S words and, if ODD, a half: `over` comes after the last vector.
template <int S, bool ODD, int kVecs>
__device__ __forceinline__ void move_down(uint32_t (&w)[kVecs][4], const uint32_t (&over)[4], int lane) {
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    uint32_t c[5];
#pragma unroll
    for (int j = 0; j < 4 + ODD; ++j) {
      if (j + S < 4) {
        c[j] = w[i][j + S];
      } else {
        // Lane 31 is followed by lane 0's next vector, which lane 0 hands round.
        const uint32_t after = i + 1 < kVecs ? w[(i + 1) % kVecs][j + S - 4] : over[j + S - 4];
        c[j] = __shfl_sync(0xffffffffu, lane == 0 ? after : w[i][j + S - 4], (lane + 1) % 32);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) w[i][j] = ODD ? __funnelshift_r(c[j], c[j + 1], 16) : c[j];
  }
}

// The aligned 16-byte vector that starts at value t0 of a row; values outside
// the row read as -infinity.
template <typename T>
__device__ __noinline__ uint4 load_edge(const T *x, int t0, int vocab) {
  constexpr int N = 16 / static_cast<int>(sizeof(T));
  const uint32_t none = bits_of<T>(from_f32<T>(-INFINITY));
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const bool in = t0 + e >= 0 && t0 + e < vocab;
    const uint32_t b = in ? bits_of<T>(x[t0 + e]) : none;
    if constexpr (sizeof(T) == 4) {
      w[e] = b;
    } else {
      w[e / 2] = e & 1 ? w[e / 2] | b << 16 : b;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Ranks the `count` <= kGather keys that a warp has gathered (distinct, or 0 for
// none): the largest `n` in order, then zeros up to n.  Returns how many there are;
// *floor: the n-th.
__device__ __noinline__ int rank_keys(uint64_t *keys, int count, int n, uint64_t *floor) {
  const int lane = threadIdx.x % 32;
  __syncwarp();
  const uint64_t a = lane < count ? keys[lane] : 0, b = lane + 32 < count ? keys[lane + 32] : 0;
  int pa = 0, pb = 0;
#pragma unroll 4
  for (int j = 0; j < count; ++j) {
    const uint64_t k = keys[j];
    pa += k > a;
    pb += k > b;
  }
  const int found = __popc(__ballot_sync(0xffffffffu, a != 0)) + __popc(__ballot_sync(0xffffffffu, b != 0));
  const int left = found < n ? found : n;
  __syncwarp();
  if (a != 0 && pa < n) keys[pa] = a;
  if (b != 0 && pb < n) keys[pb] = b;
  if (lane >= left && lane < n) keys[lane] = 0;
  __syncwarp();
  *floor = keys[n - 1];
  return left;
}

// A warp's shared memory: vectors that hold a value of interest, and keys.
struct Gather {
  uint64_t keys[kGather];
  uint4 vecs[kGather];
  int first[kGather];  // the first token of a vector
};

// Adds the values of `count` gathered vectors that reach `bound` to the keys.
// Returns how many keys there are then; *floor as of rank_keys.
template <typename T>
__device__ __noinline__ int take_keys(Gather *g, int count, int keys, float bound, int vocab, int n, uint64_t *floor) {
  constexpr int N = 16 / static_cast<int>(sizeof(T));
  const int lane = threadIdx.x % 32;
  uint64_t least = *floor;
  __syncwarp();
#pragma unroll 1
  for (int i = lane; i - lane < count * N; i += 32) {
    uint64_t key = 0;
    if (i < count * N) {
      const float v = to_f32(reinterpret_cast<const T *>(g->vecs)[i]);
      const int t = g->first[i / N] + i % N;
      if (v >= bound && t < vocab) key = order_key(v, t);
    }
    const uint32_t who = __ballot_sync(0xffffffffu, key > least);
    if (who == 0) continue;
    if (key > least) g->keys[keys + __popc(who & ((1u << lane) - 1))] = key;
    keys += __popc(who);
    if (keys > kGather - 32) keys = rank_keys(g->keys, keys, n, &least);
  }
  __syncwarp();
  *floor = least;
  return keys;
}

template <typename T, int kVecs>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 2) beam_kernel(const BeamParams p) {
  constexpr int N = 16 / static_cast<int>(sizeof(T));  // values of a vector
  constexpr int kTileVecs = 32 * kVecs;
  __shared__ Gather gathered[kWarps];
  __shared__ float2 ms[kWarps];
  __shared__ float tot[kMaxBeams * kMaxBeams];
  __shared__ int tok[kMaxBeams * kMaxBeams];
  __shared__ int parents[kMaxBeams], tokens[kMaxBeams];
  __shared__ bool over[kMaxBeams];
  __shared__ int32_t history[kHistory];
  __shared__ bool last;
  pdl_launch();
  pdl_wait();
  const lm_beam_args &a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int part = blockIdx.x % p.parts;
  const int64_t row = blockIdx.x / p.parts;
  const int n = a.beams, vocab = static_cast<int>(a.vocab);

  // A row that starts off a 16-byte boundary is read in the aligned vectors
  // that hold it and moved into place between the lanes, so that results do not
  // depend on where a row lies.
  const T *const x = static_cast<const T *>(a.logits) + row * a.row_stride;
  const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
  Gather &g = gathered[warp];
  uint64_t *const list = g.keys;
  uint64_t floor = 0;  // what a key has to beat
  int count = 0;
  float m = -INFINITY, z = 0.0f;
  for (int k = 0; k < p.tiles; ++k) {
    const int tile0 = ((part * p.tiles + k) * kWarps + warp) * kTileVecs * N;
    if (tile0 >= vocab) break;
    const int t0 = tile0 + lane * N;  // vector i holds the tokens from t0 + 32 N i on
    uint32_t w[kVecs][4];
    auto load = [&](int at) {
      return at >= 0 && at + N <= vocab ? *reinterpret_cast<const uint4 *>(x + at) : load_edge(x, at, vocab);
    };
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint4 u = load(t0 - skew + 32 * N * i);
      w[i][0] = u.x;
      w[i][1] = u.y;
      w[i][2] = u.z;
      w[i][3] = u.w;
    }
    if (skew != 0) {
      const uint4 u = load(tile0 - skew + kTileVecs * N);  // one address: the vector past the tile
      const uint32_t over[4] = {u.x, u.y, u.z, u.w};
      if constexpr (sizeof(T) == 4) {
        switch (skew) {
          case 1: move_down<1, false>(w, over, lane); break;
          case 2: move_down<2, false>(w, over, lane); break;
          default: move_down<3, false>(w, over, lane); break;
        }
      } else {
        switch (skew) {
          case 1: move_down<0, true>(w, over, lane); break;
          case 2: move_down<1, false>(w, over, lane); break;
          case 3: move_down<1, true>(w, over, lane); break;
          case 4: move_down<2, false>(w, over, lane); break;
          case 5: move_down<2, true>(w, over, lane); break;
          case 6: move_down<3, false>(w, over, lane); break;
          default: move_down<3, true>(w, over, lane); break;
        }
      }
    }
    float vt[kVecs], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      vt[i] = value_of<T>(w[i], 0);
#pragma unroll
      for (int e = 1; e < N; ++e) vt[i] = fmaxf(vt[i], value_of<T>(w[i], e));
      top = fmaxf(top, vt[i]);
    }
    const float before = m;
    m = fmaxf(m, warp_max(top));
    // A NaN or +infinity makes the sum NaN, which marks the beam.
    const float base = m == -INFINITY ? 0.0f : m;
    if (before != -INFINITY) z *= ex2((before - base) * kLog2e);
    f32x2 z2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const f32x2 x2 = pair(value_of<T>(w[i], e), value_of<T>(w[i], e + 1));
        const float2 y = unpair(mul2(add2(x2, both(-base)), both(kLog2e)));
        z2 = add2(z2, pair(ex2(y.x), ex2(y.y)));
      }
    z += unpair(z2).x + unpair(z2).y;

    // A bound from below: the n-th best so far, or the n-th largest of the
    // lanes' maxima.
    float bound = key_logit(floor);
    if (floor == 0) {
      uint32_t mine = float_to_ordered(top), kth = 0;
      for (int i = 0; i < n; ++i) {
        kth = __reduce_max_sync(0xffffffffu, mine);
        const uint32_t who = __ballot_sync(0xffffffffu, mine == kth);
        if (lane == __ffs(who) - 1) mine = 0;
      }
      bound = kth == 0 ? -INFINITY : ordered_to_float(kth);
    }
    if (!__any_sync(0xffffffffu, top >= bound)) continue;
    int queued = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t who = __ballot_sync(0xffffffffu, vt[i] >= bound);
      if (who == 0) continue;
      if (vt[i] >= bound) {
        const int at = queued + __popc(who & ((1u << lane) - 1));
        g.vecs[at] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
        g.first[at] = t0 + 32 * N * i;
      }
      queued += __popc(who);
      if (queued > kGather - 32) {
        count = take_keys<T>(&g, queued, count, bound, vocab, n, &floor);
        queued = 0;
      }
    }
    count = take_keys<T>(&g, queued, count, bound, vocab, n, &floor);
    // A first bound, or room for more.
    if (k + 1 < p.tiles && (floor == 0 || count > kGather - 32)) count = rank_keys(list, count, n, &floor);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  rank_keys(list, count, n, &floor);
  if (lane == 0) ms[warp] = make_float2(m, z);
  __syncthreads();

  // The CTA's eight lists as one part.
  uint64_t *const part_keys = p.part_keys + (row * p.parts + part) * n;
  if (warp == kWarps - 1) {
    const float2 v = lane < kWarps ? ms[lane] : make_float2(-INFINITY, 0.0f);
    const float mm = warp_max(v.x), bb = mm == -INFINITY ? 0.0f : mm;
    float zz = v.x == -INFINITY ? v.y : v.y * ex2((v.x - bb) * kLog2e);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) zz += __shfl_xor_sync(0xffffffffu, zz, o);
    if (lane == 0) p.part_ms[row * p.parts + part] = make_float2(mm, zz);
  }
  // (Zeros fill up places that no key takes: they count what they follow.)
  for (int i = threadIdx.x; i < kWarps * n; i += kThreads) {
    const int of = i / n, at = i - of * n;
    const uint64_t k = gathered[of].keys[at];
    int place = 0;
#pragma unroll 1
    for (int u = 0; u < n; ++u) {
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        const uint64_t o = gathered[j].keys[u];
        place += o > k || (o == k && j * n + u < i);
      }
    }
    if (place < n) part_keys[place] = k;
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

  // The clip's last CTA.  Its beams' histories are on their way meanwhile,
  // where they fit ...
  const int places = vocab < n ? vocab : n;
  const int64_t row0 = static_cast<int64_t>(clip) * n;
  const uint32_t width = static_cast<uint32_t>(a.width);
  const uint32_t told = a.history ? n * width : 0;
  const int32_t *const from = a.history + row0 * a.width;
  int32_t *const to = a.out_history + row0 * a.width;
  const bool ahead = told <= kHistory;
  if (ahead) {
#pragma unroll 1
    for (uint32_t i = threadIdx.x; i < told; i += kThreads)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(history + i)), "l"(from + i) : "memory");
  }
  // ... and a warp joins a beam's parts.
  for (int b = warp; b < n; b += kWarps) {
    const int64_t r = row0 + b;
    const float2 *const pm = p.part_ms + r * p.parts;
    const uint64_t *const pk = p.part_keys + r * p.parts * n;
    const int all = p.parts * n;
    const float score = a.scores[r];
    const bool ended = a.finished && a.finished[r];
    auto key_at = [&](int i) -> uint64_t {
      return i < all ? __ldcg(reinterpret_cast<const unsigned long long *>(pk + i)) : 0;
    };
    const uint64_t k0 = key_at(lane), k1 = key_at(lane + 32);
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
    const float logz = logf(zz);
    list[lane] = k0;
    list[lane + 32] = k1;
    count = rank_keys(list, all < kGather ? all : kGather, n, &floor);
    for (int i = kGather; i < all; i += 32) {
      const uint64_t k = key_at(i + lane);
      const uint32_t who = __ballot_sync(0xffffffffu, k > floor);
      if (who == 0) continue;
      if (k > floor) list[n + __popc(who & ((1u << lane) - 1))] = k;
      count = rank_keys(list, n + __popc(who), n, &floor);
    }
    if (lane < n) {
      const uint64_t l = list[lane];
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
      tot[b * n + lane] = t + 0.0f;  // -0 as 0
      tok[b * n + lane] = token;
      if (lane == 0) over[b] = ended;
    }
    __syncwarp();
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  // Offer i takes its place.
  auto select = [&](int i, int place) {
    const int b = i / n;
    const int64_t at = row0 + place;
    a.out_scores[at] = tot[i];
    a.out_tokens[at] = tok[i];
    a.out_parents[at] = b;
    a.out_finished[at] = over[b] || tok[i] == a.eos;
    parents[place] = b;
    tokens[place] = tok[i];
  };
  if (n <= 8 && places == n) {
    // A thread per offer counts those in front of it.
    const int i = threadIdx.x;
    if (i < n * n) {
      const float t = tot[i];
      int place = 0;
      for (int j = 0; j < n * n; ++j) {
        const float u = tot[j];
        place += u > t || (u == t && j < i);
      }
      if (place < n) select(i, place);
    }
  } else if (warp == 0) {
    // A beam's offers are in order: a lane per beam, and the best head n times
    // (5 beams of 1000 logits 7.8 us so, 7.1 by counting; 16 beams 12.6 and 15.6).
    int next = 0, mine = 0;
    for (int i = 0; i < n; ++i) {
      const uint32_t head = lane < n && next < places ? float_to_ordered(tot[lane * n + next]) : 0;
      const uint32_t best = __reduce_max_sync(0xffffffffu, head);
      const int who = __ffs(__ballot_sync(0xffffffffu, head == best)) - 1;
      const int offer = who * n + __shfl_sync(0xffffffffu, next, who);
      if (lane == i) mine = offer;
      next += lane == who;
    }
    if (lane < n) select(mine, lane);
  }
  if (told == 0) return;
  __syncthreads();
#pragma unroll 1
  for (uint32_t i = threadIdx.x; i < told; i += kThreads) {
    const uint32_t b = i / width, c = i - b * width;
    const int64_t at = parents[b] * static_cast<int64_t>(width) + c;
    to[i] = c == a.length ? tokens[b] : ahead ? history[at] : from[at];
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

// How rows are cut: vectors of a lane, CTAs of a row, and tiles that each of their
// warps goes over: as many as leave the device one round of CTAs (at most four an
// SM).  Two vectors instead of eight where SMs would else have no CTA, as long as
// a row's parts have no more keys than are ranked at once (one clip of 5 beams,
// 10001 bf16 logits: 8.1 against 8.4 us; 16 beams, 15.6 against 17.0 for 1000
// logits, but 26.1 against 19.9 for 50001, which are 13 parts).
struct Cut {
  int vecs, parts, tiles;
};

Cut cut(const lm_beam_args &a) {
  const int64_t rows = a.clips * a.beams, values = kWarps * 32 * (a.dtype == LM_F32 ? 4 : 8);
  Cut c;
  const int64_t big = (a.vocab + 8 * values - 1) / (8 * values);
  const int64_t small = (a.vocab + 2 * values - 1) / (2 * values);
  c.vecs = rows * big < 152 && small * a.beams <= kGather ? 2 : 8;
  const int64_t all = (a.vocab + c.vecs * values - 1) / (c.vecs * values);
  const int64_t parts = c.vecs == 2 ? all : 4 * 152 / rows > 1 ? 4 * 152 / rows : 1;
  c.tiles = static_cast<int>(parts < all ? (all + parts - 1) / parts : 1);
  c.parts = static_cast<int>((all + c.tiles - 1) / c.tiles);
  return c;
}

template <typename T>
lm_status launch(const BeamParams &p, int vecs, cudaStream_t s) {
  const int64_t ctas = p.a.clips * p.a.beams * p.parts;
  if (ctas > INT_MAX) return LM_ERR_UNSUPPORTED;
  return launch_dependent(vecs == 2 ? beam_kernel<T, 2> : beam_kernel<T, 8>, dim3(static_cast<unsigned>(ctas)),
                          kThreads, 0, s, 1, p);
}

}  // namespace
}  // namespace lm

extern "C" lm_status lm_beam_step_workspace_size(const lm_beam_args *args, size_t *bytes) {
  using namespace lm;
  if (!bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st = check(args); st != LM_OK) return st;
  if (args->clips == 0) {
    *bytes = 256;
    return LM_OK;
  }
  const size_t clips = static_cast<size_t>(args->clips < kClips ? args->clips : kClips);
  *bytes = 256 + kCounterBytes + clips * args->beams * cut(*args).parts * (sizeof(float2) + 8 * args->beams);
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
  const Cut c = cut(a);  // of all clips, also where they take several launches
  p.parts = c.parts;
  p.tiles = c.tiles;
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
      case LM_F32: st = launch<float>(p, c.vecs, s); break;
      case LM_F16: st = launch<__half>(p, c.vecs, s); break;
      default: st = launch<__nv_bfloat16>(p, c.vecs, s); break;
    }
    if (st != LM_OK) return st;
  }
  return LM_OK;
}
