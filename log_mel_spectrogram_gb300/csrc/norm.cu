// norm.cu -- layer norm over the last dimension, forward and backward.
//
// Forward: mean, then the deviations d = x - mean from the rounded mean; their
// own mean puts right what rounding left off, so that
//   var = avg(d^2) - avg(d)^2,  n = (d - avg(d)) / sqrt(var + eps).
// Backward, with h = grad * weight:
//   dx = (h - avg(h) - n avg(h n)) / sqrt(var + eps),
//   dweight = sum over rows of grad n,  dbias = sum over rows of grad.
//
// Memory bounds both: a row is read once and stays in the registers of its team, 8
// to 512 threads with 8 to 32 elements each; teams walk the rows with the next ones
// on their way into shared memory.  Backward, a thread adds its columns'
// parts of dweight and dbias up over all rows of its team; a CTA's teams meet in
// shared memory, and a second kernel joins the CTAs' sums in their order.
//
// Two elements an instruction, and no masks where a team holds exactly the width: with one element and masks
// the issue slots were two thirds full and bound it (24000 x 1024 bf16 forward 22.9 us under the profiler, now 19.5).
//
// Measured, in a graph: 24000 x 1024 f16 forward 18.0 us (5.5 TB/s; 33 to 34 in f32, 5.9 TB/s); with gradients, bf16, 50 us
// (forward 18, backward 27, the join 4) against 29 of memory traffic, and 82 in f32.  24000 x 768 15.0 and 38.5.
// 5 x 1024 1.6 us.  1499 x 771 f32 with gradients 12.3.  Through torch's autograd a pass of forward and backward takes 130
// to 150 us of the host, whatever its size.
//
// Rows wider than a team can hold are read again for each pass, out of L2 (the kernels
// at the end; above 16384 forward, for many rows of 16 bits above 8192, backward above 8192).
#include <climits>

#include "f32x2.cuh"
#include "half.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace lm {
namespace {

constexpr int kMostParts = 512;  // CTAs whose sums over rows are joined
constexpr int kLoopThreads = 256;
constexpr size_t kScratch = 2 * 32 * sizeof(float2);  // of a CTA's shared memory

struct NormParams {
  const void *x, *weight, *bias, *grad;
  void *out;              // y, or dx
  float *stats;           // [3][rows]
  float *partial;         // [parts][2][width], or null
  int64_t rows, width, x_row, grad_row, out_row;
  int32_t weight_f32, bias_f32, parts;
  float eps;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__device__ __forceinline__ float param_at(const void *p, int f32, int64_t i, float otherwise) {
  if (!p) return otherwise;
  return f32 ? static_cast<const float *>(p)[i] : to_f32(static_cast<const T *>(p)[i]);
}

// Sums over a team's threads, for each of them.  A team of several warps has a barrier of its own
// and two places for its warps' sums in turn, so that one wait a sum is enough.
template <int TEAM>
struct TeamSum {
  float2 (*scratch)[32];  // [2][32], warps of the CTA
  int turn = 0;

  __device__ __forceinline__ float2 operator()(float a, float b) {
#pragma unroll
    for (int o = (TEAM < 32 ? TEAM : 32) / 2; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (TEAM > 32) {
      const int warp = static_cast<int>(threadIdx.x) / 32, team = static_cast<int>(threadIdx.x) / TEAM;
      float2 *const at = scratch[turn];
      turn ^= 1;
      if (threadIdx.x % 32 == 0) at[warp] = make_float2(a, b);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(TEAM) : "memory");
      a = b = 0.0f;
#pragma unroll
      for (int i = 0; i < TEAM / 32; ++i) {
        const float2 v = at[team * (TEAM / 32) + i];
        a += v.x;
        b += v.y;
      }
    }
    return make_float2(a, b);
  }
};

// A thread's elements of a row: vectors of 16 bytes, TEAM vectors apart, or (rows off
// 16-byte boundaries) single elements TEAM apart.
template <typename T, int TEAM, int NE, bool VECTORS>
struct Part {
  static constexpr int kEach = VECTORS ? 16 / static_cast<int>(sizeof(T)) : 1;
  static constexpr int kWords = VECTORS ? NE * static_cast<int>(sizeof(T)) / 4 : NE;
  uint32_t w[kWords];

  // Place j of thread t in the row.
  static __device__ __forceinline__ int place(int j, int t) { return (j / kEach * TEAM + t) * kEach + j % kEach; }

  __device__ __forceinline__ void load(const T *row, int width, int t, bool any) {
    if constexpr (VECTORS) {
#pragma unroll
      for (int v = 0; v < NE / kEach; ++v) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (any && place(v * kEach, t) < width) u = *reinterpret_cast<const uint4 *>(row + place(v * kEach, t));
        w[4 * v] = u.x;
        w[4 * v + 1] = u.y;
        w[4 * v + 2] = u.z;
        w[4 * v + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        w[j] = 0;
        if (any && place(j, t) < width) {
          if constexpr (sizeof(T) == 4) {
            w[j] = *reinterpret_cast<const uint32_t *>(row + place(j, t));
          } else {
            w[j] = *reinterpret_cast<const uint16_t *>(row + place(j, t));
          }
        }
      }
    }
  }

  // Elements j and j + 1.
  __device__ __forceinline__ f32x2 two(int j) const {
    float2 v;
    if constexpr (sizeof(T) == 4) v = make_float2(__uint_as_float(w[j]), __uint_as_float(w[j + 1]));
    else if constexpr (VECTORS) v = unpack2<T>(w[j / 2]);
    else v = make_float2(unpack2<T>(w[j]).x, unpack2<T>(w[j + 1]).x);
    return pair(v.x, v.y);
  }

  __device__ __forceinline__ void set(int j, f32x2 v) {
    const float2 f = unpair(v);
    if constexpr (sizeof(T) == 4) {
      w[j] = __float_as_uint(f.x);
      w[j + 1] = __float_as_uint(f.y);
    } else if constexpr (VECTORS) {
      w[j / 2] = pack2<T>(f.x, f.y);
    } else {
      const uint32_t p = pack2<T>(f.x, f.y);
      w[j] = p & 0xffffu;
      w[j + 1] = p >> 16;
    }
  }

  __device__ __forceinline__ void store(T *row, int width, int t) const {
    if constexpr (VECTORS) {
#pragma unroll
      for (int v = 0; v < NE / kEach; ++v)
        if (place(v * kEach, t) < width)
          *reinterpret_cast<uint4 *>(row + place(v * kEach, t)) = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        if (place(j, t) >= width) continue;
        if constexpr (sizeof(T) == 4) {
          *reinterpret_cast<uint32_t *>(row + place(j, t)) = w[j];
        } else {
          *reinterpret_cast<uint16_t *>(row + place(j, t)) = static_cast<uint16_t>(w[j]);
        }
      }
    }
  }
};

// Rows on their way: in shared memory, by asynchronous copies of 16 bytes that each thread makes for itself (three
// rows of 16-bit elements, two of 32), or where rows are off 16-byte boundaries one row in registers.
template <typename P, typename T, int NE, bool VECTORS>
struct Feed {
  static constexpr int kVectors = VECTORS ? NE * static_cast<int>(sizeof(T)) / 16 : 0;
  static constexpr int kSlots = VECTORS ? (sizeof(T) == 2 ? 4 : 3) : 2;
  static constexpr int kAhead = kSlots - 1;
  uint32_t base, step;  // this thread's first vector, and from vector to vector
  uint32_t in, out, last;
  P held;

  // Bytes a thread takes.
  static constexpr size_t kBytes = static_cast<size_t>(VECTORS ? kSlots * kVectors * 16 : 0);

  __device__ __forceinline__ Feed(void *shared) {
    base = static_cast<uint32_t>(__cvta_generic_to_shared(shared)) + threadIdx.x * 16;
    step = blockDim.x * 16;
    in = out = base;
    last = base + (kSlots - 1) * kVectors * step;
  }

  __device__ __forceinline__ void push(const T *row, int width, int t, bool any) {
    if constexpr (VECTORS) {
#pragma unroll
      for (int v = 0; v < kVectors; ++v) {
        const bool there = any && P::place(v * P::kEach, t) < width;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(in + static_cast<uint32_t>(v) * step),
                     "l"(there ? row + P::place(v * P::kEach, t) : row), "r"(there ? 16 : 0)
                     : "memory");
      }
      in = in == last ? base : in + kVectors * step;
    } else {
      held.load(row, width, t, any);
    }
  }

  // The oldest row; its place is written again by the second push from here.
  __device__ __forceinline__ P pop() {
    P r;
    if constexpr (VECTORS) {
#pragma unroll
      for (int v = 0; v < kVectors; ++v)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.w[4 * v]), "=r"(r.w[4 * v + 1]), "=r"(r.w[4 * v + 2]), "=r"(r.w[4 * v + 3])
                     : "r"(out + static_cast<uint32_t>(v) * step)
                     : "memory");
      out = out == last ? base : out + kVectors * step;
    } else {
      r = held;
    }
    return r;
  }

  static __device__ __forceinline__ void commit() {
    if constexpr (VECTORS) asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // All but the last kAhead - 1 rows are there.
  static __device__ __forceinline__ void wait() {
    if constexpr (VECTORS) asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
  }
  static __device__ __forceinline__ void drain() {
    if constexpr (VECTORS) asm volatile("cp.async.wait_all;" ::: "memory");
  }
};

// Two elements, zeros for what lies past the width.
template <typename P, bool FULL>
__device__ __forceinline__ f32x2 within(f32x2 v, int j, int t, int width) {
  if (FULL) return v;
  const float2 f = unpair(v);
  return pair(P::place(j, t) < width ? f.x : 0.0f, P::place(j + 1, t) < width ? f.y : 0.0f);
}

__device__ __forceinline__ float joined(f32x2 v) {
  const float2 f = unpair(v);
  return f.x + f.y;
}

// Threads of a CTA that is alone on its SM, for so many registers a thread: whole teams, at most 15
// of several warps (a CTA has 16 barriers).
constexpr int threads_for(int team, int regs) {
  const int most = 65536 / ((regs + 7) / 8 * 8) / 32 * 32;
  const int teams = (most < 1024 ? most : 1024) / team;
  return teams < 1 ? team : team > 32 && teams > 15 ? 15 * team : (teams * team) / 32 * 32;
}

// ---- forward ----

// The weight and bias stay in registers where a thread has 8 elements, else in shared memory; for teams of 512 with 32
// elements, whose rows take it all, they are read from the L1 each time.
template <typename P, int NE>
constexpr int forward_regs() { return 62 + P::kWords / 2 + NE + (NE == 8 ? 16 : 0); }
// Several teams of a CTA share the weight and bias.  (Vectors of 32 bits: a CTA of 128 threads, for the room
// that their rows take.)
template <typename P, int TEAM, int NE>
constexpr int forward_threads() { return TEAM <= 32 || (TEAM <= 128 && P::kEach != 4) ? 256 : TEAM < 128 ? 128 : TEAM; }
template <typename P, int TEAM, int NE>
constexpr int forward_ctas() {
  const int n = threads_for(32, forward_regs<P, NE>()) / forward_threads<P, TEAM, NE>();
  return n < 1 ? 1 : n;
}

// FULL: the width is what a team holds.
template <typename T, int TEAM, int NE, bool VECTORS, bool FULL>
__global__ void __launch_bounds__(forward_threads<Part<T, TEAM, NE, VECTORS>, TEAM, NE>(),
                                  forward_ctas<Part<T, TEAM, NE, VECTORS>, TEAM, NE>()) norm_rows(const NormParams p) {
  using P = Part<T, TEAM, NE, VECTORS>;
  constexpr bool HOLD = NE == 8, SHARED = !HOLD && TEAM * NE <= 8192;
  extern __shared__ float4 dynamic[];  // the sums' places; then weight and bias of two elements, [NE / 2][TEAM]
  TeamSum<TEAM> sum{reinterpret_cast<float2(*)[32]>(dynamic)};
  float4 *const params = dynamic + kScratch / sizeof(float4);
  const int t = static_cast<int>(threadIdx.x) % TEAM, width = FULL ? TEAM * NE : static_cast<int>(p.width);
  const int64_t teams = static_cast<int64_t>(gridDim.x) * (blockDim.x / TEAM);
  const int64_t team = static_cast<int64_t>(blockIdx.x) * (blockDim.x / TEAM) + threadIdx.x / TEAM;
  const int64_t lead = TEAM < 32 ? team - threadIdx.x % 32 / TEAM : team;  // the warp's first
  const float inv = 1.0f / static_cast<float>(width);
  pdl_launch();
  pdl_wait();
  Feed<P, T, NE, VECTORS> feed(params + (SHARED ? NE / 2 * TEAM : 0));
  const int64_t x_step = teams * p.x_row;
  const T *x = static_cast<const T *>(p.x) + team * p.x_row;
  int64_t fetched = team;  // the row to fetch next
  auto push = [&]() {
    feed.push(fetched < p.rows ? x : static_cast<const T *>(p.x), width, t, fetched < p.rows);
    feed.commit();
    x += x_step;
    fetched += teams;
  };
#pragma unroll
  for (int i = 0; i < feed.kAhead; ++i) push();
  auto param = [&](int j, int thread) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int i = P::place(j, thread), k = P::place(j + 1, thread);
    if (i < width) {
      v.x = param_at<T>(p.weight, p.weight_f32, i, 1.0f);
      v.z = param_at<T>(p.bias, p.bias_f32, i, 0.0f);
    }
    if (k < width) {
      v.y = param_at<T>(p.weight, p.weight_f32, k, 1.0f);
      v.w = param_at<T>(p.bias, p.bias_f32, k, 0.0f);
    }
    return v;
  };
  float4 held[HOLD ? NE / 2 : 1];
  if (HOLD) {
#pragma unroll
    for (int j = 0; j < NE; j += 2) held[HOLD ? j / 2 : 0] = param(j, t);
  } else if (SHARED) {
    for (int i = threadIdx.x; i < NE / 2 * TEAM; i += blockDim.x) params[i] = param(i / TEAM * 2, i % TEAM);
    __syncthreads();
  }
  for (int64_t row = team, first = lead; first < p.rows; row += teams, first += teams) {
    const bool any = row < p.rows;
    f32x2 v[NE / 2], s = both(0.0f), q = both(0.0f);
    feed.wait();
    const P now = feed.pop();
    push();
#pragma unroll
    for (int j = 0; j < NE; j += 2) {
      v[j / 2] = now.two(j);
      s = add2(s, v[j / 2]);
    }
    const float mean = sum(joined(s), 0.0f).x * inv;
    s = both(0.0f);
#pragma unroll
    for (int j = 0; j < NE; j += 2) {
      const f32x2 d = within<P, FULL>(add2(v[j / 2], both(-mean)), j, t, width);
      v[j / 2] = d;
      s = add2(s, d);
      q = fma2(d, d, q);
    }
    const float2 u = sum(joined(s), joined(q));
    const float off = u.x * inv, var = u.y * inv - off * off;
    const float r = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + p.eps);
    if (p.stats && t == 0 && any) {
      p.stats[row] = mean;
      p.stats[p.rows + row] = off;
      p.stats[2 * p.rows + row] = r;
    }
    if (!any) continue;
    P out;
    const f32x2 r2 = both(r), c2 = both(-off * r);
#pragma unroll
    for (int j = 0; j < NE; j += 2) {
      const float4 c = HOLD ? held[HOLD ? j / 2 : 0] : SHARED ? params[j / 2 * TEAM + t] : param(j, t);
      out.set(j, fma2(fma2(v[j / 2], r2, c2), pair(c.x, c.y), pair(c.z, c.w)));
    }
    out.store(static_cast<T *>(p.out) + row * p.out_row, width, t);
  }
  feed.drain();
}

// ---- backward ----

// Registers that a thread needs, and shared memory for its rows.
template <typename P, int TEAM, int NE>
constexpr int backward_threads() { return threads_for(TEAM, 58 + 4 * NE + (P::kEach == 1 ? 2 * P::kWords : 0)); }

template <typename T, int TEAM, int NE, bool VECTORS, bool FULL>
__global__ void __launch_bounds__(backward_threads<Part<T, TEAM, NE, VECTORS>, TEAM, NE>(), 1)
    norm_backward(const NormParams p) {
  using P = Part<T, TEAM, NE, VECTORS>;
  constexpr int PLACES = NE * TEAM;
  using Rows = Feed<P, T, NE, VECTORS>;
  // The sums' places; the weight of two elements, [NE / 2][TEAM]; rows of x and of the gradient, later [..][NE][TEAM].
  extern __shared__ float4 dynamic[];
  TeamSum<TEAM> sum{reinterpret_cast<float2(*)[32]>(dynamic)};
  float2 *const shared = reinterpret_cast<float2 *>(dynamic + kScratch / sizeof(float4));
  const int t = static_cast<int>(threadIdx.x) % TEAM, width = FULL ? TEAM * NE : static_cast<int>(p.width);
  const int64_t teams = static_cast<int64_t>(gridDim.x) * (blockDim.x / TEAM);
  const int64_t team = static_cast<int64_t>(blockIdx.x) * (blockDim.x / TEAM) + threadIdx.x / TEAM;
  const int64_t lead = TEAM < 32 ? team - threadIdx.x % 32 / TEAM : team;
  const float inv = 1.0f / static_cast<float>(width);
  f32x2 dw2[NE / 2], db2[NE / 2];
#pragma unroll
  for (int j = 0; j < NE / 2; ++j) dw2[j] = db2[j] = both(0.0f);
  pdl_launch();
  pdl_wait();
  char *const rows = reinterpret_cast<char *>(shared + PLACES / 2);
  Rows feed_x(rows), feed_g(rows + Rows::kBytes * blockDim.x);
  const int64_t x_step = teams * p.x_row, g_step = teams * p.grad_row;
  const T *from_x = static_cast<const T *>(p.x) + team * p.x_row, *from_g = static_cast<const T *>(p.grad) + team * p.grad_row;
  int64_t fetched = team;  // the row to fetch next
  auto push = [&]() {
    const bool there = fetched < p.rows;
    feed_x.push(there ? from_x : static_cast<const T *>(p.x), width, t, there);
    feed_g.push(there ? from_g : static_cast<const T *>(p.grad), width, t, there);
    Rows::commit();
    from_x += x_step;
    from_g += g_step;
    fetched += teams;
  };
#pragma unroll
  for (int i = 0; i < Rows::kAhead; ++i) push();
  float mean = 0.0f, off = 0.0f, r = 0.0f;
  auto load_stats = [&](int64_t row) {
    if (row >= p.rows) {  // (a warp's other teams have one: zeros for n here, which the last row's mean need not give)
      mean = off = r = 0.0f;
      return;
    }
    mean = p.stats[row];
    off = p.stats[p.rows + row];
    r = p.stats[2 * p.rows + row];
  };
  load_stats(team);
  for (int i = threadIdx.x; i < PLACES / 2; i += blockDim.x) {
    const int a = P::place(i / TEAM * 2, i % TEAM), b = P::place(i / TEAM * 2 + 1, i % TEAM);
    shared[i] = make_float2(a < width ? param_at<T>(p.weight, p.weight_f32, a, 1.0f) : 0.0f,
                            b < width ? param_at<T>(p.weight, p.weight_f32, b, 1.0f) : 0.0f);
  }
  __syncthreads();
  for (int64_t row = team, first = lead; first < p.rows; row += teams, first += teams) {
    f32x2 n[NE / 2], h[NE / 2], s = both(0.0f), q = both(0.0f);
    const f32x2 m2 = both(-mean), r2 = both(r), o2 = both(-off * r);
    const float scale = r;
    Rows::wait();
    const P x = feed_x.pop(), e = feed_g.pop();
    push();
    load_stats(row + teams);
#pragma unroll
    for (int j = 0; j < NE; j += 2) {
      const float2 w = shared[j / 2 * TEAM + t];
      // (A place past the width has no part, whatever its row.)
      const f32x2 g = e.two(j), u = within<P, FULL>(fma2(add2(x.two(j), m2), r2, o2), j, t, width);
      n[j / 2] = u;
      h[j / 2] = mul2(g, pair(w.x, w.y));
      s = add2(s, h[j / 2]);
      q = fma2(h[j / 2], u, q);
      dw2[j / 2] = fma2(g, u, dw2[j / 2]);
      db2[j / 2] = add2(db2[j / 2], g);
    }
    const float2 u = sum(joined(s), joined(q));
    if (p.out && row < p.rows) {
      // dx = h r - avg(h) r - n avg(h n) r
      const f32x2 k = both(scale), c1 = both(-(u.x * inv) * scale), c2 = both(-(u.y * inv) * scale);
      P out;
#pragma unroll
      for (int j = 0; j < NE; j += 2) out.set(j, fma2(n[j / 2], c2, fma2(h[j / 2], k, c1)));
      out.store(static_cast<T *>(p.out) + row * p.out_row, width, t);
    }
  }
  Rows::drain();
  if (!p.partial) return;
  __syncthreads();  // the rows' places are free
  float dw[NE], db[NE];
#pragma unroll
  for (int j = 0; j < NE; j += 2) {
    const float2 a = unpair(dw2[j / 2]), b = unpair(db2[j / 2]);
    dw[j] = a.x;
    dw[j + 1] = a.y;
    db[j] = b.x;
    db[j + 1] = b.y;
  }
  // A warp's teams join by shuffles; then the upper half of the groups (teams, or warps of smaller ones) hand
  // their sums to the lower, until one is left.
  constexpr int GROUP = TEAM < 32 ? 32 : TEAM;
#pragma unroll
  for (int o = 16; o >= TEAM; o >>= 1)
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], o);
      db[j] += __shfl_xor_sync(0xffffffffu, db[j], o);
    }
  const int group = static_cast<int>(threadIdx.x) / GROUP;
  const bool mine = static_cast<int>(threadIdx.x) % GROUP < TEAM;
  float2 *const slots = reinterpret_cast<float2 *>(rows);
  for (int n = static_cast<int>(blockDim.x) / GROUP; n > 1;) {
    const int half = (n + 1) / 2;
    if (group >= half && group < n && mine) {
#pragma unroll
      for (int j = 0; j < NE; ++j) slots[(group - half) * PLACES + j * TEAM + t] = make_float2(dw[j], db[j]);
    }
    __syncthreads();
    if (group < n - half && mine) {
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        const float2 v = slots[group * PLACES + j * TEAM + t];
        dw[j] += v.x;
        db[j] += v.y;
      }
    }
    __syncthreads();
    n = half;
  }
  if (group != 0 || !mine) return;
  float *const to = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * width;
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int at = P::place(j, t);
    if (at >= width) continue;
    to[at] = dw[j];
    to[width + at] = db[j];
  }
}

// Joins the parts: a CTA has 32 columns, warp w parts w, w + 32, ..., and then one column.
template <typename T>
__global__ void __launch_bounds__(1024) norm_join(const float *partial, int parts, int64_t width, void *dweight,
                                                  int weight_f32, void *dbias, int bias_f32) {
  __shared__ float sums[32][33];
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (i < 2 * width) {
#pragma unroll 8
    for (int c = warp; c < parts; c += 32) s += partial[static_cast<int64_t>(c) * 2 * width + i];
  }
  sums[warp][lane] = s;
  __syncthreads();
  s = warp_sum(sums[lane][warp]);
  i = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  void *const to = i < width ? dweight : dbias;
  if (lane != 0 || i >= 2 * width || !to) return;
  const int64_t at = i < width ? i : i - width;
  if (i < width ? weight_f32 : bias_f32) {
    static_cast<float *>(to)[at] = s;
  } else {
    static_cast<T *>(to)[at] = from_f32<T>(s);
  }
}

// ---- rows that no team holds ----

// The sums of two values over the CTA, for every thread.
__device__ __forceinline__ float2 cta_sum2(float a, float b, float2 *scratch) {
  a = warp_sum(a);
  b = warp_sum(b);
  __syncthreads();
  if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = make_float2(a, b);
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
  for (int i = 0; i < kLoopThreads / 32; ++i) {
    s.x += scratch[i].x;
    s.y += scratch[i].y;
  }
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kLoopThreads) norm_rows_loop(const NormParams p) {
  __shared__ float2 scratch[kLoopThreads / 32];
  pdl_launch();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const T *const x = static_cast<const T *>(p.x) + row * p.x_row;
  T *const out = static_cast<T *>(p.out) + row * p.out_row;
  const float inv = 1.0f / static_cast<float>(p.width);
  float s = 0.0f, q = 0.0f;
  for (int64_t i = threadIdx.x; i < p.width; i += kLoopThreads) s += to_f32(x[i]);
  const float mean = cta_sum2(s, 0.0f, scratch).x * inv;
  s = 0.0f;
  for (int64_t i = threadIdx.x; i < p.width; i += kLoopThreads) {
    const float d = to_f32(x[i]) - mean;
    s += d;
    q += d * d;
  }
  const float2 t = cta_sum2(s, q, scratch);
  const float off = t.x * inv, var = t.y * inv - off * off;
  const float r = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + p.eps);
  if (p.stats && threadIdx.x == 0) {
    p.stats[row] = mean;
    p.stats[p.rows + row] = off;
    p.stats[2 * p.rows + row] = r;
  }
  for (int64_t i = threadIdx.x; i < p.width; i += kLoopThreads) {
    const float n = ((to_f32(x[i]) - mean) - off) * r;
    out[i] = from_f32<T>(n * param_at<T>(p.weight, p.weight_f32, i, 1.0f) + param_at<T>(p.bias, p.bias_f32, i, 0.0f));
  }
}

template <typename T>
__global__ void __launch_bounds__(kLoopThreads) norm_backward_rows_loop(const NormParams p) {
  __shared__ float2 scratch[kLoopThreads / 32];
  pdl_launch();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const T *const x = static_cast<const T *>(p.x) + row * p.x_row;
  const T *const g = static_cast<const T *>(p.grad) + row * p.grad_row;
  T *const out = static_cast<T *>(p.out) + row * p.out_row;
  const float mean = p.stats[row], off = p.stats[p.rows + row], r = p.stats[2 * p.rows + row];
  const float inv = 1.0f / static_cast<float>(p.width);
  float s = 0.0f, q = 0.0f;
  for (int64_t i = threadIdx.x; i < p.width; i += kLoopThreads) {
    const float n = ((to_f32(x[i]) - mean) - off) * r;
    const float h = to_f32(g[i]) * param_at<T>(p.weight, p.weight_f32, i, 1.0f);
    s += h;
    q += h * n;
  }
  const float2 t = cta_sum2(s, q, scratch);
  for (int64_t i = threadIdx.x; i < p.width; i += kLoopThreads) {
    const float n = ((to_f32(x[i]) - mean) - off) * r;
    const float h = to_f32(g[i]) * param_at<T>(p.weight, p.weight_f32, i, 1.0f);
    out[i] = from_f32<T>((h - t.x * inv - n * (t.y * inv)) * r);
  }
}

// Sums over a part of the rows (blockIdx.y) for a thread's column.
template <typename T>
__global__ void __launch_bounds__(kLoopThreads) norm_backward_columns_loop(const NormParams p) {
  pdl_launch();
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kLoopThreads + threadIdx.x;
  if (i >= p.width) return;
  const int64_t first = p.rows * blockIdx.y / p.parts, end = p.rows * (blockIdx.y + 1) / p.parts;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = first; row < end; ++row) {
    const float g = to_f32(static_cast<const T *>(p.grad)[row * p.grad_row + i]);
    const float d = to_f32(static_cast<const T *>(p.x)[row * p.x_row + i]) - p.stats[row];
    dw += g * ((d - p.stats[p.rows + row]) * p.stats[2 * p.rows + row]);
    db += g;
  }
  float *const to = p.partial + static_cast<int64_t>(blockIdx.y) * 2 * p.width + i;
  to[0] = dw;
  to[p.width] = db;
}

int64_t size_of(int32_t dtype) { return dtype == LM_F32 ? 4 : 2; }
bool aligned(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(n) == 0; }
bool float_type(int32_t t) { return t == LM_F32 || t == LM_F16 || t == LM_BF16; }

lm_status check_sizes(int64_t rows, int64_t width, int64_t x_row, int64_t other_row, int32_t dtype, int32_t weight_dtype,
                      int32_t bias_dtype) {
  if (rows < 0 || width < 0 || x_row < 0 || other_row < 0) return LM_ERR_INVALID_ARG;
  if (!float_type(dtype) || (weight_dtype != LM_F32 && weight_dtype != dtype) ||
      (bias_dtype != LM_F32 && bias_dtype != dtype))
    return LM_ERR_UNSUPPORTED;
  const int64_t most = INT_MAX - 512;
  if (rows > most || width > most || (width > 0 && rows > (1ll << 60) / width) || x_row > (1ll << 38) ||
      other_row > (1ll << 38))
    return LM_ERR_UNSUPPORTED;
  return LM_OK;
}

int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

// Whether rows and their step are whole vectors of 16 bytes.
bool vectors(const void *p, int64_t step, int64_t rows, int64_t size) {
  return aligned(p, 16) && (rows == 1 || step * size % 16 == 0);
}

// Threads a row and elements a thread.
struct Shape {
  int team, each;
};

// Few rows are shared out among many threads, for the least time of one; of many, as few threads as hold one, with
// 24 or 32 elements each: a team's sums wait for one another, so that more rows at once count for more (bf16, 96 MB in
// and out: 19660 x 1280 24.4 us, with 128 threads of 16 elements 47; 12288 x 2048 19.5, 33.5; 4096 x 6144 24.6, 36.5
// with 512 of 16; in f32 above 4096 those are the faster, because a CTA's rows take an SM's shared memory).  Many rows
// of 16 bits above 8192 are read again instead of kept: 1536 x 16384 45 us, 70 with 512 threads of 32.
Shape forward_shape(int64_t rows, int64_t width, int64_t size, int sms) {
  const bool few = rows <= 4 * sms;
  if (width > 512 * 32) return {0, 0};
  if (width <= 64) return {8, 8};
  if (width <= 128) return {16, 8};
  if (width <= 256) return {32, 8};
  if (few) return width <= 1024 ? Shape{128, 8} : Shape{512, width <= 4096 ? 8 : width <= 8192 ? 16 : 32};
  if (width <= 512) return {32, 16};
  if (width > 8192 && size == 2) return {0, 0};
  int team = 32;
  while (team * 32 < width) team *= 2;
  if (team == 512 || (team == 256 && size == 4)) return {512, width <= 8192 ? 16 : 32};
  return {team, width <= 24 * team ? 24 : 32};
}

// At most 24 elements a thread, 16 where rows are off 16-byte boundaries (and wait in registers): it also holds
// their sums over rows.
Shape backward_shape(int64_t width, bool vectors) {
  if (width > 512 * 16) return {0, 0};
  if (width <= 64) return {8, 8};
  if (width <= 128) return {16, 8};
  if (width <= 256) return {32, 8};
  if (vectors && width > 512 && width <= 768) return {32, 24};
  int team = 32;
  while (team * 16 < width) team *= 2;
  return {team, 16};
}

// Threads of a CTA of whole teams, at most `most`: few enough for every SM to have some.
int spread(int team, int64_t rows, int most, int sms) {
  const int unit = team < 32 ? 32 : team;
  const int64_t units = (rows * team + unit - 1) / unit;
  return unit * static_cast<int>(least(most / unit, (units + sms - 1) / sms));
}

template <typename T, int TEAM, int NE, bool VECTORS>
lm_status forward_as(const NormParams &p, int sms, cudaStream_t s) {
  using P = Part<T, TEAM, NE, VECTORS>;
  constexpr int most = forward_threads<P, TEAM, NE>();
  const int threads = spread(TEAM, p.rows, most, sms);
  const int64_t ctas = (p.rows + threads / TEAM - 1) / (threads / TEAM);
  const size_t shared = kScratch + (NE == 8 || TEAM * NE > 8192 ? 0 : sizeof(float4) * NE / 2 * TEAM) +
                        Feed<P, T, NE, VECTORS>::kBytes * static_cast<size_t>(threads);
  int64_t each = forward_ctas<P, TEAM, NE>() * (most / threads);  // CTAs of an SM
  each = least(each, static_cast<int64_t>(222 * 1024 / (shared + 1024)));
  if (each < 1) each = 1;
  const auto kernel = VECTORS && p.width == TEAM * NE ? norm_rows<T, TEAM, NE, VECTORS, VECTORS> : norm_rows<T, TEAM, NE, VECTORS, false>;
  if (shared > 40 * 1024)
    if (lm_status st = ensure_smem_attribute(reinterpret_cast<const void *>(kernel), static_cast<int>(shared)); st != LM_OK)
      return st;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(least(ctas, sms * each))), threads, shared, s, 1, p);
}

template <typename T, int TEAM, int NE, bool VECTORS>
lm_status backward_as(NormParams &p, int sms, cudaStream_t s) {
  using P = Part<T, TEAM, NE, VECTORS>;
  const int threads = spread(TEAM, p.rows, backward_threads<P, TEAM, NE>(), sms);
  const int64_t ctas = (p.rows + threads / TEAM - 1) / (threads / TEAM);
  p.parts = static_cast<int>(least(least(ctas, kMostParts), sms));
  const int groups = threads / (TEAM < 32 ? 32 : TEAM);
  const size_t rows = 2 * Feed<P, T, NE, VECTORS>::kBytes * static_cast<size_t>(threads);
  const size_t sums = sizeof(float2) * TEAM * NE * static_cast<size_t>(groups / 2);
  const size_t shared = kScratch + sizeof(float2) * TEAM * NE / 2 + (rows > sums ? rows : sums);
  const auto kernel =
      VECTORS && p.width == TEAM * NE ? norm_backward<T, TEAM, NE, VECTORS, VECTORS> : norm_backward<T, TEAM, NE, VECTORS, false>;
  if (shared > 40 * 1024)
    if (lm_status st = ensure_smem_attribute(reinterpret_cast<const void *>(kernel), static_cast<int>(shared)); st != LM_OK)
      return st;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(p.parts)), threads, shared, s, 1, p);
}

template <typename T, bool VECTORS>
lm_status forward_shaped(const NormParams &p, Shape h, int sms, cudaStream_t s) {
  if (h.team == 8) return forward_as<T, 8, 8, VECTORS>(p, sms, s);
  if (h.team == 16) return forward_as<T, 16, 8, VECTORS>(p, sms, s);
  if (h.team == 32)
    return h.each == 8    ? forward_as<T, 32, 8, VECTORS>(p, sms, s)
           : h.each == 16 ? forward_as<T, 32, 16, VECTORS>(p, sms, s)
           : h.each == 24 ? forward_as<T, 32, 24, VECTORS>(p, sms, s)
                          : forward_as<T, 32, 32, VECTORS>(p, sms, s);
  if (h.team == 64) return h.each == 24 ? forward_as<T, 64, 24, VECTORS>(p, sms, s) : forward_as<T, 64, 32, VECTORS>(p, sms, s);
  if (h.team == 128)
    return h.each == 8    ? forward_as<T, 128, 8, VECTORS>(p, sms, s)
           : h.each == 24 ? forward_as<T, 128, 24, VECTORS>(p, sms, s)
                          : forward_as<T, 128, 32, VECTORS>(p, sms, s);
  if constexpr (sizeof(T) == 2)
    if (h.team == 256)
      return h.each == 24 ? forward_as<T, 256, 24, VECTORS>(p, sms, s) : forward_as<T, 256, 32, VECTORS>(p, sms, s);
  return h.each == 8    ? forward_as<T, 512, 8, VECTORS>(p, sms, s)
         : h.each == 16 ? forward_as<T, 512, 16, VECTORS>(p, sms, s)
                        : forward_as<T, 512, 32, VECTORS>(p, sms, s);
}

template <typename T, bool VECTORS>
lm_status backward_shaped(NormParams &p, Shape h, int sms, cudaStream_t s) {
  switch (h.team) {
    case 8: return backward_as<T, 8, 8, VECTORS>(p, sms, s);
    case 16: return backward_as<T, 16, 8, VECTORS>(p, sms, s);
    case 32:
      return h.each == 8    ? backward_as<T, 32, 8, VECTORS>(p, sms, s)
             : h.each == 16 ? backward_as<T, 32, 16, VECTORS>(p, sms, s)
                            : backward_as<T, 32, VECTORS ? 24 : 16, VECTORS>(p, sms, s);
    case 64: return backward_as<T, 64, 16, VECTORS>(p, sms, s);
    case 128: return backward_as<T, 128, 16, VECTORS>(p, sms, s);
    case 256: return backward_as<T, 256, 16, VECTORS>(p, sms, s);
    default: return backward_as<T, 512, 16, VECTORS>(p, sms, s);
  }
}

template <typename T>
lm_status forward(const NormParams &p, cudaStream_t s) {
  DeviceInfo dev;
  if (lm_status st = current_device_info(&dev); st != LM_OK) return st;
  const Shape h = forward_shape(p.rows, p.width, sizeof(T), dev.sm_count);
  if (h.team == 0)
    return launch_dependent(norm_rows_loop<T>, dim3(static_cast<unsigned>(p.rows)), kLoopThreads, 0, s, 1, p);
  const int64_t size = sizeof(T);
  const bool v = p.width * size % 16 == 0 && vectors(p.x, p.x_row, p.rows, size) && vectors(p.out, p.out_row, p.rows, size);
  return v ? forward_shaped<T, true>(p, h, dev.sm_count, s) : forward_shaped<T, false>(p, h, dev.sm_count, s);
}

template <typename T>
lm_status backward(NormParams p, void *dweight, void *dbias, cudaStream_t s) {
  if (!dweight && !dbias) p.partial = nullptr;
  float *const partial = p.partial;
  if (p.rows > 0) {
    DeviceInfo dev;
    if (lm_status st = current_device_info(&dev); st != LM_OK) return st;
    const int64_t size = sizeof(T);
    const bool v = p.width * size % 16 == 0 && vectors(p.x, p.x_row, p.rows, size) &&
                   vectors(p.grad, p.grad_row, p.rows, size) && vectors(p.out, p.out_row, p.rows, size);
    const Shape h = backward_shape(p.width, v);
    if (h.team != 0) {
      if (lm_status st = v ? backward_shaped<T, true>(p, h, dev.sm_count, s) : backward_shaped<T, false>(p, h, dev.sm_count, s);
          st != LM_OK)
        return st;
    } else {
      if (p.out)
        if (lm_status st = launch_dependent(norm_backward_rows_loop<T>, dim3(static_cast<unsigned>(p.rows)), kLoopThreads, 0,
                                            s, 1, p);
            st != LM_OK)
          return st;
      p.parts = static_cast<int>(least(p.rows, 256));
      const unsigned across = static_cast<unsigned>((p.width + kLoopThreads - 1) / kLoopThreads);
      if (partial)
        if (lm_status st = launch_dependent(norm_backward_columns_loop<T>, dim3(across, static_cast<unsigned>(p.parts)),
                                            kLoopThreads, 0, s, 1, p);
            st != LM_OK)
          return st;
    }
  }
  if (!partial) return LM_OK;
  return launch_dependent(norm_join<T>, dim3(static_cast<unsigned>((2 * p.width + 31) / 32)), 1024, 0, s, 1,
                          static_cast<const float *>(partial), p.parts, p.width, dweight, p.weight_f32, dbias, p.bias_f32);
}

}  // namespace
}  // namespace lm

extern "C" lm_status lm_layer_norm(const lm_norm_args *a, lm_stream_t stream) {
  using namespace lm;
  if (!a) return LM_ERR_INVALID_ARG;
  if (lm_status st =
          check_sizes(a->rows, a->width, a->x_row_stride, a->out_row_stride, a->dtype, a->weight_dtype, a->bias_dtype);
      st != LM_OK)
    return st;
  if (!(a->eps >= 0.0f)) return LM_ERR_INVALID_ARG;
  if (a->rows == 0 || a->width == 0) return LM_OK;
  if (!a->x || !a->out) return LM_ERR_INVALID_ARG;
  const int64_t size = size_of(a->dtype), ws = size_of(a->weight_dtype), bs = size_of(a->bias_dtype);
  if (!aligned(a->x, size) || !aligned(a->out, size) || !aligned(a->weight, ws) || !aligned(a->bias, bs) ||
      !aligned(a->stats, 4))
    return LM_ERR_MISALIGNED;
  const ByteRows out{a->out, a->rows, a->out_row_stride * size, a->width * size};
  const ByteRows x{a->x, a->rows, a->x_row_stride * size, a->width * size};
  const bool same = a->out == a->x && (a->rows == 1 || a->out_row_stride == a->x_row_stride);
  if ((a->rows > 1 && a->out_row_stride < a->width) || (!same && rows_meet(out, x)) ||
      (a->weight && rows_meet(out, {a->weight, 1, 0, a->width * ws})) ||
      (a->bias && rows_meet(out, {a->bias, 1, 0, a->width * bs})))
    return LM_ERR_INVALID_ARG;
  if (a->stats) {
    const ByteRows stats{a->stats, 1, 0, a->rows * 12};
    if (rows_meet(stats, out) || rows_meet(stats, x) || (a->weight && rows_meet(stats, {a->weight, 1, 0, a->width * ws})) ||
        (a->bias && rows_meet(stats, {a->bias, 1, 0, a->width * bs})))
      return LM_ERR_INVALID_ARG;
  }
  NormParams p = {};
  p.x = a->x;
  p.weight = a->weight;
  p.bias = a->bias;
  p.out = a->out;
  p.stats = a->stats;
  p.rows = a->rows;
  p.width = a->width;
  p.x_row = a->x_row_stride;
  p.out_row = a->out_row_stride;
  p.weight_f32 = a->weight_dtype == LM_F32;
  p.bias_f32 = a->bias_dtype == LM_F32;
  p.eps = a->eps;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return a->dtype == LM_F32 ? forward<float>(p, s) : a->dtype == LM_F16 ? forward<__half>(p, s)
                                                                       : forward<__nv_bfloat16>(p, s);
}

extern "C" lm_status lm_layer_norm_backward_workspace_size(const lm_norm_backward_args *a, size_t *bytes) {
  using namespace lm;
  if (!a || !bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st =
          check_sizes(a->rows, a->width, a->x_row_stride, a->grad_row_stride, a->dtype, a->weight_dtype, a->bias_dtype);
      st != LM_OK)
    return st;
  *bytes = 256 + static_cast<size_t>(a->rows < lm::kMostParts ? a->rows : lm::kMostParts) * 8 * static_cast<size_t>(a->width);
  return LM_OK;
}

extern "C" lm_status lm_layer_norm_backward(const lm_norm_backward_args *a, void *workspace, size_t workspace_bytes,
                                            lm_stream_t stream) {
  using namespace lm;
  size_t need = 0;
  if (lm_status st = lm_layer_norm_backward_workspace_size(a, &need); st != LM_OK) return st;
  if (a->width == 0 || (!a->dx && !a->dweight && !a->dbias)) return LM_OK;
  if (a->rows > 0 && (!a->x || !a->grad || !a->stats)) return LM_ERR_INVALID_ARG;
  const int64_t size = size_of(a->dtype), ws = size_of(a->weight_dtype), bs = size_of(a->bias_dtype);
  if (!aligned(a->x, size) || !aligned(a->grad, size) || !aligned(a->dx, size) || !aligned(a->weight, ws) ||
      !aligned(a->dweight, ws) || !aligned(a->dbias, bs) || !aligned(a->stats, 4) || !aligned(workspace, 16))
    return LM_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < need) return LM_ERR_WORKSPACE;
  const ByteRows in[] = {{a->x, a->rows, a->x_row_stride * size, a->width * size},
                         {a->grad, a->rows, a->grad_row_stride * size, a->width * size},
                         {a->weight, a->weight ? 1 : 0, 0, a->width * ws},
                         {a->stats, 1, 0, a->rows * 12}};
  const ByteRows outs[] = {{a->dx, a->dx ? 1 : 0, 0, a->rows * a->width * size},
                           {a->dweight, a->dweight ? 1 : 0, 0, a->width * ws},
                           {a->dbias, a->dbias ? 1 : 0, 0, a->width * bs}};
  for (int i = 0; i < 3; ++i) {
    for (const ByteRows &r : in)
      if (rows_meet(outs[i], r)) return LM_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (rows_meet(outs[i], outs[j])) return LM_ERR_INVALID_ARG;
  }
  NormParams p = {};
  p.x = a->x;
  p.weight = a->weight;
  p.grad = a->grad;
  p.out = a->dx;
  p.stats = const_cast<float *>(a->stats);
  p.partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + 256);
  p.rows = a->rows;
  p.width = a->width;
  p.x_row = a->x_row_stride;
  p.grad_row = a->grad_row_stride;
  p.out_row = a->width;
  p.weight_f32 = a->weight_dtype == LM_F32;
  p.bias_f32 = a->bias_dtype == LM_F32;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return a->dtype == LM_F32   ? backward<float>(p, a->dweight, a->dbias, s)
         : a->dtype == LM_F16 ? backward<__half>(p, a->dweight, a->dbias, s)
                              : backward<__nv_bfloat16>(p, a->dweight, a->dbias, s);
}
