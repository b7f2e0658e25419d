// kv_attend.cu -- attention over the 8-bit key/value cache.
//
// A CTA serves one row and key head: the row's queries that read that head
// (tokens x group) fill tiles of 16 rows, and each of its four warps
// walks its own tiles of 32 tokens with a running maximum and sum per row (enum Mode
// has two other ways, for many rows of few tokens and for many queries).  A
// warp fetches keys and values -- contiguous pieces of a block -- by bulk
// copies into a ring of its own, so warps never wait for one another until
// the end, and only the bytes of the cache travel.
//
// Bytes become 16-bit floats exactly, in registers, on their way into
// m16n8k16 products with 32-bit sums: decoding has few query rows and is bound by
// the cache's bytes, so the products only have to keep up with those (16 query
// rows at full memory speed are 0.2 PFLOP/s).
//
// The order of head elements in a product over k, and of tokens within 16, is
// free: a thread takes contiguous bytes of its token as its part of k, and
// every fourth token, which makes the shared-memory reads wide and free of
// conflicts.
//
// Scales.  With s = scale * q k8 * k_scale * log2 e, a token's weight times its
// value scale is 2^(s + log2 v_scale); the running maximum M is taken over
// those exponents, so that the weights p = 2^(s + log2 v_scale - M) that
// multiply v8 are at most 1 and keep their precision in 16 bits whatever the
// block's scale; the softmax's sum is that of p / v_scale, in 32 bits.
//
// Long rows are split over CTAs; the last one to finish a row and head joins
// the parts in order.
//
// Measured: 5 queries of 64 rows over up to 1500 tokens, 16 heads of 64, 36.6 us
// (3.3 TB/s: 1024 CTAs in two rounds, each 4 us of start-up and end; in between
// latency, as a warp's products, maxima, exponentials and products follow one another:
// 0.48 instructions a cycle from 21% of the warps, which is what registers allow); two rows of
// 131000 tokens, 8 heads of 128, 97 us (5.5 TB/s, 83% of copy bandwidth); a step of 5 rows of
// up to 448 tokens, 6.3 us (launch, three dependent loads, the join of 4 warps).
// 223 causal queries over up to 448 tokens, 16 rows of 16 heads, 33.4 us (74 TFLOP/s):
// start-up and end of CTAs that have at most 14 tiles, and the tensor pipe at 22%.
#include <climits>
#include <type_traits>

#include "f32x2.cuh"
#include "half.cuh"
#include "internal.h"
#include "kv_cache.cuh"
#include "mma.cuh"
#include "pdl.cuh"
#include "ptx.cuh"
#include "waits.cuh"

namespace lm {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTok = 32;              // tokens of a warp's tile
constexpr int kRows = 16;             // query rows of a warp
constexpr uint32_t kGaveUp = 1 << 16;  // more than a unit's parts
constexpr int kMinChunk = 512;        // tokens below which a row is not split
constexpr int kBalance = 2048;        // ... where parts are for balance only (512: 43 us, 1024: 39, none: 36 for
                                      // 1024 units of up to 1500 tokens)
// Value scales count as at least 2^-90 (values of at most 1e-25, which are off
// by as much): a weight divided by its scale then still has 23 bits below the
// largest one in 32-bit floats, for scales of up to 2^13.
constexpr float kMinScale = 8.0779357e-28f;

// Bytes of a stage (keys and values of kTok tokens), ring depth, and the CTAs
// that an SM holds: shared memory (a ring per warp) and registers allow 4, 4
// and 3 of head_dim 32, 64 and 128.
constexpr int stage_bytes(int d) { return 2 * kTok * d; }
constexpr int ring_stages(int d, bool shared) { return shared ? 4 : d == 128 ? 2 : d == 64 ? 3 : 6; }
constexpr int resident_ctas(int d) { return d == 128 ? 3 : 4; }
constexpr int full_ctas(int d) { return 152 * resident_ctas(d); }

__device__ uint32_t g_attend_error;  // bits of every call on the device, whatever its workspace

struct AttendParams {
  KvView c;
  const void *q;
  void *out;
  int64_t row_s, tok_s, head_s;
  const int32_t *counts;
  uint32_t *err, *done;          // done: per unit, parts that are ready, and kGaveUp for each that gave up
  float2 *part_ml;               // [unit][split][rows]: maximum, sum
  float *part_acc;               // [unit][split][rows][head_dim]
  int32_t tokens, q_heads, new_tokens, causal, group, qrows, qtiles, splits, part_rows, min_chunk, qvec;
  float scale;
  uint64_t wait_ns;              // limit of a wait
  int64_t withheld;              // CTA whose first stage never fills (tests), or -1
};

// Shared memory: the rings (at the end the warps' partial results), then this.
struct Shared {
  uint64_t full[kWarps][8];
  float2 ml[kWarps][kRows];  // maximum and sum per warp and query row
  int abort;
  int last;    // of a unit's parts
  int failed;  // one of them gave up
};

constexpr int big_bytes(int d, bool shared) {
  // (Shared: and two tiles as f16.)
  const int ring = (shared ? 1 : kWarps) * ring_stages(d, shared) * stage_bytes(d) + (shared ? 4 * stage_bytes(d) : 0);
  const int joined = kWarps * (shared ? kRows * d * 4 : ring_stages(d, shared) * stage_bytes(d));
  return ring > joined ? ring : joined;
}

__device__ __forceinline__ uint4 lds_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts_u32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// N 32-bit words of shared memory.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = lds_u32(a);
  } else if constexpr (N == 2) {
    const uint2 v = lds_v2(a);
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = lds_v4(a + 16 * i);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  }
}

// Where row `row` of a tile of f16 (D elements a row) has its 16-byte piece
// `piece`: pieces are permuted so that eight rows' pieces of one column lie in
// different banks.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
  return static_cast<uint32_t>(row * D * 2 + ((piece ^ (D == 32 ? (row >> 1) & 3 : row & 7)) * 16));
}

// How the four warps share the work (see cut() for the choice):
//  - kTokens: 16 query rows of one head, every fourth tile of tokens each;
//  - kHeads, where there are many rows of few tokens: 16 query rows of a head of
//    its own each, no joins and a fourth of the CTAs;
//  - kQueries, for many query rows: 16 of 64 query rows each, all over the same
//    tokens in one ring.  Each warp turns a quarter of a tile into f16 in shared
//    memory, laid out so that ldmatrix gives all warps the operands that they would
//    make of the bytes themselves (250 instructions a tile and warp instead of 400).
// E = 1: at most eight query rows, so that the lower half of a product's rows is
// left out of the softmax (55 of 400 instructions a tile; 5 queries of 64 rows over
// up to 1500 tokens: 38.0 -> 36.2 us).
enum class Mode { kTokens, kHeads, kQueries };

template <typename T, int D, int E, Mode MODE>
__global__ void __launch_bounds__(kThreads, resident_ctas(D))
    attend_kernel(const AttendParams p) {
  constexpr bool SHARED = MODE == Mode::kQueries, ALONE = MODE == Mode::kHeads;
  constexpr int STAGES = ring_stages(D, SHARED);
  constexpr int JOIN = SHARED ? kRows * D * 4 : STAGES * stage_bytes(D);  // bytes between the warps' results
  constexpr int KW = D / 16;   // 32-bit words of a token's key per thread; also 16-element steps of k
  constexpr int VB = D / 8;    // bytes of a token's value per thread; also 8-column tiles of the output
  constexpr int QT = SHARED ? kWarps * kRows : kRows;  // query rows of the CTA
  extern __shared__ __align__(128) uint8_t smem[];
  Shared &sh = *reinterpret_cast<Shared *>(smem + big_bytes(D, SHARED));

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r8 = lane / 4, c4 = lane % 4;
  // Grid: (key heads and parts, row, tile of queries).  Later queries see more:
  // their tiles go first.
  const int split = p.splits > 1 ? static_cast<int>(blockIdx.x) / p.c.heads : 0;
  const int head = ALONE ? static_cast<int>(blockIdx.x) * kWarps + warp : static_cast<int>(blockIdx.x) - split * p.c.heads;
  const int h = ALONE ? min(head, p.c.heads - 1) : head;
  const int row = blockIdx.y;
  const int qt = p.qtiles - 1 - static_cast<int>(blockIdx.z);
  const int64_t unit = (static_cast<int64_t>(blockIdx.z) * p.c.rows + row) * p.c.heads + h;

  if (threadIdx.x < kWarps) {
    const int64_t cta = (static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
    for (int i = 0; i < STAGES; ++i) mbar_init(&sh.full[threadIdx.x][i], threadIdx.x + i == 0 && cta == p.withheld ? 2 : 1);
  }
  if (threadIdx.x == 0) sh.abort = 0;
  fence_mbar_init();
  pdl_launch();
  pdl_wait();

  // What no other load has to wait for goes out first: lengths, queries and,
  // for the first part of a row (the only one, mostly), its blocks.
  const int block_shift = 31 - __clz(p.c.block);
  const int32_t *const table = p.c.table + static_cast<int64_t>(row) * p.c.width;
  const int held_ = p.c.lens[row];
  const int fresh_ = p.counts ? p.counts[row] : p.new_tokens;
  int early[2] = {-1, -1};
  if (split == 0 && p.c.width > 0) {
    const int t = (MODE != Mode::kTokens ? lane : lane * kWarps + warp) * kTok;
#pragma unroll
    for (int e = 0; e < 2; ++e) early[e] = table[min((t + 16 * e) >> block_shift, p.c.width - 1)];
  }
  const int q_first = qt * QT, q_rows = min(QT, p.qrows - q_first);
  uint32_t raw[E][2 * KW];
  int q_i[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int at = q_first + (SHARED ? warp * kRows : 0) + 8 * e + r8;
    const bool in = at < p.qrows;
    const int i = !in ? 0 : p.group == 1 ? at : at / p.group, g = in ? at - i * p.group : 0;
    q_i[e] = in ? i : -1;
    const T *const src = static_cast<const T *>(p.q) + row * p.row_s + i * p.tok_s +
                         (static_cast<int64_t>(h) * p.group + g) * p.head_s + c4 * (D / 4);
    uint32_t *const w = raw[e];
    if (!in) {
#pragma unroll
      for (int j = 0; j < 2 * KW; ++j) w[j] = 0;
    } else if (p.qvec) {
#pragma unroll
      for (int j = 0; j < 2 * KW; j += 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(src + 2 * j);
        w[j] = v.x;
        w[j + 1] = v.y;
        w[j + 2] = v.z;
        w[j + 3] = v.w;
      }
    } else {
      const uint16_t *const s16 = reinterpret_cast<const uint16_t *>(src);
#pragma unroll
      for (int j = 0; j < 2 * KW; ++j)
        w[j] = s16[2 * j] | static_cast<uint32_t>(s16[2 * j + 1]) << 16;
    }
  }
  __syncthreads();

  // How far this tile of queries sees.
  const int cap = p.c.width * p.c.block;
  const int held = min(max(held_, 0), cap);
  int fresh = max(fresh_, 0);
  if (p.causal) fresh = min(fresh, p.tokens);
  const int total = static_cast<int>(min(static_cast<int64_t>(held) + fresh, static_cast<int64_t>(cap)));
  int end = total;
  if (p.causal) {
    const int i_first = q_first / p.group, i_last = min((q_first + q_rows - 1) / p.group, fresh - 1);
    end = i_first < fresh ? min(total, held + i_last + 1) : 0;
  }
  // Equal parts of whole CTA strides; a part that would be empty has no CTA.
  int chunk = end, parts = 1;
  if (p.splits > 1) {
    chunk = ((end + p.splits - 1) / p.splits + kWarps * kTok - 1) / (kWarps * kTok) * (kWarps * kTok);
    chunk = max(chunk, p.min_chunk);
    parts = max((end + chunk - 1) / chunk, 1);
  }
  if (split >= parts) return;
  const int begin = split * chunk, stop = min(end, begin + chunk);

  uint8_t *const ring = smem + (SHARED ? 0 : warp * STAGES * stage_bytes(D));
  const uint32_t ring_a = smem_u32(ring);
  uint64_t *const full = sh.full[SHARED ? 0 : warp];
  const int64_t tiles0 = p.c.layer_tiles + h;
  // This warp's tiles: number j starts at token begin + j * kTok, or of kTokens
  // begin + (j * kWarps + warp) * kTok.
  const int mine = MODE != Mode::kTokens ? (head < p.c.heads ? (stop - begin + kTok - 1) / kTok : 0)
                                         : max((stop - begin - warp * kTok + kWarps * kTok - 1) / (kWarps * kTok), 0);
  auto token_of = [&](int j) { return begin + (MODE != Mode::kTokens ? j : j * kWarps + warp) * kTok; };
  // The block of a tile's half (16 tokens), or -1.
  auto block_of = [&](int j, int half) {
    const int t = token_of(j) + 16 * half;
    if (j >= mine || t >= stop) return -1;
    const int b = j < 32 && split == 0 ? early[half] : table[t >> block_shift];
    return b >= 0 && b < p.c.blocks ? b : -1;
  };
  int fb0 = -1, fb1 = -1;  // blocks of the 32 tiles that are fetched next, one per lane
  auto fetch = [&](int j) {
    if (j % 32 == 0) {
      fb0 = block_of(j + lane, 0);
      fb1 = block_of(j + lane, 1);
    }
    const int b0 = __shfl_sync(0xffffffffu, fb0, j % 32), b1 = __shfl_sync(0xffffffffu, fb1, j % 32);
    if (lane == 0 && j < mine) {
      const int s = j % STAGES;
      const uint32_t bytes = 16 * D;
      mbar_arrive_expect_tx(&full[s], ((b0 >= 0) + (b1 >= 0)) * 2 * bytes);
      uint8_t *const k_at = ring + s * stage_bytes(D), *const v_at = k_at + kTok * D;
      const int t = token_of(j), in = t & (p.c.block - 1);
      const int64_t at0 = ((tiles0 + static_cast<int64_t>(b0) * p.c.heads) * p.c.block + in) * D;
      // (A row may name one block of 16 tokens in two columns: then the halves are equal, not
      // consecutive.)
      if (b0 >= 0 && b0 == b1 && p.c.block >= kTok) {
        bulk_g2s_plain(k_at, p.c.k8 + at0, 2 * bytes, &full[s]);
        bulk_g2s_plain(v_at, p.c.v8 + at0, 2 * bytes, &full[s]);
      } else {
        if (b0 >= 0) {
          bulk_g2s_plain(k_at, p.c.k8 + at0, bytes, &full[s]);
          bulk_g2s_plain(v_at, p.c.v8 + at0, bytes, &full[s]);
        }
        if (b1 >= 0) {
          const int64_t at1 =
              ((tiles0 + static_cast<int64_t>(b1) * p.c.heads) * p.c.block + ((in + 16) & (p.c.block - 1))) * D;
          bulk_g2s_plain(k_at + bytes, p.c.k8 + at1, bytes, &full[s]);
          bulk_g2s_plain(v_at + bytes, p.c.v8 + at1, bytes, &full[s]);
        }
      }
    }
  };
  const bool fetches = !SHARED || warp == 0;
  int fetched = 0;
  if (fetches)
    for (; fetched < min(mine, STAGES); ++fetched) fetch(fetched);

  // Queries, k permuted: step s of the product over k takes elements
  // c4 * D/4 + 4s .. + 3 of the head from this thread.  bf16 queries become f16
  // times a power of two that puts the row's largest between 2^14 and 2^15:
  // exact but for values below 2^-28 of that one, which are off by 2^-39 of
  // it.  (Bytes turn into f16 in two instructions, into bf16 in three.)
  uint32_t q[KW][4];
  int limit[E];
  // Key bytes go in as they are, whole numbers in f16.  (As k + 128, in subnormal f16, they take
  // three instructions a word instead of five -- two rows of 131000 tokens 94.2 us, so 96.9 -- but
  // 128 sum q has to be taken off again, and a score is then off by the rounding of the largest one
  // that the block's scale allows: too much where one element of the head is an outlier.)
  float back[E];  // the power's inverse, times scale and log2 e
  const float log2e = 1.4426950408889634f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = q_i[e];
    limit[e] = i < 0 ? INT_MAX : !p.causal ? total : i < fresh ? min(total, held + i + 1) : 0;
    uint32_t *const w = raw[e];
    back[e] = p.scale * log2e;
    if constexpr (sizeof(T) == 2 && !std::is_same<T, __half>::value) {
      uint32_t top = 0;  // |q| as integers
#pragma unroll
      for (int j = 0; j < 2 * KW; ++j) top = max(top, max(w[j] << 16 & 0x7fffffffu, w[j] & 0x7fff0000u));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      uint32_t ex = max(top >> 23, 15u);
      if (ex == 255) ex = 141;  // infinity or NaN: as it is
      const float up = __uint_as_float((268 - ex) << 23);
      back[e] *= __uint_as_float((ex - 14) << 23);
#pragma unroll
      for (int j = 0; j < 2 * KW; ++j) {
        const float2 f = unpack2<T>(w[j]);
        w[j] = pack2<__half>(f.x * up, f.y * up);
      }
    }
#pragma unroll
    for (int s = 0; s < KW; ++s) {
      q[s][e] = w[2 * s];
      q[s][2 + e] = w[2 * s + 1];
      if (E == 1) q[s][1] = q[s][3] = 0;
    }
  }

  float acc[VB][4];
  float top[E], sum[E];
#pragma unroll
  for (int j = 0; j < VB; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    top[e] = -INFINITY;
    sum[e] = 0.0f;
  }

  // Byte n of two words, in the low bytes of the halves.
  constexpr uint32_t kPick[4] = {0x0400, 0x0501, 0x0602, 0x0703};
  const uint32_t tiles_a = ring_a + STAGES * stage_bytes(D);  // SHARED: two tiles of f16 keys and values
  // Of the 32 tiles that are consumed next, one per lane and half: the key
  // scale, log2 and inverse of the value scale; absent blocks are masked.
  float f_s[2] = {0, 0}, l_s[2] = {0, 0}, i_s[2] = {0, 0};
  // SHARED: this warp's quarter of tile j as f16.
  auto convert = [&](int j) {
    if (j >= mine) return true;
    const int s = j % STAGES;
    if (!mbar_wait_warp(&full[s], (j / STAGES) & 1, p.wait_ns, &sh.abort, p.err)) return false;
    const uint32_t k_at = ring_a + s * stage_bytes(D), v_at = k_at + kTok * D;
    const uint32_t k16 = tiles_a + (j & 1) * 2 * stage_bytes(D), v16 = k16 + kTok * D * 2;
    // Token r8 of this warp's eight: place 2 (r8 % 4) + r8 / 4 among them.
    const int to = 8 * warp + 2 * (r8 & 3) + (r8 >> 2);
    uint32_t w[KW];
    lds_words(k_at + (8 * warp + r8) * D + c4 * (D / 4), w);
#pragma unroll
    for (int ks = 0; ks < KW; ++ks) {
      uint32_t b0, b1;
      word_to_f16(w[ks], b0, b1);
      sts_u32(k16 + piece_at<D>(to, 2 * ks) + 4 * c4, b0);
      sts_u32(k16 + piece_at<D>(to, 2 * ks + 1) + 4 * c4, b1);
    }
    lds_words(v_at + (8 * warp + r8) * D + c4 * (D / 4), w);
#pragma unroll
    for (int n = 0; n < VB; ++n)
      sts_u32(v16 + piece_at<D>(to, n) + 4 * c4,
              bytes_to_f16(__byte_perm(w[n / 4], w[VB / 4 + n / 4], kPick[n % 4])));
    return true;
  };
  bool ok = true;
  if constexpr (SHARED) ok = convert(0);
  int done = 0;
  for (; done < mine; ++done) {
    const int j = done;
    if (j % 32 == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int b = block_of(j + lane, e);
        f_s[e] = l_s[e] = i_s[e] = 0.0f;
        if (b >= 0) {
          const int64_t tile = tiles0 + static_cast<int64_t>(b) * p.c.heads;
          const float vs = fmaxf(p.c.v_scale[tile], kMinScale);
          f_s[e] = p.c.k_scale[tile];
          l_s[e] = __log2f(vs);
          i_s[e] = ex2(-l_s[e]);  // of the logarithm that the weight has: they cancel
        } else {
          i_s[e] = -1.0f;
        }
      }
    }
    const int t0 = token_of(j);
    const int s = j % STAGES;
    const uint32_t k_at = ring_a + s * stage_bytes(D), v_at = k_at + kTok * D;
    const uint32_t k16 = tiles_a + (j & 1) * 2 * stage_bytes(D), v16 = k16 + kTok * D * 2;
    if constexpr (SHARED) {
      // The tile is whole, and its bytes are no longer needed.
      if (__syncthreads_or(!ok)) break;
      if (fetches && fetched < mine) fetch(fetched++);
    } else {
      ok = mbar_wait_warp(&full[s], (j / STAGES) & 1, p.wait_ns, &sh.abort, p.err);
      if (!ok) break;
    }

    // Scores: column n of 8-token tile n8 is token 16 (n8/2) + 8 (n8%2) + n/2 + 4 (n%2).
    float sc[4][4];
#pragma unroll
    for (int n8 = 0; n8 < 4; ++n8) {
      sc[n8][0] = sc[n8][1] = sc[n8][2] = sc[n8][3] = 0.0f;
      if constexpr (SHARED) {
#pragma unroll
        for (int k2 = 0; k2 < KW / 2; ++k2) {
          uint32_t b[4];
          ldmatrix4<false>(b, k16 + piece_at<D>(8 * n8 + lane % 8, 4 * k2 + lane / 8));
          mma16816(sc[n8], q[2 * k2], b[0], b[1]);
          mma16816(sc[n8], q[2 * k2 + 1], b[2], b[3]);
        }
      } else {
        const int tok = 16 * (n8 / 2) + 8 * (n8 & 1) + (r8 >> 1) + 4 * (r8 & 1);
        uint32_t w[KW];
        lds_words(k_at + tok * D + c4 * (D / 4), w);
#pragma unroll
        for (int ks = 0; ks < KW; ++ks) {
          uint32_t b0, b1;
          word_to_f16(w[ks], b0, b1);
          mma16816(sc[n8], q[ks], b0, b1);
        }
      }
    }
    const float f0 = __shfl_sync(0xffffffffu, f_s[0], j % 32), f1 = __shfl_sync(0xffffffffu, f_s[1], j % 32);
    const float l0 = __shfl_sync(0xffffffffu, l_s[0], j % 32), l1 = __shfl_sync(0xffffffffu, l_s[1], j % 32);
    const float i0 = __shfl_sync(0xffffffffu, i_s[0], j % 32), i1 = __shfl_sync(0xffffffffu, i_s[1], j % 32);
    const bool partial = i0 < 0.0f || i1 < 0.0f;
    bool cut = partial;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float g0 = f0 * back[e], g1 = f1 * back[e];
#pragma unroll
      for (int n8 = 0; n8 < 4; ++n8) {
#pragma unroll
        for (int x = 2 * e; x < 2 * e + 2; ++x)
          sc[n8][x] = fmaf(sc[n8][x], n8 < 2 ? g0 : g1, n8 < 2 ? l0 : l1);
      }
      cut = cut || t0 > limit[e] - kTok;
    }
    // Tokens past a row's end, and absent ones.  (Selected, not added: their
    // bytes and scales may be anything.)
    if (__any_sync(0xffffffffu, cut)) {
#pragma unroll
      for (int n8 = 0; n8 < 4; ++n8) {
        const bool absent = (n8 < 2 ? i0 : i1) < 0.0f;
#pragma unroll
        for (int x = 0; x < 2 * E; ++x) {
          const int tok = t0 + 16 * (n8 / 2) + 8 * (n8 & 1) + c4 + 4 * (x & 1);
          if (absent || tok >= limit[x >> 1]) sc[n8][x] = -INFINITY;
        }
      }
    }
    float next[E];
    bool rise = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float t = top[e];
#pragma unroll
      for (int n8 = 0; n8 < 4; ++n8) t = fmaxf(t, fmaxf(sc[n8][2 * e], sc[n8][2 * e + 1]));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
      next[e] = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
      rise = rise || next[e] > top[e];
    }
    // Maxima rise ever more rarely along a row.
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float shrink = ex2(top[e] - (next[e] == -INFINITY ? 0.0f : next[e]));
        top[e] = next[e];
        sum[e] *= shrink;
#pragma unroll
        for (int n = 0; n < VB; ++n) {
          acc[n][2 * e] *= shrink;
          acc[n][2 * e + 1] *= shrink;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float zero = top[e] == -INFINITY ? 0.0f : top[e];
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
      for (int n8 = 0; n8 < 4; ++n8) {
#pragma unroll
        for (int x = 2 * e; x < 2 * e + 2; ++x) {
          const float w = ex2(sc[n8][x] - zero);
          sc[n8][x] = w;
          if (n8 < 2) {
            s0 += w;
          } else {
            s1 += w;
          }
        }
      }
      sum[e] = fmaf(s0, fabsf(i0), fmaf(s1, fabsf(i1), sum[e]));
    }
    // The next tile, in the shadow of this one's weights and products (223 queries over
    // 1500 tokens 2.5% faster; before the weights 1% slower).
    if constexpr (SHARED) ok = convert(j + 1);
    // Values: this thread's bytes VB r8 .. + VB-1 of every fourth token.
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t a[4];
      a[0] = pack2<__half>(sc[2 * half][0], sc[2 * half][1]);
      a[1] = E == 1 ? 0u : pack2<__half>(sc[2 * half][2], sc[2 * half][3]);
      a[2] = pack2<__half>(sc[2 * half + 1][0], sc[2 * half + 1][1]);
      a[3] = E == 1 ? 0u : pack2<__half>(sc[2 * half + 1][2], sc[2 * half + 1][3]);
      if constexpr (SHARED) {
#pragma unroll
        for (int n = 0; n < VB; n += 2) {
          uint32_t b[4];
          ldmatrix4<true>(b, v16 + piece_at<D>(16 * half + lane % 16, n + lane / 16));
          mma16816(acc[n], a, b[0], b[1]);
          mma16816(acc[n + 1], a, b[2], b[3]);
        }
      } else {
        uint32_t w[4][VB / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) lds_words(v_at + (16 * half + 4 * i + c4) * D + VB * r8, w[i]);
#pragma unroll
        for (int n = 0; n < VB; ++n) {
          // Byte n of tokens c4, c4 + 4 and of c4 + 8, c4 + 12.
          const uint32_t b0 = bytes_to_f16(__byte_perm(w[0][n / 4], w[1][n / 4], kPick[n % 4]));
          const uint32_t b1 = bytes_to_f16(__byte_perm(w[2][n / 4], w[3][n / 4], kPick[n % 4]));
          mma16816(acc[n], a, b0, b1);
        }
      }
    }
    __syncwarp();
    if (!SHARED && fetched < mine) fetch(fetched++);
  }
  if (fetches && done < mine && lane == 0) {  // gave up: the copies in flight still have to land
    for (int f = done; f < fetched; ++f)
      if (!mbar_drain(&full[f % STAGES], (f / STAGES) & 1, p.wait_ns, p.err)) break;
  }
  __syncwarp();
  if (SHARED) __syncthreads();  // the ring and the tiles are free
  // Every warp's sums, in its own ring's memory.
  float *const acc_s = reinterpret_cast<float *>(smem + warp * JOIN);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int rr = 8 * e + r8;
    float s = sum[e];
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if (c4 == 0) sh.ml[warp][rr] = make_float2(top[e], s);
    if ((SHARED ? warp * kRows : 0) + rr < q_rows) {
      float4 *const o = reinterpret_cast<float4 *>(acc_s + rr * D + c4 * (D / 4));
#pragma unroll
      for (int n = 0; n < VB; n += 4) {
        o[n / 4] = make_float4(acc[n][2 * e], acc[n + 1][2 * e], acc[n + 2][2 * e], acc[n + 3][2 * e]);
        o[(VB + n) / 4] = make_float4(acc[n][2 * e + 1], acc[n + 1][2 * e + 1], acc[n + 2][2 * e + 1],
                                      acc[n + 3][2 * e + 1]);
      }
    }
  }
  constexpr int PER = D / 4;  // 4-element vectors of a row
  auto emit = [&](int rr, int d, float4 v, float l) {
    const int at = q_first + rr, i = p.group == 1 ? at : at / p.group, g = at - i * p.group;
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    T *const o = static_cast<T *>(p.out) +
                 ((static_cast<int64_t>(row) * p.tokens + i) * p.q_heads + h * p.group + g) * D + d;
    *reinterpret_cast<uint2 *>(o) = make_uint2(pack2<T>(v.x * f, v.y * f), pack2<T>(v.z * f, v.w * f));
  };
  if constexpr (ALONE) {
    __syncwarp();
    if (done < mine && lane == 0) atomicOr(&g_attend_error, kErrMbarTimeout);
    if (head >= p.c.heads || done < mine) return;
    for (int x = lane; x < q_rows * PER; x += 32) {
      const int rr = x / PER, d = x % PER * 4;
      emit(rr, d, *reinterpret_cast<const float4 *>(acc_s + rr * D + d), sh.ml[warp][rr].y);
    }
    return;
  }
  __syncthreads();
  const bool gave_up = sh.abort;
  if (gave_up && threadIdx.x == 0) atomicOr(&g_attend_error, kErrMbarTimeout);
  const int64_t part0 = (unit * p.splits + split) * p.part_rows;
  const float2 *const ml_s = &sh.ml[0][0];  // SHARED: row rr is in place rr; else in warp w's place rr
  constexpr int FROM = SHARED ? 1 : kWarps;
  for (int x = threadIdx.x; x < (gave_up ? 0 : q_rows * PER); x += kThreads) {
    const int rr = x / PER, d = x % PER * 4;
    float t = ml_s[rr].x;
#pragma unroll
    for (int w = 1; w < FROM; ++w) t = fmaxf(t, ml_s[w * kRows + rr].x);
    const float zero = t == -INFINITY ? 0.0f : t;
    float4 v = make_float4(0, 0, 0, 0);
    float l = 0.0f;
#pragma unroll
    for (int w = 0; w < FROM; ++w) {
      const float2 ml = ml_s[w * kRows + rr];
      const float f = ex2(ml.x - zero);
      const float4 a = *reinterpret_cast<const float4 *>(smem + w * JOIN + (rr * D + d) * 4);
      v.x = fmaf(a.x, f, v.x);
      v.y = fmaf(a.y, f, v.y);
      v.z = fmaf(a.z, f, v.z);
      v.w = fmaf(a.w, f, v.w);
      l = fmaf(ml.y, f, l);
    }
    if (parts == 1) {
      emit(rr, d, v, l);
    } else {
      *reinterpret_cast<float4 *>(p.part_acc + (part0 + rr) * D + d) = v;
      if (d == 0) p.part_ml[part0 + rr] = make_float2(t, l);
    }
  }
  if (parts == 1) return;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    // A part that gave up counts as well, so that the counter goes back to zero; the unit is
    // then not joined.
    const uint32_t before = atomicAdd(&p.done[unit], gave_up ? 1 + kGaveUp : 1u);
    sh.last = before % kGaveUp == static_cast<uint32_t>(parts - 1);
    sh.failed = gave_up || before >= kGaveUp;
  }
  __syncthreads();
  if (!sh.last) return;
  __threadfence();
  if (threadIdx.x == 0) p.done[unit] = 0;
  if (sh.failed) return;
  // Eight threads a row find each part's factor and the sum of weights ...
  const int64_t unit0 = unit * p.splits * p.part_rows;
  float *const factor = reinterpret_cast<float *>(smem);  // [row][part]; cut() sees that it fits
  for (int r0 = 0; r0 < q_rows; r0 += kThreads / 8) {
    const int rr = r0 + static_cast<int>(threadIdx.x) / 8, l8 = threadIdx.x % 8;
    const bool in = rr < q_rows;
    const float2 *const ml = p.part_ml + unit0 + (in ? rr : 0);
    const float2 none = make_float2(-INFINITY, 0.0f);
    const float2 first = in && l8 < parts ? __ldcg(&ml[l8 * p.part_rows]) : none;
    float t = first.x;
#pragma unroll 4
    for (int w = l8 + 8; w < parts; w += 8) t = fmaxf(t, __ldcg(&ml[w * p.part_rows]).x);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
    const float zero = t == -INFINITY ? 0.0f : t;
    float l = 0.0f;
#pragma unroll 4
    for (int w = l8; w < parts; w += 8) {
      const float2 m = w < 8 ? first : __ldcg(&ml[w * p.part_rows]);
      const float f = ex2(m.x - zero);
      if (in) factor[rr * parts + w] = f;
      l = fmaf(m.y, f, l);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (in && l8 == 0) sh.ml[rr / kRows][rr % kRows].y = l;
  }
  __syncthreads();
  // ... and groups of threads add up every `groups`-th part.
  const int items = q_rows * PER, groups = max(kThreads / items, 1);
  float4 *const group_sums = reinterpret_cast<float4 *>(smem + big_bytes(D, SHARED) - kThreads * 16);
  for (int x0 = 0; x0 < items; x0 += kThreads) {
    const int g = groups == 1 ? 0 : threadIdx.x / items;
    const int x = x0 + (groups == 1 ? threadIdx.x : threadIdx.x - g * items);
    const bool in = x < items && g < groups;
    const int rr = x / PER, d = x % PER * 4;
    float4 v = make_float4(0, 0, 0, 0);
    if (in) {
      const float *const acc_p = p.part_acc + (unit0 + rr) * D + d;
#pragma unroll 8
      for (int w = g; w < parts; w += groups) {
        const float f = factor[rr * parts + w];
        const float4 a = __ldcg(reinterpret_cast<const float4 *>(acc_p + static_cast<int64_t>(w) * p.part_rows * D));
        v.x = fmaf(a.x, f, v.x);
        v.y = fmaf(a.y, f, v.y);
        v.z = fmaf(a.z, f, v.z);
        v.w = fmaf(a.w, f, v.w);
      }
    }
    if (groups > 1) {
      group_sums[threadIdx.x] = v;
      __syncthreads();
      if (in && g == 0) {
        for (int i = 1; i < groups; ++i) {
          const float4 a = group_sums[threadIdx.x + i * items];
          v.x += a.x;
          v.y += a.y;
          v.z += a.z;
          v.w += a.w;
        }
      }
    }
    if (in && g == 0) emit(rr, d, v, sh.ml[rr / kRows][rr % kRows].y);
  }
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

lm_status check(const lm_kv_cache *cache, int32_t tokens, int32_t q_heads) {
  if (lm_status st = kv_check(cache); st != LM_OK) return st;
  if (tokens < 0 || q_heads < 1 || q_heads % cache->heads != 0) return LM_ERR_INVALID_ARG;
  if (static_cast<int64_t>(tokens) * (q_heads / cache->heads) > INT_MAX - 64) return LM_ERR_UNSUPPORTED;
  return LM_OK;
}

// How a call is cut: the warps' mode, query rows per tile, tiles, units (row, key
// head, tile) and parts of the tokens.
struct Cut {
  Mode mode;
  int qrows, qtiles, splits, part_rows, chunk;
  int64_t units;
  size_t done_bytes, ml_bytes, acc_bytes;
};

// The mode with the least estimated time: rounds of CTAs, times 5 for a CTA's start
// and end and 1 for each tile of tokens that a warp goes over (a unit is about a
// microsecond).  Rows are mostly of unequal length, which the modes with long walks
// cannot even out: a tenth in favour of kTokens, and a fourth on the walks where all
// CTAs run at once.  Measured, in us, kTokens / kQueries / kHeads, heads of 64: rows of unequal
// length, 320 x 16 heads, one query over up to 448 tokens 57 / - / 47, over 128 31 / - / 18; 64 x 16,
// 20 over up to 1500, not causal 62 / 100 / 81; rows of one length, causal, 157 x 10, 30 over 30
// 24 / 15 / 12; 64 x 16, 96 over 448 95 / 85 / 73; 8 x 8, 64 over 448 11 / 16 / 15, 448 over 448
// 22 / 25 / 27 (here the estimate takes kQueries); not causal, 64 x 16, 448 over 1052 804 / 600 / 693.
Cut cut(const lm_kv_cache *c, int32_t tokens, int32_t q_heads) {
  Cut k = {};
  const int qrows = tokens * (q_heads / c->heads);
  const int64_t cap = static_cast<int64_t>(c->width) * c->block, tiles = (cap + kTok - 1) / kTok;
  const int64_t slots = full_ctas(c->head_dim);
  double least = 0.0;
  for (const Mode mode : {Mode::kTokens, Mode::kQueries, Mode::kHeads}) {
    Cut m = {};
    m.mode = mode;
    m.qrows = qrows;
    const int tile = mode == Mode::kQueries ? kWarps * kRows : kRows;
    if (mode == Mode::kQueries && qrows <= kRows) continue;
    m.qtiles = static_cast<int>((static_cast<int64_t>(qrows) + tile - 1) / tile);
    m.part_rows = qrows < tile ? qrows : tile;
    m.units = static_cast<int64_t>(c->rows) * c->heads * m.qtiles;
    // As many parts as fill the device once.  Where the units alone come near
    // that, parts are for balance between rows of unequal length: four rounds of
    // them.  None below kMinChunk or kBalance tokens, nor more than the join's
    // factors have room for.
    // (kTokens only: the others have units enough.)
    int64_t s = m.units == 0 || mode != Mode::kTokens ? 1
                : 2 * m.units > slots                 ? (4 * slots + m.units - 1) / m.units
                                                      : slots / m.units;
    m.chunk = 2 * m.units > slots ? kBalance : kMinChunk;
    const int64_t most = (cap + m.chunk - 1) / m.chunk;
    const int64_t room = (big_bytes(c->head_dim, false) - kThreads * 16) / (4 * kRows);
    s = s < most ? s : most;
    s = s < room ? s : room;
    m.splits = static_cast<int>(s < 1 ? 1 : s);
    const int64_t ctas = mode == Mode::kHeads ? static_cast<int64_t>(c->rows) * ((c->heads + kWarps - 1) / kWarps) * m.qtiles
                                              : m.units * m.splits;
    const double walked = static_cast<double>(tiles) / m.splits / (mode == Mode::kTokens ? kWarps : 1);
    const int64_t rounds = (ctas + slots - 1) / slots;
    const double tile_time = mode != Mode::kTokens && rounds <= 1 ? 1.25 : 1.0;
    const double time = (mode == Mode::kTokens ? 0.9 : 1.0) * static_cast<double>(rounds) * (5.0 + tile_time * walked);
    if (mode == Mode::kTokens || time < least) {
      least = time;
      k = m;
    }
  }
  const int64_t parts = k.splits > 1 ? k.units * k.splits * k.part_rows : 0;
  // One place for the counters whatever the shape: calls of other shapes
  // that share the workspace must not write over them.  Units that are split
  // are fewer than 4 * full_ctas().
  k.done_bytes = (4 * full_ctas(32) * 4 + 255) / 256 * 256;
  k.ml_bytes = (static_cast<size_t>(parts) * 8 + 255) / 256 * 256;
  k.acc_bytes = static_cast<size_t>(parts) * c->head_dim * 4;
  return k;
}

template <typename T, int D, int E, Mode MODE>
lm_status launch(const AttendParams &p, dim3 grid, cudaStream_t s) {
  auto *const kernel = attend_kernel<T, D, E, MODE>;
  constexpr int smem = big_bytes(D, MODE == Mode::kQueries) + static_cast<int>(sizeof(Shared));
  if (lm_status st = ensure_smem_attribute(reinterpret_cast<const void *>(kernel), smem); st != LM_OK) return st;
  return launch_dependent(kernel, grid, kThreads, smem, s, 1, p);
}

template <typename T, int D>
lm_status launch_form(const AttendParams &p, const Cut &k, dim3 grid, cudaStream_t s) {
  if (k.mode == Mode::kQueries) return launch<T, D, 2, Mode::kQueries>(p, grid, s);
  if (k.mode == Mode::kHeads)
    return k.qrows <= 8 ? launch<T, D, 1, Mode::kHeads>(p, grid, s) : launch<T, D, 2, Mode::kHeads>(p, grid, s);
  return k.qrows <= 8 ? launch<T, D, 1, Mode::kTokens>(p, grid, s) : launch<T, D, 2, Mode::kTokens>(p, grid, s);
}

template <typename T>
lm_status launch_dim(const AttendParams &p, const Cut &k, dim3 grid, cudaStream_t s) {
  switch (p.c.head_dim) {
    case 32: return launch_form<T, 32>(p, k, grid, s);
    case 64: return launch_form<T, 64>(p, k, grid, s);
    default: return launch_form<T, 128>(p, k, grid, s);
  }
}

// lm_kv_attend; `fault` is null outside tests.
lm_status attend(const lm_kv_cache *cache, int32_t layer, const void *q, const int64_t *q_strides, int32_t tokens,
                 int32_t q_heads, const int32_t *counts, int32_t new_tokens, int32_t causal, float scale, int32_t dtype,
                 void *out, void *workspace, size_t workspace_bytes, cudaStream_t s, const WaitFault *fault) {
  if (lm_status st = check(cache, tokens, q_heads); st != LM_OK) return st;
  if (layer < 0 || layer >= cache->layers || !q_strides || new_tokens < 0) return LM_ERR_INVALID_ARG;
  if (dtype != LM_F16 && dtype != LM_BF16) return LM_ERR_UNSUPPORTED;
  if (cache->rows == 0 || tokens == 0) return LM_OK;
  if (!q || !out) return LM_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (q_strides[i] < 0) return LM_ERR_INVALID_ARG;
  if (!aligned(q, 2) || !aligned(out, 16) || !aligned(workspace, 16)) return LM_ERR_MISALIGNED;
  const Cut k = cut(cache, tokens, q_heads);
  if (!workspace || workspace_bytes < 256 + k.done_bytes + k.ml_bytes + k.acc_bytes) return LM_ERR_WORKSPACE;
  // A part of a row may still read queries when another writes its output.
  const int64_t head_bytes = 2 * cache->head_dim;
  const int64_t row_bytes = 2 * ((tokens - 1) * q_strides[1] + (q_heads - 1) * q_strides[2]) + head_bytes;
  if (rows_meet({q, cache->rows, 2 * q_strides[0], row_bytes},
                {out, 1, 0, static_cast<int64_t>(cache->rows) * tokens * q_heads * head_bytes}))
    return LM_ERR_INVALID_ARG;
  if (cache->rows > 65535 || k.qtiles > 65535 || static_cast<int64_t>(cache->heads) * k.splits > INT_MAX)
    return LM_ERR_UNSUPPORTED;
  const unsigned across = k.mode == Mode::kHeads ? (cache->heads + kWarps - 1) / kWarps
                                                 : static_cast<unsigned>(cache->heads) * k.splits;
  const dim3 grid(across, cache->rows, k.qtiles);
  char *const w = static_cast<char *>(workspace);
  AttendParams p;
  p.c = kv_view(cache, layer);
  p.q = q;
  p.out = out;
  p.row_s = q_strides[0];
  p.tok_s = q_strides[1];
  p.head_s = q_strides[2];
  p.counts = counts;
  p.err = reinterpret_cast<uint32_t *>(w);
  p.done = reinterpret_cast<uint32_t *>(w + 256);
  p.part_ml = reinterpret_cast<float2 *>(w + 256 + k.done_bytes);
  p.part_acc = reinterpret_cast<float *>(w + 256 + k.done_bytes + k.ml_bytes);
  p.tokens = tokens;
  p.q_heads = q_heads;
  p.new_tokens = new_tokens;
  p.causal = causal != 0;
  p.group = q_heads / cache->heads;
  p.qrows = k.qrows;
  p.qtiles = k.qtiles;
  p.splits = k.splits;
  p.part_rows = k.part_rows;
  p.min_chunk = k.chunk;
  p.qvec = aligned(q, 16) && q_strides[0] % 8 == 0 && q_strides[1] % 8 == 0 && q_strides[2] % 8 == 0;
  p.scale = scale;
  p.wait_ns = fault ? fault->wait_ns : kWaitTimeoutNs;
  p.withheld = fault ? fault->withheld_cta : -1;
  return dtype == LM_F16 ? launch_dim<__half>(p, k, grid, s) : launch_dim<__nv_bfloat16>(p, k, grid, s);
}

}  // namespace

lm_status attend_error(uint32_t *value, bool clear, cudaStream_t s) { return read_sticky(g_attend_error, value, clear, s); }

}  // namespace lm

extern "C" lm_status lm_kv_attend_workspace_size(const lm_kv_cache *cache, int32_t tokens, int32_t q_heads,
                                                 size_t *bytes) {
  if (!bytes) return LM_ERR_INVALID_ARG;
  if (lm_status st = lm::check(cache, tokens, q_heads); st != LM_OK) return st;
  const lm::Cut k = lm::cut(cache, tokens, q_heads);
  *bytes = 256 + k.done_bytes + k.ml_bytes + k.acc_bytes;
  return LM_OK;
}

extern "C" lm_status lm_kv_attend(const lm_kv_cache *cache, int32_t layer, const void *q, const int64_t *q_strides,
                                  int32_t tokens, int32_t q_heads, const int32_t *counts, int32_t new_tokens,
                                  int32_t causal, float scale, int32_t dtype, void *out, void *workspace,
                                  size_t workspace_bytes, lm_stream_t stream) {
  return lm::attend(cache, layer, q, q_strides, tokens, q_heads, counts, new_tokens, causal, scale, dtype, out,
                    workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream), nullptr);
}

extern "C" lm_status lm_debug_kv_attend_withhold(const lm_kv_cache *cache, int32_t layer, const void *q,
                                                 const int64_t *q_strides, int32_t tokens, int32_t q_heads,
                                                 const int32_t *counts, int32_t new_tokens, int32_t causal, float scale,
                                                 int32_t dtype, void *out, void *workspace, size_t workspace_bytes,
                                                 int64_t withheld_cta, uint64_t wait_ns, lm_stream_t stream) {
  if (withheld_cta < 0 || wait_ns < 100000ull || wait_ns > lm::kWaitTimeoutNs) return LM_ERR_INVALID_ARG;
  const lm::WaitFault fault{withheld_cta, wait_ns};
  return lm::attend(cache, layer, q, q_strides, tokens, q_heads, counts, new_tokens, causal, scale, dtype, out,
                    workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream), &fault);
}
