// kv_cache.cu -- the 8-bit key/value cache: quantising tokens into blocks,
// reading them back, and letting the block tables follow a beam step.
//
// A block of `block` tokens of one head is one contiguous tile of
// block * head_dim bytes with one scale.  One "unit" below is such a tile of
// keys or of values: block * head_dim / 64 threads work on it, 64 elements
// (eight 8-element vectors) each, so that a unit's new tokens stay in
// registers between the maximum and the rounding and are read once.
#include <climits>

#include "half.cuh"
#include "internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace lm {

namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;  // 8-element vectors per thread

struct AppendParams {
  KvView c;
  const void *src[2];            // k, v
  int64_t row_s[2], tok_s[2], head_s[2];
  void *values[2];
  const int32_t *counts;
  int32_t tokens, spans;         // spans: blocks per row that a step can touch
  int64_t units;                 // rows * spans * heads
  bool vec;                      // 16-byte loads of src are aligned
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, bool vec, float (&x)[8]) {
  if (vec) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<T>(u[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(p[i]);
  }
}

__device__ __forceinline__ int byte_of(uint2 w, int i) {
  const uint32_t u = i < 4 ? w.x : w.y;
  return static_cast<int>(u << (24 - 8 * (i & 3))) >> 24;
}

// One unit: row r's span s of head h.  D and BS are the head dimension and
// the tokens of a block; NT threads work on the unit.
template <typename T, int D, int BS>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
  constexpr int NT = BS * D / 64;
  constexpr int PER = kThreads / NT;  // units per CTA
  __shared__ float part[kThreads / 32];
  const int tid = threadIdx.x % NT;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * PER + threadIdx.x / NT;
  const int which = blockIdx.y;
  const bool in = unit < p.units;
  const int64_t uu = in ? unit : 0;
  const int h = static_cast<int>(uu % p.c.heads);
  const int span = static_cast<int>(uu / p.c.heads % p.spans);
  const int r = static_cast<int>(uu / p.c.heads / p.spans);

  const int held = min(max(p.c.lens[r], 0), p.c.width * BS);
  const int fresh = p.counts ? min(max(p.counts[r], 0), p.tokens) : p.tokens;
  const int col = held / BS + span;
  const int base = col * BS;  // first token of the block
  // Row r's tokens end here; what lies past the table is dropped.
  const int end = static_cast<int>(min(static_cast<int64_t>(held) + fresh, static_cast<int64_t>(p.c.width) * BS));
  const int blk = in && col < p.c.width ? p.c.table[static_cast<int64_t>(r) * p.c.width + col] : -1;
  const bool ok = blk >= 0 && blk < p.c.blocks && base < end;
  const int64_t tile = ok ? (static_cast<int64_t>(blk) * p.c.heads + h) : 0;
  int8_t *const q8 = (which ? p.c.v8 : p.c.k8) + p.c.layer_tiles * BS * D + tile * BS * D;
  float *const qs = (which ? p.c.v_scale : p.c.k_scale) + p.c.layer_tiles + tile;

  const T *const src = static_cast<const T *>(p.src[which]) + r * p.row_s[which] + h * p.head_s[which];
  float x[kVecs][8];
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = i * NT + tid;
    const int tok = base + v / (D / 8), d = v % (D / 8) * 8;
    if (ok && tok >= held && tok < end) {
      load8(src + static_cast<int64_t>(tok - held) * p.tok_s[which] + d, p.vec, x[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = fabsf(x[i][j]);
        top = fmaxf(top, a <= 3.402823466e38f ? a : __int_as_float(0x7f800000));
      }
    }
  }
  // The unit's maximum.
#pragma unroll
  for (int o = (NT < 32 ? NT : 32) / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (NT > 32) {
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
    __syncthreads();
    const int w0 = threadIdx.x / NT * (NT / 32);
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) top = fmaxf(top, part[w0 + w]);
  }
  const float before = ok && base < held ? *qs : 0.0f;
  float now = fmaxf(before, top * (1.0f / 127.0f));
  if (now == 0.0f) now = 1.0f;
  const float shrink = before / now;
  // Every thread of the unit has read the old scale before one writes it.
  if (NT > 32) {
    __syncthreads();
  } else {
    __syncwarp();
  }
  if (ok && tid == 0) *qs = now;

  T *const out = p.values[which] ? static_cast<T *>(p.values[which]) : nullptr;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = i * NT + tid;
    const int tok = base + v / (D / 8), d = v % (D / 8) * 8;
    float val[8] = {};
    if (ok && tok < end) {
      int q[8];
      const bool is_new = tok >= held;
      uint2 w = make_uint2(0, 0);
      uint2 *const at = reinterpret_cast<uint2 *>(q8 + (tok - base) * D + d);
      if (is_new) {
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = static_cast<int>(rintf(x[i][j] / now));
      } else if (out || shrink != 1.0f) {
        w = *at;
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = static_cast<int>(rintf(static_cast<float>(byte_of(w, j)) * shrink));
      }
      if (is_new || shrink != 1.0f) {
        w.x = (q[0] & 255) | (q[1] & 255) << 8 | (q[2] & 255) << 16 | static_cast<uint32_t>(q[3]) << 24;
        w.y = (q[4] & 255) | (q[5] & 255) << 8 | (q[6] & 255) << 16 | static_cast<uint32_t>(q[7]) << 24;
        *at = w;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) val[j] = static_cast<float>(q[j]) * now;
    }
    if (out && in) {
      const int64_t at = ((static_cast<int64_t>(r) * p.spans * BS + span * BS + v / (D / 8)) * p.c.heads + h) * D + d;
      *reinterpret_cast<uint4 *>(out + at) = make_uint4(pack2<T>(val[0], val[1]), pack2<T>(val[2], val[3]),
                                                        pack2<T>(val[4], val[5]), pack2<T>(val[6], val[7]));
    }
  }
}

struct ReadParams {
  KvView c;
  void *out[2];
  int32_t start, count, layers;
  int64_t vecs;  // layers * rows * count * heads * head_dim / 8
};

template <typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams p) {
  const int64_t v = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (v >= p.vecs) return;
  const int which = blockIdx.y;
  const int per = p.c.head_dim / 8;
  const int d = static_cast<int>(v % per) * 8;
  int64_t u = v / per;
  const int h = static_cast<int>(u % p.c.heads);
  u /= p.c.heads;
  const int64_t tok = p.start + u % p.count;
  u /= p.count;
  const int r = static_cast<int>(u % p.c.rows);
  const int64_t layer = u / p.c.rows;
  const int64_t col = tok / p.c.block;
  uint4 w = make_uint4(0, 0, 0, 0);
  if (tok < p.c.lens[r] && col < p.c.width) {
    const int blk = p.c.table[static_cast<int64_t>(r) * p.c.width + col];
    if (blk >= 0 && blk < p.c.blocks) {
      const int64_t tile = p.c.layer_tiles + (layer * p.c.blocks + blk) * p.c.heads + h;
      const float s = (which ? p.c.v_scale : p.c.k_scale)[tile];
      const uint2 q = *reinterpret_cast<const uint2 *>((which ? p.c.v8 : p.c.k8) +
                                                       (tile * p.c.block + tok % p.c.block) * p.c.head_dim + d);
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = static_cast<float>(byte_of(q, j)) * s;
      w = make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
    }
  }
  reinterpret_cast<uint4 *>(p.out[which])[v] = w;
}

struct ReorderParams {
  KvView c;
  const int32_t *parents;
  uint32_t *done;    // per clip: CTAs that have copied
  int32_t beams, parts;
};

// The parent row of row r, r itself where the given one is out of range.
__device__ __forceinline__ int parent_row(const ReorderParams &p, int r) {
  const int q = p.parents[r];
  return q >= 0 && q < p.beams ? r / p.beams * p.beams + q : r;
}

// Grid: (part, row).  Each CTA copies its part of the row's open block (over
// layers, keys and values, heads) from the parent's to the row's spare one.
// The tables still show the old state meanwhile; the last CTA of a clip to
// finish then rewrites them.
__global__ void __launch_bounds__(kThreads) reorder_kernel(const ReorderParams p) {
  const int r = blockIdx.y;
  const int clip = r / p.beams;
  const int64_t width = p.c.width;
  const int len = max(p.c.lens[clip * p.beams], 0);
  const int col = len / p.c.block;
  const bool open = len % p.c.block != 0 && col < width;
  const int from_row = parent_row(p, r);
  if (open && from_row != r) {
    const int from = p.c.table[from_row * width + col], to = p.c.spare[r];
    if (from >= 0 && from < p.c.blocks && to >= 0 && to < p.c.blocks) {
      // 16-byte vectors of a block's keys or values over all heads, per layer.
      const int64_t vecs = static_cast<int64_t>(p.c.heads) * p.c.block * p.c.head_dim / 16;
      const int64_t all = vecs * p.c.layers;
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < all;
           i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t layer = i / vecs, v = i % vecs;
        const int64_t a = (layer * p.c.blocks + from) * vecs + v, b = (layer * p.c.blocks + to) * vecs + v;
        reinterpret_cast<uint4 *>(p.c.k8)[b] = reinterpret_cast<const uint4 *>(p.c.k8)[a];
        reinterpret_cast<uint4 *>(p.c.v8)[b] = reinterpret_cast<const uint4 *>(p.c.v8)[a];
      }
      const int scales = p.c.heads * p.c.layers;
      for (int i = blockIdx.x * kThreads + threadIdx.x; i < scales; i += gridDim.x * kThreads) {
        const int64_t layer = i / p.c.heads, h = i % p.c.heads;
        const int64_t a = (layer * p.c.blocks + from) * p.c.heads + h, b = (layer * p.c.blocks + to) * p.c.heads + h;
        p.c.k_scale[b] = p.c.k_scale[a];
        p.c.v_scale[b] = p.c.v_scale[a];
      }
    }
  }
  // Last CTA of the clip: every reader of the old tables has finished.
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(&p.done[clip], 1u) == static_cast<uint32_t>(p.beams * p.parts - 1);
  }
  __syncthreads();
  if (!last) return;
  if (threadIdx.x == 0) p.done[clip] = 0;
  // A column at a time per thread: its entries of all beams are read before
  // one is written.
  const int row0 = clip * p.beams;
  const int cols = static_cast<int>(min(static_cast<int64_t>(col) + (open ? 1 : 0), width));
  for (int c = threadIdx.x; c < cols; c += kThreads) {
    int32_t was[32];
    for (int i = 0; i < p.beams; ++i) was[i] = p.c.table[(row0 + i) * width + c];
    for (int i = 0; i < p.beams; ++i) {
      const int from = parent_row(p, row0 + i) - row0;
      if (from == i) continue;
      if (c < col) {
        p.c.table[(row0 + i) * width + c] = was[from];
      } else {
        p.c.table[(row0 + i) * width + c] = p.c.spare[row0 + i];
        p.c.spare[row0 + i] = was[i];
      }
    }
  }
}

template <typename T, int D>
lm_status append_block(const AppendParams &p, int block, cudaStream_t s) {
  const int nt = block * D / 64;
  const int64_t ctas = (p.units * nt + kThreads - 1) / kThreads;
  if (ctas > INT_MAX) return LM_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(ctas), 2);
  switch (block) {
    case 16: append_kernel<T, D, 16><<<grid, kThreads, 0, s>>>(p); break;
    case 32: append_kernel<T, D, 32><<<grid, kThreads, 0, s>>>(p); break;
    case 64: append_kernel<T, D, 64><<<grid, kThreads, 0, s>>>(p); break;
    default: append_kernel<T, D, 128><<<grid, kThreads, 0, s>>>(p); break;
  }
  LM_CUDA_TRY(cudaGetLastError());
  return LM_OK;
}

template <typename T>
lm_status append_dim(const AppendParams &p, int dim, int block, cudaStream_t s) {
  switch (dim) {
    case 32: return append_block<T, 32>(p, block, s);
    case 64: return append_block<T, 64>(p, block, s);
    default: return append_block<T, 128>(p, block, s);
  }
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

lm_status kv_check(const lm_kv_cache *c) {
  if (!c) return LM_ERR_INVALID_ARG;
  if (c->rows != 0 && !c->lens) return LM_ERR_INVALID_ARG;
  if (c->rows != 0 && c->width != 0 && (!c->k8 || !c->v8 || !c->k_scale || !c->v_scale || !c->table))
    return LM_ERR_INVALID_ARG;
  if (c->blocks < 0 || c->layers < 1 || c->rows < 0 || c->width < 0 || c->heads < 1) return LM_ERR_INVALID_ARG;
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) return LM_ERR_UNSUPPORTED;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) return LM_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->width) * c->block > INT_MAX - 65536 || c->blocks > INT_MAX) return LM_ERR_UNSUPPORTED;
  if (!aligned(c->k8, 16) || !aligned(c->v8, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->table, 4) || !aligned(c->lens, 4))
    return LM_ERR_MISALIGNED;
  return LM_OK;
}

KvView kv_view(const lm_kv_cache *c, int32_t layer) {
  KvView v;
  v.k8 = c->k8;
  v.v8 = c->v8;
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.table = c->table;
  v.spare = c->spare;
  v.lens = c->lens;
  v.blocks = c->blocks;
  v.layer_tiles = static_cast<int64_t>(layer < 0 ? 0 : layer) * c->blocks * c->heads;
  v.layers = c->layers;
  v.rows = c->rows;
  v.width = c->width;
  v.heads = c->heads;
  v.head_dim = c->head_dim;
  v.block = c->block;
  return v;
}

}  // namespace lm

extern "C" lm_status lm_kv_append(const lm_kv_cache *cache, int32_t layer, const void *k, const void *v,
                                  const int64_t *k_strides, const int64_t *v_strides, int32_t tokens,
                                  const int32_t *counts, int32_t dtype, void *k_values, void *v_values,
                                  lm_stream_t stream) {
  using namespace lm;
  if (lm_status st = kv_check(cache); st != LM_OK) return st;
  if (layer < 0 || layer >= cache->layers || tokens < 0 || !k_strides || !v_strides) return LM_ERR_INVALID_ARG;
  if (dtype != LM_F16 && dtype != LM_BF16) return LM_ERR_UNSUPPORTED;
  if ((k_values == nullptr) != (v_values == nullptr)) return LM_ERR_INVALID_ARG;
  if (cache->rows == 0 || tokens == 0) return LM_OK;
  if (!k || !v) return LM_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (k_strides[i] < 0 || v_strides[i] < 0) return LM_ERR_INVALID_ARG;
  if (!aligned(k, 2) || !aligned(v, 2) || !aligned(k_values, 16) || !aligned(v_values, 16)) return LM_ERR_MISALIGNED;
  if (tokens > INT_MAX - 256) return LM_ERR_UNSUPPORTED;
  AppendParams p;
  p.c = kv_view(cache, layer);
  p.src[0] = k;
  p.src[1] = v;
  p.values[0] = k_values;
  p.values[1] = v_values;
  p.vec = aligned(k, 16) && aligned(v, 16);
  for (int w = 0; w < 2; ++w) {
    const int64_t *s = w ? v_strides : k_strides;
    p.row_s[w] = s[0];
    p.tok_s[w] = s[1];
    p.head_s[w] = s[2];
    for (int i = 0; i < 3; ++i) p.vec = p.vec && s[i] % 8 == 0;
  }
  p.counts = counts;
  p.tokens = tokens;
  p.spans = (tokens - 1 + cache->block - 1) / cache->block + 1;
  p.units = static_cast<int64_t>(cache->rows) * p.spans * cache->heads;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == LM_F16 ? append_dim<__half>(p, cache->head_dim, cache->block, s)
                         : append_dim<__nv_bfloat16>(p, cache->head_dim, cache->block, s);
}

extern "C" lm_status lm_kv_read(const lm_kv_cache *cache, int32_t layer, int32_t start, int32_t count, int32_t dtype,
                                void *k_out, void *v_out, lm_stream_t stream) {
  using namespace lm;
  if (lm_status st = kv_check(cache); st != LM_OK) return st;
  if (layer < -1 || layer >= cache->layers || start < 0 || count < 0) return LM_ERR_INVALID_ARG;
  if (dtype != LM_F16 && dtype != LM_BF16) return LM_ERR_UNSUPPORTED;
  if (cache->rows == 0 || count == 0) return LM_OK;
  if (!k_out || !v_out) return LM_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return LM_ERR_MISALIGNED;
  ReadParams p;
  p.c = kv_view(cache, layer);
  p.out[0] = k_out;
  p.out[1] = v_out;
  p.start = start;
  p.count = count;
  p.layers = layer < 0 ? cache->layers : 1;
  p.vecs = static_cast<int64_t>(p.layers) * cache->rows * count * cache->heads * (cache->head_dim / 8);
  const int64_t ctas = (p.vecs + kThreads - 1) / kThreads;
  if (ctas > INT_MAX) return LM_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(ctas), 2);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == LM_F16) {
    read_kernel<__half><<<grid, kThreads, 0, s>>>(p);
  } else {
    read_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
  }
  LM_CUDA_TRY(cudaGetLastError());
  return LM_OK;
}

extern "C" lm_status lm_kv_reorder(const lm_kv_cache *cache, const int32_t *parents, int32_t beams, void *workspace,
                                   size_t workspace_bytes, lm_stream_t stream) {
  using namespace lm;
  if (lm_status st = kv_check(cache); st != LM_OK) return st;
  if (beams < 1 || cache->rows % beams != 0) return LM_ERR_INVALID_ARG;
  if (beams > 32 || cache->rows > 65535) return LM_ERR_UNSUPPORTED;
  if (cache->rows == 0 || cache->width == 0) return LM_OK;
  if (!parents || !cache->spare) return LM_ERR_INVALID_ARG;
  const int clips = cache->rows / beams;
  if (!workspace || workspace_bytes < kWorkspaceHeaderBytes + 4 * static_cast<size_t>(clips)) return LM_ERR_WORKSPACE;
  if (!aligned(workspace, 16) || !aligned(parents, 4) || !aligned(cache->spare, 4)) return LM_ERR_MISALIGNED;
  ReorderParams p;
  p.c = kv_view(cache, 0);
  p.parents = parents;
  p.done = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + kWorkspaceHeaderBytes);
  p.beams = beams;
  // 8 vectors of keys and of values per thread, within one wave of CTAs or so.
  const int64_t vecs = static_cast<int64_t>(cache->layers) * cache->heads * cache->block * cache->head_dim / 16;
  p.parts = static_cast<int32_t>(vecs / (8 * kThreads) > 0 ? (vecs / (8 * kThreads) < 64 ? vecs / (8 * kThreads) : 64) : 1);
  reorder_kernel<<<dim3(p.parts, cache->rows), kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  LM_CUDA_TRY(cudaGetLastError());
  return LM_OK;
}
