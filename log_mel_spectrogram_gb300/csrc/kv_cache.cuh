// kv_cache.cuh -- the 8-bit key/value cache as its kernels see it.
#pragma once

#include <cstdint>

#include "logmel.h"

namespace lm {

struct KvView {
  int8_t *k8, *v8;
  float *k_scale, *v_scale;
  int32_t *table, *spare, *lens;
  int64_t blocks;
  int64_t layer_tiles;  // (block, head) tiles in front of the layer
  int32_t layers, rows, width, heads, head_dim, block;
};

// Argument rules of every cache entry point.
lm_status kv_check(const lm_kv_cache *c);

// The cache from `layer` on (the first for -1).
KvView kv_view(const lm_kv_cache *c, int32_t layer);

}  // namespace lm
