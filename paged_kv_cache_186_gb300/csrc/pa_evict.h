// Internal interface of the eviction kernels (not part of the public ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

struct EvictArgs {
  void* k_cache;  // (NB, bs, Hkv, D) of row_bytes per (slot, head)
  void* v_cache;
  float* k_scale;  // 8-bit caches: (NB, Hkv, bs), else NULL
  float* v_scale;
  float* scores;  // (NB, Hkv, bs)
  const int32_t* block_tables;  // (B, max_blocks)
  const int32_t* context_lens;  // (B)
  int32_t* kept;                // (B, Hkv, budget)
  int32_t* new_lens;            // (B)
  uint32_t* err;
  int batch, num_kv_heads, block_size, num_blocks, max_blocks, len_cap;
  int row_bytes;  // head_dim * element size
  int budget, sinks, recent;
};

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream);

}  // namespace pa
