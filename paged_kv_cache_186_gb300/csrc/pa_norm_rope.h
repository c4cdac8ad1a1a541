// Internal interface of the norm + rotation + store kernel (not part of the
// public ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

struct NormRopeArgs {
  const void* q;  // (T, H, D) bf16, tokens q_stride elements apart
  const void* k;  // (T, Hkv, D) bf16
  const void* v;
  long long q_stride, k_stride, v_stride;
  const void* q_weight;  // (D) bf16, or NULL: no norm
  const void* k_weight;
  const float* cos_sin;  // (max_positions, rotary_dim), or NULL
  const int64_t* positions;
  const int64_t* slot_mapping;
  void* q_out;  // (T, H, D) bf16
  void* k_cache;
  void* v_cache;
  float* k_scale;  // 8-bit caches: (NB, Hkv, bs)
  float* v_scale;
  float* scores;  // (NB, Hkv, bs) or NULL
  uint32_t* err;
  long long num_slots;
  int num_tokens, num_heads, num_kv_heads, head_dim, block_size;
  int max_positions, rotary_dim, interleaved;
  int kv;  // kKvBf16, kKvE4m3 or kKvInt8
  float eps;
  int num_sms;
  int rows_per_warp;  // set by the launch
};

cudaError_t launch_norm_rope_store(const NormRopeArgs& a, cudaStream_t stream);

}  // namespace pa
