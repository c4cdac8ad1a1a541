// Internal interface of the shared-context kernels (pa_decode_shared,
// pa_prefill_shared); not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pa {

// What the plan launch writes for the launches behind it. A row is a token of
// the packed q (a sequence, in a decode step).
struct SharedPlan {
  int* cu;          // (groups+1) first sequence of each group, made to ascend within [0, batch]
  int* keys;        // (groups) shared keys: whole blocks; 0: the group shares nothing
  int* owner;       // (groups) sequence whose block table row names the shared blocks
  int* tok;         // (groups, 2) the group's rows: first, past the last
  int* seg;         // (groups+1) segments (kv head, row tile) before the group
  long long* unit;  // (groups+1) units (a segment's 128-key tiles) before the group
  int2* parts;      // (segments) slot of the segment's first partial, partials
  int* row_vis;     // (rows) keys the row sees; -1: the row belongs to no sequence
  int* row_grp;     // (rows) the row's group, -1 if that shares nothing
  int* row_start;   // (rows) keys of the row's sequence that its group attends to
};

struct SharedArgs {
  const int32_t* block_tables;
  const int32_t* context_lens;  // decode, else NULL
  const int32_t* cu_q;          // prefill, else NULL
  const int32_t* cu_k;
  const int32_t* cu_groups;
  const int32_t* prefix_lens;
  void* out;      // (rows, H, D) bf16
  uint32_t* err;
  const float* k_scale;  // 8-bit caches: (NB, Hkv, bs)
  const float* v_scale;
  SharedPlan plan;
  float* part_o;    // (slots, rows of a segment, D) fp32, of the shared keys
  float2* part_ml;  // (slots, rows of a segment): max, sum
  float* own_o;     // (rows, H, D) fp32, of each row's own keys
  float2* own_ml;   // (rows, H)
  // decode: where a sequence and kv head's own result is: (-1, 1) in own_o, else
  // (first warp, parts) in the decode kernel's partial slots; the plan sets (-1, 0),
  // nowhere
  int2* own_parts;         // (rows, Hkv), NULL for prefill
  const float* slot_o;     // (slots, slot_rows, D)
  const float2* slot_ml;   // (slots, slot_rows)
  int slot_rows;
  int batch, num_groups, rows;
  int num_heads, num_kv_heads, group, head_dim, block_size, max_blocks, num_blocks;
  int len_cap;          // keys a sequence may have
  int tokens_per_tile;  // rows of q in a tile: 128 / group
  int row_tiles;        // tiles of a segment: 1 or 2
  int max_segments;     // segments the workspace has room for
  int ctas;             // grid of the launch over the shared keys
  int kv;               // kKvBf16, kKvE4m3 or kKvInt8
  int always;           // prefill: share whether or not it pays
  int own_tokens;       // prefill: new tokens a CTA of the launch over own keys takes
  float scale_log2;
};

// Sizes of a call: grid, segment form and the workspace's parts (byte offsets).
struct SharedLayout {
  int tokens_per_tile, row_tiles, max_segments, ctas;
  size_t plan, part_ml, part_o, own_parts, own_ml, own_o, bytes;
};
SharedLayout shared_layout(size_t base, int rows, int num_heads, int num_kv_heads, int head_dim,
                           int num_groups, int num_sms);
// Bytes that serve this call and every one of fewer rows or groups (base: what those
// need in front of it).
size_t shared_workspace_bytes(size_t base, int rows, int num_heads, int num_kv_heads, int head_dim,
                              int num_groups, int num_sms);
// Fill the workspace pointers of `a` (rows, num_groups set) from a layout.
void shared_pointers(SharedArgs& a, const SharedLayout& l, void* workspace);

// The launches of a call, in order: plan, (the caller's launch over each
// sequence's own keys), shared keys, merge.
cudaError_t launch_shared_plan(const SharedArgs& a, cudaStream_t stream);
cudaError_t launch_shared_keys(const SharedArgs& a, const CUtensorMap& qmap,
                               const CUtensorMap& kmap, const CUtensorMap& vmap,
                               cudaStream_t stream);
cudaError_t launch_shared_merge(const SharedArgs& a, cudaStream_t stream);

}  // namespace pa
