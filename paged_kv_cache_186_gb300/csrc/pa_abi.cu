// C-ABI entry points: argument validation, tensor-map encoding, launch.
// Every check happens on the host before any launch; nothing here reads
// device memory or synchronises (except pa_get_device_error).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <atomic>
#include <mutex>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_evict.h"
#include "pa_launch.h"
#include "pa_norm_rope.h"
#include "pa_prefill.h"
#include "pa_shared.h"

namespace {

// Per-device error word (PA_DEVERR_* bits), set by kernels with atomicOr.
__device__ uint32_t g_device_error;

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  bool ready = false;
  uint32_t* err = nullptr;
  int num_sms = 0;
};

std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

// Resolve per-device state (error-word address, SM count) for the current
// device; the first call on a device does the lookup.
pa_status device_info(DeviceInfo** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return PA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.ready) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return PA_ERR_CUDA;
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return PA_ERR_CUDA;
    d.err = static_cast<uint32_t*>(p);
    d.num_sms = sms;
    d.ready = true;
  }
  if (g_encode == nullptr) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr)
      return PA_ERR_CUDA;
    g_encode = reinterpret_cast<EncodeTiledFn>(fn);
  }
  *out = &d;
  return PA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

pa_status check_cache(const pa_kv_cache* c) {
  if (c == nullptr || c->k_cache == nullptr || c->v_cache == nullptr) return PA_ERR_NULL;
  if (c->num_blocks <= 0 || c->block_size <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0)
    return PA_ERR_SHAPE;
  if (c->dtype != PA_KV_BF16 && c->dtype != PA_KV_FP8_E4M3 && c->dtype != PA_KV_INT8)
    return PA_ERR_DTYPE;
  const bool q8 = c->dtype != PA_KV_BF16;  // 8-bit codes with scales
  if (q8 && (c->k_scale == nullptr || c->v_scale == nullptr)) return PA_ERR_DTYPE;
  if (!q8 && (c->k_scale != nullptr || c->v_scale != nullptr)) return PA_ERR_DTYPE;
  if (c->block_size != 16 && c->block_size != 32) return PA_ERR_UNSUPPORTED;
  if (q8 ? c->head_dim != 128 : (c->head_dim != 64 && c->head_dim != 128))
    return PA_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->num_blocks) * c->block_size > 0x7fffffffLL) return PA_ERR_SHAPE;
  if (!aligned16(c->k_cache) || !aligned16(c->v_cache)) return PA_ERR_ALIGN;
  if (q8 && (!aligned16(c->k_scale) || !aligned16(c->v_scale))) return PA_ERR_ALIGN;
  return PA_OK;
}

int elem_bytes(const pa_kv_cache* c) { return c->dtype == PA_KV_BF16 ? 2 : 1; }

// Tensor maps over a cache, 128B-swizzled to match the kernels' shared-memory
// layouts. A tile is block_size rows of one kv head, stored as 128-byte-wide
// subtiles one after the other (subtile j holds bytes [128 j, 128 j + 128) of
// every row).
//   kind kSubtileMap (prefill): the cache as 3-D (head_dim, num_kv_heads,
//     num_blocks*block_size); one box is one subtile.
//   kind kRowMap (decode): the cache as 4-D (128 bytes of a row, row,
//     subtile, kv head), box (128 bytes, block_size, all subtiles, 1): one box
//     is a whole tile, one copy instead of one per subtile.
constexpr int kSubtileMap = 0, kRowMap = 1;
pa_status encode_cache_map(CUtensorMap* map, void* base, const pa_kv_cache* c, int kind) {
  const int eb = elem_bytes(c);
  const cuuint64_t row_bytes = static_cast<cuuint64_t>(c->head_dim) * eb;
  const cuuint64_t rows = static_cast<cuuint64_t>(c->num_blocks) * c->block_size;
  const CUtensorMapDataType dt =
      eb == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  // rows are head_dim*elem bytes apart from the next head's: promote L2
  // fills no wider than one row so no neighbouring head is fetched
  const CUtensorMapL2promotion promo =
      eb == 1 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  CUresult r;
  if (kind == kSubtileMap) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c->head_dim),
                                static_cast<cuuint64_t>(c->num_kv_heads), rows};
    const cuuint64_t strides[2] = {row_bytes, row_bytes * c->num_kv_heads};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(pa::kSwizzleBytes / eb), 1u,
                               static_cast<cuuint32_t>(c->block_size)};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    r = g_encode(map, dt, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                 CU_TENSOR_MAP_SWIZZLE_128B, promo, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else {
    const cuuint64_t nsub = row_bytes / pa::kSwizzleBytes;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(pa::kSwizzleBytes / eb), rows, nsub,
                                static_cast<cuuint64_t>(c->num_kv_heads)};
    const cuuint64_t strides[3] = {row_bytes * c->num_kv_heads,
                                   static_cast<cuuint64_t>(pa::kSwizzleBytes), row_bytes};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(pa::kSwizzleBytes / eb),
                               static_cast<cuuint32_t>(c->block_size),
                               static_cast<cuuint32_t>(nsub), 1u};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    r = g_encode(map, dt, 4, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                 CU_TENSOR_MAP_SWIZZLE_128B, promo, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  return r == CUDA_SUCCESS ? PA_OK : PA_ERR_CUDA;
}

// Recently encoded cache tensor maps: encoding is pure host work but costs a
// few microseconds, and a decode loop passes the same caches every step (four
// maps a layer where shared keys are attended to beside each sequence's own).
struct MapEntry {
  void* base;
  int num_blocks, block_size, num_kv_heads, head_dim, dtype, device, kind;
  CUtensorMap map;
};
constexpr int kMapCache = 256;
MapEntry g_maps[kMapCache];
int g_map_count = 0, g_map_next = 0;
std::mutex g_map_mu;

pa_status cached_cache_map(CUtensorMap* out, void* base, const pa_kv_cache* c, int kind) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_map_mu);
  for (int i = 0; i < g_map_count; ++i) {
    const MapEntry& e = g_maps[i];
    if (e.base == base && e.num_blocks == c->num_blocks && e.block_size == c->block_size &&
        e.num_kv_heads == c->num_kv_heads && e.head_dim == c->head_dim && e.dtype == c->dtype &&
        e.device == dev && e.kind == kind) {
      *out = e.map;
      return PA_OK;
    }
  }
  MapEntry e{base, c->num_blocks, c->block_size, c->num_kv_heads, c->head_dim, c->dtype, dev,
             kind, {}};
  const pa_status st = encode_cache_map(&e.map, base, c, kind);
  if (st != PA_OK) return st;
  g_maps[g_map_next] = e;
  g_map_next = (g_map_next + 1) % kMapCache;
  if (g_map_count < kMapCache) ++g_map_count;
  *out = e.map;
  return PA_OK;
}

// Failure-detection test hook (pa_debug_inject_wait_timeout): the copy the
// first warp of decode CTA 0 leaves unissued (-1: none) and the wait bound
// of decode launches (0: kWaitLimitNs).
std::atomic<int> g_debug_skip_copy{-1};
std::atomic<unsigned long long> g_debug_wait_limit_ns{0};

// Tag of one decode call in the workspace's arrival counters: a call counter
// passed through a 64-bit finalising mix (the one of SplitMix64, a bijection
// of 64-bit words), upper half kept, never 0 (a zeroed counter never matches
// the current call). Consecutive calls thus get unrelated tags, and a word of
// arbitrary earlier contents carries the current call's tag with probability
// 2^-32, not "whenever it holds a small integer".
uint32_t next_epoch() {
  static std::atomic<uint64_t> counter{0};
  while (true) {
    uint64_t z = counter.fetch_add(1) + 0x9e3779b97f4a7c15ull;
    z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
    z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
    z ^= z >> 31;
    const uint32_t e = static_cast<uint32_t>(z >> 32);
    if (e != 0) return e;
  }
}

int decode_len_cap(const pa_kv_cache* c, int32_t max_blocks_per_seq, int32_t max_context_len) {
  const long long cap = static_cast<long long>(max_blocks_per_seq) * c->block_size;
  long long v = max_context_len > 0 ? std::min<long long>(max_context_len, cap) : cap;
  return static_cast<int>(std::min<long long>(v, 0x7fffffffLL));
}

}  // namespace

extern "C" {

int32_t pa_abi_version(void) { return PA_ABI_VERSION; }

const char* pa_status_string(pa_status s) {
  switch (s) {
    case PA_OK: return "ok";
    case PA_ERR_NULL: return "required pointer is NULL";
    case PA_ERR_SHAPE: return "invalid or inconsistent size";
    case PA_ERR_DTYPE: return "cache dtype and scale pointers do not match";
    case PA_ERR_UNSUPPORTED: return "unsupported head_dim, block_size or head grouping";
    case PA_ERR_CUDA: return "CUDA call or kernel launch failed";
    case PA_ERR_WORKSPACE: return "workspace missing or too small";
    case PA_ERR_ALIGN: return "pointer not 16-byte aligned";
    case PA_ERR_TOO_LARGE: return "shape needs more scratch than the static buffer holds";
  }
  return "unknown status";
}

pa_status pa_store_kv(const void* k, const void* v, const float* k_scale_new,
                      const float* v_scale_new, const int64_t* slot_mapping, int32_t num_tokens,
                      const pa_kv_cache* cache, void* stream) {
  pa_status st = check_cache(cache);
  if (st != PA_OK) return st;
  if (num_tokens < 0) return PA_ERR_SHAPE;
  if (num_tokens == 0) return PA_OK;
  if (k == nullptr || v == nullptr || slot_mapping == nullptr) return PA_ERR_NULL;
  const bool q8 = cache->dtype != PA_KV_BF16;  // 8-bit codes with scales
  if (q8 != (k_scale_new != nullptr) || q8 != (v_scale_new != nullptr)) return PA_ERR_DTYPE;
  if (!aligned16(k) || !aligned16(v)) return PA_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != PA_OK) return st;
  pa::StoreArgs a{};
  a.k = k;
  a.v = v;
  a.k_scale_new = k_scale_new;
  a.v_scale_new = v_scale_new;
  a.slot_mapping = slot_mapping;
  a.k_cache = cache->k_cache;
  a.v_cache = cache->v_cache;
  a.k_scale = q8 ? cache->k_scale : nullptr;
  a.v_scale = q8 ? cache->v_scale : nullptr;
  a.num_tokens = num_tokens;
  a.row_bytes = cache->num_kv_heads * cache->head_dim * elem_bytes(cache);
  a.num_kv_heads = cache->num_kv_heads;
  a.block_size = cache->block_size;
  a.num_slots = static_cast<long long>(cache->num_blocks) * cache->block_size;
  a.err = dev->err;
  return pa::launch_store_kv(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK
                                                                                  : PA_ERR_CUDA;
}

}  // extern "C"

namespace {

// Shared body of pa_norm_rope_store (num_axes 0) and pa_norm_rope_axes_store.
pa_status norm_rope_common(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, const pa_norm_rope* params,
                           const int64_t* positions, const int64_t* slot_mapping,
                           int32_t num_tokens, int32_t num_heads, const pa_kv_cache* cache,
                           float* scores, void* q_out, void* stream, int32_t num_axes = 0,
                           const uint8_t* pair_axis = nullptr) {
  pa_status st = check_cache(cache);
  if (st != PA_OK) return st;
  if (params == nullptr) return PA_ERR_NULL;
  if (num_tokens < 0 || num_heads <= 0) return PA_ERR_SHAPE;
  const int D = cache->head_dim, rot = params->rotary_dim;
  if (rot < 0 || rot > D || (rot > 0 && params->max_positions <= 0)) return PA_ERR_SHAPE;
  if (rot % 16 != 0) return PA_ERR_UNSUPPORTED;
  if (!(params->eps >= 0.f) || !std::isfinite(params->eps)) return PA_ERR_SHAPE;
  const int64_t qrow = static_cast<int64_t>(num_heads) * D;
  const int64_t krow = static_cast<int64_t>(cache->num_kv_heads) * D;
  if (q_stride < qrow || k_stride < krow || v_stride < krow) return PA_ERR_SHAPE;
  if (q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0) return PA_ERR_SHAPE;
  if (q_out == q && q_stride != qrow) return PA_ERR_SHAPE;
  if (num_tokens == 0) return PA_OK;
  if (q == nullptr || k == nullptr || v == nullptr || slot_mapping == nullptr || q_out == nullptr ||
      (rot > 0 && (positions == nullptr || params->cos_sin == nullptr)))
    return PA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
      !aligned16(params->q_weight) || !aligned16(params->k_weight) || !aligned16(params->cos_sin) ||
      !aligned16(scores))
    return PA_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != PA_OK) return st;
  const bool q8 = cache->dtype != PA_KV_BF16;
  pa::NormRopeArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_weight = params->q_weight;
  a.k_weight = params->k_weight;
  a.cos_sin = params->cos_sin;
  a.positions = positions;
  a.slot_mapping = slot_mapping;
  a.q_out = q_out;
  a.k_cache = cache->k_cache;
  a.v_cache = cache->v_cache;
  a.k_scale = q8 ? cache->k_scale : nullptr;
  a.v_scale = q8 ? cache->v_scale : nullptr;
  a.scores = scores;
  a.err = dev->err;
  a.num_slots = static_cast<long long>(cache->num_blocks) * cache->block_size;
  a.num_tokens = num_tokens;
  a.num_heads = num_heads;
  a.num_kv_heads = cache->num_kv_heads;
  a.head_dim = D;
  a.block_size = cache->block_size;
  a.max_positions = params->max_positions;
  a.rotary_dim = rot;
  a.interleaved = params->interleaved != 0;
  a.kv = static_cast<int>(cache->dtype);
  a.eps = params->eps;
  a.num_sms = dev->num_sms;
  a.num_axes = num_axes;
  if (num_axes > 0) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    for (int i = 0; i < rot / 2; ++i) w[i / 16] |= static_cast<uint32_t>(pair_axis[i]) << (2 * (i % 16));
    a.pair_axis = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return pa::launch_norm_rope_store(a, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // namespace

extern "C" {

pa_status pa_norm_rope_store(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, const pa_norm_rope* params,
                             const int64_t* positions, const int64_t* slot_mapping,
                             int32_t num_tokens, int32_t num_heads, const pa_kv_cache* cache,
                             float* scores, void* q_out, void* stream) {
  return norm_rope_common(q, q_stride, k, k_stride, v, v_stride, params, positions, slot_mapping,
                          num_tokens, num_heads, cache, scores, q_out, stream);
}

pa_status pa_norm_rope_axes_store(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                  const void* v, int64_t v_stride, const pa_norm_rope* params,
                                  const int64_t* positions, int32_t num_axes,
                                  const uint8_t* pair_axis, const int64_t* slot_mapping,
                                  int32_t num_tokens, int32_t num_heads, const pa_kv_cache* cache,
                                  float* scores, void* q_out, void* stream) {
  const pa_status st = check_cache(cache);
  if (st != PA_OK) return st;
  if (params == nullptr || pair_axis == nullptr) return PA_ERR_NULL;
  if (num_axes < 1 || params->rotary_dim <= 0 || params->rotary_dim > cache->head_dim)
    return PA_ERR_SHAPE;
  if (num_axes > 4) return PA_ERR_UNSUPPORTED;
  for (int i = 0; i < params->rotary_dim / 2; ++i)
    if (pair_axis[i] >= num_axes) return PA_ERR_SHAPE;
  return norm_rope_common(q, q_stride, k, k_stride, v, v_stride, params, positions, slot_mapping,
                          num_tokens, num_heads, cache, scores, q_out, stream, num_axes, pair_axis);
}

size_t pa_decode_workspace_size(const pa_kv_cache* cache, int32_t batch, int32_t num_heads,
                                int32_t max_blocks_per_seq, int32_t max_context_len) {
  if (check_cache(cache) != PA_OK || batch <= 0 || num_heads <= 0 || max_blocks_per_seq <= 0)
    return 0;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev) != PA_OK) return 0;
  const int cap = decode_len_cap(cache, max_blocks_per_seq, max_context_len);
  return pa::plan_decode(batch, num_heads, cache->num_kv_heads, cache->head_dim, cache->block_size,
                         static_cast<int>(cache->dtype), cap, dev->num_sms)
      .workspace_bytes;
}

}  // extern "C"

namespace {

// The groups and the workspace of a call over shared context.
struct SharedCall {
  const int32_t* cu_groups;
  const int32_t* prefix_lens;
  int32_t num_groups;
  bool share;   // decode: attend to the shared keys once
  bool always;  // prefill: likewise, whether or not it pays
  void* workspace;
  size_t workspace_bytes;
};

// Q viewed as (head_dim, num_heads, rows), bf16: one box is the G heads of a kv
// head for `tokens` consecutive rows, 64 dims (128 bytes) wide.
pa_status encode_q_map(CUtensorMap* map, const void* q, int head_dim, int num_heads, int rows,
                       int group, int tokens) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(num_heads),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {head_dim * static_cast<cuuint64_t>(2),
                                 static_cast<cuuint64_t>(num_heads) * head_dim * 2};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(tokens)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
                 CUDA_SUCCESS
             ? PA_OK
             : PA_ERR_CUDA;
}

// What the launches of a call over shared context have in common.
pa::SharedArgs shared_args(const SharedCall& call, const pa::SharedLayout& layout,
                           const pa_kv_cache* cache, const int32_t* block_tables, int32_t max_blocks,
                           int32_t batch, int32_t rows, int32_t num_heads, int len_cap, float scale,
                           void* out, uint32_t* err, const int32_t* context_lens) {
  pa::SharedArgs a{};
  a.context_lens = context_lens;
  a.block_tables = block_tables;
  a.cu_groups = call.cu_groups;
  a.prefix_lens = call.prefix_lens;
  a.out = out;
  a.err = err;
  a.batch = batch;
  a.num_groups = call.num_groups;
  a.rows = rows;
  a.num_heads = num_heads;
  a.num_kv_heads = cache->num_kv_heads;
  a.group = num_heads / cache->num_kv_heads;
  a.head_dim = cache->head_dim;
  a.block_size = cache->block_size;
  a.max_blocks = max_blocks;
  a.num_blocks = cache->num_blocks;
  a.len_cap = len_cap;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.kv = static_cast<int>(cache->dtype);
  a.scale_log2 = scale * 1.4426950408889634f;
  pa::shared_pointers(a, layout, call.workspace);
  return a;
}

// The workspace of pa_decode_shared: enough for every smaller batch and number of
// groups too.
size_t decode_shared_bytes(const pa_kv_cache* cache, int32_t batch, int32_t num_heads, int cap,
                           int32_t num_groups, int num_sms) {
  const size_t decode_bytes = pa::decode_workspace_upto(
      batch, num_heads, cache->num_kv_heads, cache->head_dim, cache->block_size,
      static_cast<int>(cache->dtype), cap, num_sms);
  return pa::shared_workspace_bytes(decode_bytes, batch, num_heads, cache->num_kv_heads,
                                    cache->head_dim, num_groups, num_sms);
}

// The workspace of pa_decode_scored: pa_decode's, then (from ml on) the final
// (max, 1 / sum) of every query head, then the scores of every key.
struct ScoredWorkspace {
  size_t ml, raw, bytes;
};
ScoredWorkspace scored_workspace(size_t decode_bytes, int32_t batch, int32_t num_heads, int cap,
                                 int block_size) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t heads = static_cast<size_t>(batch) * num_heads;
  const size_t keys = (static_cast<size_t>(cap) + block_size - 1) / block_size * block_size;
  ScoredWorkspace w;
  w.ml = up(decode_bytes);
  w.raw = up(w.ml + heads * sizeof(float2));
  w.bytes = w.raw + heads * keys * sizeof(float);
  return w;
}

// Shared body of pa_decode and pa_decode_append (k_new == NULL: no append),
// pa_decode_scored (scores != NULL) and pa_decode_shared (shared != NULL).
pa_status decode_common(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                        int32_t max_blocks_per_seq, const int32_t* context_lens,
                        int32_t max_context_len, int32_t batch, int32_t num_heads, float scale,
                        void* out, void* workspace, size_t workspace_bytes, void* stream,
                        const void* k_new, const void* v_new, const float* k_scale_new,
                        const float* v_scale_new, int32_t window, int32_t sinks,
                        float* scores = nullptr, const SharedCall* shared = nullptr) {
  pa_status st = check_cache(cache);
  if (st != PA_OK) return st;
  if (sinks < 0) return PA_ERR_SHAPE;
  if (batch < 0 || num_heads <= 0 || max_blocks_per_seq <= 0) return PA_ERR_SHAPE;
  if (batch == 0) return PA_OK;
  if (q == nullptr || block_tables == nullptr || context_lens == nullptr || out == nullptr)
    return PA_ERR_NULL;
  if (num_heads % cache->num_kv_heads != 0) return PA_ERR_SHAPE;
  const int group = num_heads / cache->num_kv_heads;
  if (group > 8) return PA_ERR_UNSUPPORTED;
  if (batch > 65535) return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return PA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(out)) return PA_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != PA_OK) return st;
  const int cap = decode_len_cap(cache, max_blocks_per_seq, max_context_len);
  const bool q8 = cache->dtype != PA_KV_BF16;  // 8-bit codes with scales
  const pa::DecodePlan plan = pa::plan_decode(batch, num_heads, cache->num_kv_heads,
                                              cache->head_dim, cache->block_size,
                                              static_cast<int>(cache->dtype), cap,
                                              dev->num_sms);
  if (scores != nullptr && plan.persistent_ctas == 0) return PA_ERR_UNSUPPORTED;
  const ScoredWorkspace sw =
      scored_workspace(plan.workspace_bytes, batch, num_heads, cap, cache->block_size);
  pa::SharedLayout layout{};
  size_t need = scores != nullptr ? sw.bytes : plan.workspace_bytes;
  if (shared != nullptr) {
    layout = pa::shared_layout(plan.workspace_bytes, batch, num_heads, cache->num_kv_heads,
                               cache->head_dim, shared->num_groups, dev->num_sms);
    need = decode_shared_bytes(cache, batch, num_heads, cap, shared->num_groups, dev->num_sms);
  }
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)))
    return PA_ERR_WORKSPACE;
  if (window > 0 && plan.persistent_ctas == 0) return PA_ERR_UNSUPPORTED;
  CUtensorMap kmap, vmap;
  if ((st = cached_cache_map(&kmap, cache->k_cache, cache, kRowMap)) != PA_OK) return st;
  if ((st = cached_cache_map(&vmap, cache->v_cache, cache, kRowMap)) != PA_OK) return st;
  const cudaStream_t strm = static_cast<cudaStream_t>(stream);
  const bool fused_append = k_new != nullptr && plan.persistent_ctas > 0;
  if (k_new != nullptr && !fused_append) {
    // grid-split path: append with its own launch first, then attend
    pa::StoreArgs s{};
    s.k = k_new;
    s.v = v_new;
    s.k_scale_new = k_scale_new;
    s.v_scale_new = v_scale_new;
    s.k_cache = cache->k_cache;
    s.v_cache = cache->v_cache;
    s.k_scale = q8 ? cache->k_scale : nullptr;
    s.v_scale = q8 ? cache->v_scale : nullptr;
    s.num_tokens = batch;
    s.row_bytes = cache->num_kv_heads * cache->head_dim * elem_bytes(cache);
    s.num_kv_heads = cache->num_kv_heads;
    s.block_size = cache->block_size;
    s.num_slots = static_cast<long long>(cache->num_blocks) * cache->block_size;
    s.err = dev->err;
    if (pa::launch_store_new_tokens(s, block_tables, max_blocks_per_seq, context_lens, cap,
                                    strm) != cudaSuccess)
      return PA_ERR_CUDA;
  }
  pa::DecodeArgs a{};
  a.q = q;
  if (fused_append) {
    a.k_new = k_new;
    a.v_new = v_new;
    a.k_scale_new = q8 ? k_scale_new : nullptr;
    a.v_scale_new = q8 ? v_scale_new : nullptr;
    a.k_cache = cache->k_cache;
    a.v_cache = cache->v_cache;
  }
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.k_scale = q8 ? cache->k_scale : nullptr;
  a.v_scale = q8 ? cache->v_scale : nullptr;
  a.out = out;
  a.slot_rows = plan.slot_rows;
  if (plan.workspace_bytes > 0) {
    const size_t rows = plan.partial_slots * plan.slot_rows;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = a.part_o + rows * cache->head_dim;
    a.prefix_out = reinterpret_cast<int*>(a.part_ml + rows * 2);
    // 8-byte aligned arrival counters after the prefix sums
    const uintptr_t cp = reinterpret_cast<uintptr_t>(a.prefix_out + batch + 1);
    a.seg_counters = reinterpret_cast<unsigned long long*>((cp + 15) & ~static_cast<uintptr_t>(15));
    a.grp_counters = a.seg_counters + static_cast<size_t>(batch) * cache->num_kv_heads;
    a.epoch = next_epoch();
  }
  a.err = dev->err;
  a.batch = batch;
  a.num_heads = num_heads;
  a.num_kv_heads = cache->num_kv_heads;
  a.group = group;
  a.head_dim = cache->head_dim;
  a.block_size = cache->block_size;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = cache->num_blocks;
  a.len_cap = cap;
  a.window = window > 0 ? window : 0;
  a.sinks = window > 0 ? sinks : 0;
  a.persistent_ctas = plan.persistent_ctas;
  a.blocks_per_split = plan.blocks_per_split;
  a.num_splits = plan.num_splits;
  a.kv = static_cast<int>(cache->dtype);
  a.scale_log2 = scale * 1.4426950408889634f;  // log2(e): scores kept in base-2 units
  const unsigned long long limit = g_debug_wait_limit_ns.load();
  a.wait_limit_ns = limit > 0 ? limit : pa::kWaitLimitNs;
  a.debug_skip_copy = g_debug_skip_copy.load();
  if (scores != nullptr) {
    char* const ws = static_cast<char*>(workspace);
    a.head_ml = reinterpret_cast<float2*>(ws + sw.ml);
    a.raw_scores = reinterpret_cast<float*>(ws + sw.raw);
  }
  if (shared != nullptr && shared->share) {
    pa::SharedArgs h = shared_args(*shared, layout, cache, block_tables, max_blocks_per_seq, batch,
                                   batch, num_heads, cap, scale, out, dev->err, context_lens);
    h.slot_o = a.part_o;
    h.slot_ml = reinterpret_cast<const float2*>(a.part_ml);
    h.slot_rows = a.slot_rows;
    a.own_start = h.plan.row_start;
    a.own_parts = h.own_parts;
    a.own_o = h.own_o;
    a.own_ml = reinterpret_cast<float*>(h.own_ml);
    CUtensorMap qmap, ksub, vsub;
    if ((st = encode_q_map(&qmap, q, cache->head_dim, num_heads, batch, group, h.tokens_per_tile)) !=
            PA_OK ||
        (st = cached_cache_map(&ksub, cache->k_cache, cache, kSubtileMap)) != PA_OK ||
        (st = cached_cache_map(&vsub, cache->v_cache, cache, kSubtileMap)) != PA_OK)
      return st;
    return pa::launch_shared_plan(h, strm) == cudaSuccess &&
                   pa::launch_decode(a, kmap, vmap, strm) == cudaSuccess &&
                   pa::launch_shared_keys(h, qmap, ksub, vsub, strm) == cudaSuccess &&
                   pa::launch_shared_merge(h, strm) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
  }
  if (pa::launch_decode(a, kmap, vmap, strm) != cudaSuccess) return PA_ERR_CUDA;
  if (scores != nullptr && pa::launch_add_scores(a, scores, dev->num_sms, strm) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_decode(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                    int32_t max_blocks_per_seq, const int32_t* context_lens,
                    int32_t max_context_len, int32_t batch, int32_t num_heads, float scale,
                    void* out, void* workspace, size_t workspace_bytes, void* stream) {
  return decode_common(q, cache, block_tables, max_blocks_per_seq, context_lens, max_context_len,
                       batch, num_heads, scale, out, workspace, workspace_bytes, stream, nullptr,
                       nullptr, nullptr, nullptr, 0, 0);
}

pa_status pa_decode_window(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* context_lens,
                           int32_t max_context_len, int32_t batch, int32_t num_heads,
                           float scale, int32_t window, int32_t sinks, void* out, void* workspace,
                           size_t workspace_bytes, void* stream) {
  return decode_common(q, cache, block_tables, max_blocks_per_seq, context_lens, max_context_len,
                       batch, num_heads, scale, out, workspace, workspace_bytes, stream, nullptr,
                       nullptr, nullptr, nullptr, window, sinks);
}

size_t pa_decode_scored_workspace_size(const pa_kv_cache* cache, int32_t batch, int32_t num_heads,
                                       int32_t max_blocks_per_seq, int32_t max_context_len) {
  const size_t decode_bytes =
      pa_decode_workspace_size(cache, batch, num_heads, max_blocks_per_seq, max_context_len);
  if (decode_bytes == 0 || batch > pa::kMaxPersistentBatch) return 0;
  return scored_workspace(decode_bytes, batch, num_heads,
                          decode_len_cap(cache, max_blocks_per_seq, max_context_len),
                          cache->block_size)
      .bytes;
}

pa_status pa_decode_scored(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* context_lens,
                           int32_t max_context_len, int32_t batch, int32_t num_heads, float scale,
                           float* scores, void* out, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (batch > 0 && scores == nullptr) return PA_ERR_NULL;
  if (!aligned16(scores)) return PA_ERR_ALIGN;
  return decode_common(q, cache, block_tables, max_blocks_per_seq, context_lens, max_context_len,
                       batch, num_heads, scale, out, workspace, workspace_bytes, stream, nullptr,
                       nullptr, nullptr, nullptr, 0, 0, scores);
}

pa_status pa_evict(const pa_kv_cache* cache, float* scores, const int32_t* block_tables,
                   int32_t max_blocks_per_seq, const int32_t* context_lens,
                   int32_t max_context_len, int32_t batch, int32_t budget, int32_t sinks,
                   int32_t recent, int32_t* kept, int32_t* new_lens, void* stream) {
  pa_status st = check_cache(cache);
  if (st != PA_OK) return st;
  if (batch < 0 || max_blocks_per_seq <= 0 || budget < 1 || sinks < 0 || recent < 0 ||
      static_cast<int64_t>(sinks) + recent > budget)
    return PA_ERR_SHAPE;
  if (batch == 0) return PA_OK;
  if (scores == nullptr || block_tables == nullptr || context_lens == nullptr || kept == nullptr ||
      new_lens == nullptr)
    return PA_ERR_NULL;
  if (new_lens < context_lens + batch && context_lens < new_lens + batch) return PA_ERR_SHAPE;
  const int cap = decode_len_cap(cache, max_blocks_per_seq, max_context_len);
  // (the kernels step 32-bit positions and rows past the length bound and the budget)
  if (batch > 65535 || cap > (1 << 30) || budget > (1 << 30)) return PA_ERR_UNSUPPORTED;
  if (!aligned16(scores)) return PA_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != PA_OK) return st;
  pa::EvictArgs a{};
  a.k_cache = cache->k_cache;
  a.v_cache = cache->v_cache;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.scores = scores;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.kept = kept;
  a.new_lens = new_lens;
  a.err = dev->err;
  a.batch = batch;
  a.num_kv_heads = cache->num_kv_heads;
  a.block_size = cache->block_size;
  a.num_blocks = cache->num_blocks;
  a.max_blocks = max_blocks_per_seq;
  a.len_cap = cap;
  a.row_bytes = cache->head_dim * elem_bytes(cache);
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  return pa::launch_evict(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK
                                                                               : PA_ERR_CUDA;
}

pa_status pa_decode_append(const void* q, const void* k_new, const void* v_new,
                           const float* k_scale_new, const float* v_scale_new,
                           const pa_kv_cache* cache, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* context_lens,
                           int32_t max_context_len, int32_t batch, int32_t num_heads,
                           float scale, void* out, void* workspace, size_t workspace_bytes,
                           void* stream) {
  return pa_decode_window_append(q, k_new, v_new, k_scale_new, v_scale_new, cache, block_tables,
                                 max_blocks_per_seq, context_lens, max_context_len, batch,
                                 num_heads, scale, 0, 0, out, workspace, workspace_bytes, stream);
}

pa_status pa_decode_window_append(const void* q, const void* k_new, const void* v_new,
                                  const float* k_scale_new, const float* v_scale_new,
                                  const pa_kv_cache* cache, const int32_t* block_tables,
                                  int32_t max_blocks_per_seq, const int32_t* context_lens,
                                  int32_t max_context_len, int32_t batch, int32_t num_heads,
                                  float scale, int32_t window, int32_t sinks, void* out,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  pa_status st = check_cache(cache);
  if (st != PA_OK) return st;
  if (batch > 0 && (k_new == nullptr || v_new == nullptr)) return PA_ERR_NULL;
  const bool q8 = cache->dtype != PA_KV_BF16;  // 8-bit codes with scales
  if (q8 != (k_scale_new != nullptr) || q8 != (v_scale_new != nullptr)) return PA_ERR_DTYPE;
  if (batch > 0 && (!aligned16(k_new) || !aligned16(v_new))) return PA_ERR_ALIGN;
  return decode_common(q, cache, block_tables, max_blocks_per_seq, context_lens, max_context_len,
                       batch, num_heads, scale, out, workspace, workspace_bytes, stream, k_new,
                       v_new, k_scale_new, v_scale_new, window, sinks);
}

}  // extern "C"

namespace {

// A window no key lies outside of, with room for the kernel's differences.
constexpr int kNoWindow = 0x7ffffe00;

// Shared body of pa_prefill_varlen (window 0), pa_prefill_window and
// pa_prefill_shared.
pa_status prefill_common(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                         int32_t max_blocks_per_seq, const int32_t* cu_seqlens_q,
                         const int32_t* cu_seqlens_k, int32_t batch, int32_t num_heads,
                         int32_t total_q, int32_t max_q_len, float scale, int32_t window,
                         int32_t sinks, void* out, void* stream,
                         const SharedCall* shared = nullptr) {
  pa_status st = check_cache(cache);
  if (st != PA_OK) return st;
  if (batch < 0 || num_heads <= 0 || total_q < 0 || max_blocks_per_seq <= 0) return PA_ERR_SHAPE;
  if (batch == 0 || total_q == 0) return PA_OK;
  if (q == nullptr || block_tables == nullptr || cu_seqlens_q == nullptr ||
      cu_seqlens_k == nullptr || out == nullptr)
    return PA_ERR_NULL;
  if (num_heads % cache->num_kv_heads != 0) return PA_ERR_SHAPE;
  const int group = num_heads / cache->num_kv_heads;
  if (cache->dtype != PA_KV_BF16 || cache->head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (group != 1 && group != 2 && group != 4 && group != 8 && group != 16)
    return PA_ERR_UNSUPPORTED;
  if (batch > 65535 || cache->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;

  if (!std::isfinite(scale) || !(scale > 0.f)) return PA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(out)) return PA_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != PA_OK) return st;
  const int tpt = pa::prefill_tokens_per_tile(group);
  const int qbound = max_q_len > 0 ? std::min(max_q_len, total_q) : total_q;
  // the grid's z extent is the number of query-tile pairs of the longest sequence
  if ((static_cast<long long>(qbound) + 2 * tpt - 1) / (2 * tpt) > 65535) return PA_ERR_UNSUPPORTED;
  pa::SharedLayout layout{};
  if (shared != nullptr) {
    layout = pa::shared_layout(0, total_q, num_heads, cache->num_kv_heads, 128, shared->num_groups,
                               dev->num_sms);
    const size_t need = pa::shared_workspace_bytes(0, total_q, num_heads, cache->num_kv_heads, 128,
                                                   shared->num_groups, dev->num_sms);
    if (shared->workspace == nullptr || shared->workspace_bytes < need ||
        !aligned16(shared->workspace))
      return PA_ERR_WORKSPACE;
  }
  CUtensorMap qmap, kmap, vmap;
  if ((st = encode_q_map(&qmap, q, 128, num_heads, total_q, group, tpt)) != PA_OK) return st;
  if ((st = cached_cache_map(&kmap, cache->k_cache, cache, kSubtileMap)) != PA_OK) return st;
  if ((st = cached_cache_map(&vmap, cache->v_cache, cache, kSubtileMap)) != PA_OK) return st;
  pa::PrefillArgs a{};
  a.block_tables = block_tables;
  a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.out = out;
  a.err = dev->err;
  a.batch = batch;
  a.num_heads = num_heads;
  a.num_kv_heads = cache->num_kv_heads;
  a.group = group;
  a.head_dim = cache->head_dim;
  a.block_size = cache->block_size;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = cache->num_blocks;
  a.tokens_per_tile = tpt;
  a.num_qtiles = (qbound + tpt - 1) / tpt;
  a.scale_log2 = scale * 1.4426950408889634f;
  // (the kernel subtracts the window and a key's offset from a position)
  a.window = std::min(window, kNoWindow);
  a.sinks = sinks;
  if (shared != nullptr) {
    const cudaStream_t strm = static_cast<cudaStream_t>(stream);
    pa::SharedArgs h = shared_args(*shared, layout, cache, block_tables, max_blocks_per_seq, batch,
                                   total_q, num_heads, decode_len_cap(cache, max_blocks_per_seq, 0),
                                   scale, out, dev->err, nullptr);
    h.cu_q = cu_seqlens_q;
    h.cu_k = cu_seqlens_k;
    h.always = shared->always;
    h.own_tokens = pa::prefill_shared_tokens(tpt, a.num_qtiles);
    a.own_start = h.plan.row_start;
    a.own_group = h.plan.row_grp;
    a.own_o = h.own_o;
    a.own_ml = h.own_ml;
    return pa::launch_shared_plan(h, strm) == cudaSuccess &&
                   pa::launch_prefill(a, qmap, kmap, vmap, strm) == cudaSuccess &&
                   pa::launch_shared_keys(h, qmap, kmap, vmap, strm) == cudaSuccess &&
                   pa::launch_shared_merge(h, strm) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
  }
  return pa::launch_prefill(a, qmap, kmap, vmap, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // namespace

extern "C" {

pa_status pa_prefill_varlen(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                            int32_t max_blocks_per_seq, const int32_t* cu_seqlens_q,
                            const int32_t* cu_seqlens_k, int32_t batch, int32_t num_heads,
                            int32_t total_q, int32_t max_q_len, float scale, void* out,
                            void* stream) {
  return prefill_common(q, cache, block_tables, max_blocks_per_seq, cu_seqlens_q, cu_seqlens_k,
                        batch, num_heads, total_q, max_q_len, scale, 0, 0, out, stream);
}

pa_status pa_prefill_window(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                            int32_t max_blocks_per_seq, const int32_t* cu_seqlens_q,
                            const int32_t* cu_seqlens_k, int32_t batch, int32_t num_heads,
                            int32_t total_q, int32_t max_q_len, float scale, int32_t window,
                            int32_t sinks, void* out, void* stream) {
  const pa_status st = check_cache(cache);
  if (st != PA_OK) return st;
  if (window < 1 || sinks < 0) return PA_ERR_SHAPE;
  return prefill_common(q, cache, block_tables, max_blocks_per_seq, cu_seqlens_q, cu_seqlens_k,
                        batch, num_heads, total_q, max_q_len, scale, window, sinks, out, stream);
}

size_t pa_decode_shared_workspace_size(const pa_kv_cache* cache, int32_t batch, int32_t num_heads,
                                       int32_t max_blocks_per_seq, int32_t num_groups,
                                       int32_t max_context_len) {
  if (check_cache(cache) != PA_OK || batch <= 0 || batch > pa::kMaxPersistentBatch ||
      max_blocks_per_seq <= 0 || num_groups < 0 || num_groups > pa::kMaxPersistentBatch ||
      num_heads <= 0 || num_heads % cache->num_kv_heads != 0 || num_heads / cache->num_kv_heads > 8)
    return 0;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev) != PA_OK) return 0;
  const int cap = decode_len_cap(cache, max_blocks_per_seq, max_context_len);
  return decode_shared_bytes(cache, batch, num_heads, cap, num_groups, dev->num_sms);
}

pa_status pa_decode_shared(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* context_lens,
                           int32_t max_context_len, const int32_t* cu_groups,
                           const int32_t* prefix_lens, int32_t num_groups, int32_t always,
                           int32_t batch, int32_t num_heads, float scale, void* out, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const pa_status st = check_cache(cache);
  if (st != PA_OK) return st;
  if (num_groups < 0 || !(scale > 0.f)) return PA_ERR_SHAPE;
  if (batch > 0 && num_groups > 0 && (cu_groups == nullptr || prefix_lens == nullptr))
    return PA_ERR_NULL;
  if (batch > pa::kMaxPersistentBatch || num_groups > pa::kMaxPersistentBatch)
    return PA_ERR_UNSUPPORTED;
  // Sharing costs three more launches and spares at most this many bytes of K and V:
  // the host has a bound of the lengths, not the prefixes, and takes the whole of it
  // for shared. Where that is about so (64 own keys), shared / unshared us on one
  // GB300, from graphs, 8 kv heads of 128: bf16, 4 query heads each, 8 sequences
  // behind 8192 keys (237 MB) 33 / 32 and 12288 (354 MB) 35 / 40, 16 behind 4096 (256
  // MB) 31 / 28 and 6144 (381 MB) 32 / 36, 64 behind 1024 (281 MB) 33 / 28 and 1536
  // (413 MB) 34 / 36; 8 query heads each, 8 behind 8192 37 / 43, 64 behind 1024 37 / 32;
  // kv heads of 64, 8 behind 16384 (236 MB) 30 / 39. 8-bit codes, 8 query heads: 8 behind
  // 2048 (30 MB) 32 / 35, 16 behind 1024 (33 MB) 29 / 30, 64 behind 512 (74 MB) 36 / 32; 4
  // query heads: 26 / 23, 25 / 21, 24 / 25. So the sides cross at 200-400 MB (bf16) and 30-80
  // MB (8 bits) by shape, and the thresholds miss by up to 5 us there. Short prefixes of
  // long contexts are taken for shared: 64 sequences, bf16, 16 keys shared and 4096 own
  // 173 / 161, 2048 and 2048 110 / 88.
  const double saved = static_cast<double>(std::max(0, batch - num_groups)) * 2.0 *
                       decode_len_cap(cache, std::max(max_blocks_per_seq, 0), max_context_len) *
                       cache->num_kv_heads * cache->head_dim * elem_bytes(cache);
  const bool pays = saved >= (cache->dtype == PA_KV_BF16 ? 240e6 : 28e6);
  const SharedCall shared{cu_groups, prefix_lens, num_groups, always != 0 || pays, false,
                          workspace, workspace_bytes};
  return decode_common(q, cache, block_tables, max_blocks_per_seq, context_lens, max_context_len,
                       batch, num_heads, scale, out, workspace, workspace_bytes, stream, nullptr,
                       nullptr, nullptr, nullptr, 0, 0, nullptr,
                       num_groups > 0 ? &shared : nullptr);
}

size_t pa_prefill_shared_workspace_size(const pa_kv_cache* cache, int32_t num_heads,
                                        int32_t total_q, int32_t num_groups) {
  if (check_cache(cache) != PA_OK || cache->dtype != PA_KV_BF16 || cache->head_dim != 128 ||
      num_heads <= 0 || num_heads % cache->num_kv_heads != 0 ||
      num_heads / cache->num_kv_heads > 16 || total_q <= 0 || num_groups < 0 ||
      num_groups > pa::kMaxPersistentBatch)
    return 0;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev) != PA_OK) return 0;
  return pa::shared_workspace_bytes(0, total_q, num_heads, cache->num_kv_heads, 128, num_groups,
                                    dev->num_sms);
}

pa_status pa_prefill_shared(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                            int32_t max_blocks_per_seq, const int32_t* cu_seqlens_q,
                            const int32_t* cu_seqlens_k, const int32_t* cu_groups,
                            const int32_t* prefix_lens, int32_t num_groups, int32_t always,
                            int32_t batch, int32_t num_heads, int32_t total_q, int32_t max_q_len,
                            float scale, void* out, void* workspace, size_t workspace_bytes,
                            void* stream) {
  const pa_status st = check_cache(cache);
  if (st != PA_OK) return st;
  if (num_groups < 0) return PA_ERR_SHAPE;
  if (batch > 0 && num_groups > 0 && (cu_groups == nullptr || prefix_lens == nullptr))
    return PA_ERR_NULL;
  if (batch > pa::kMaxPersistentBatch || num_groups > pa::kMaxPersistentBatch)
    return PA_ERR_UNSUPPORTED;
  const SharedCall shared{cu_groups, prefix_lens, num_groups, true, always != 0, workspace,
                          workspace_bytes};
  const bool share = num_groups > 0;
  return prefill_common(q, cache, block_tables, max_blocks_per_seq, cu_seqlens_q, cu_seqlens_k,
                        batch, num_heads, total_q, max_q_len, scale, share ? kNoWindow : 0, 0, out,
                        stream, share ? &shared : nullptr);
}

pa_status pa_debug_inject_wait_timeout(int32_t skip_copy, uint64_t wait_limit_ns) {
  if (skip_copy < 0) {
    g_debug_skip_copy.store(-1);
    g_debug_wait_limit_ns.store(0);
    return PA_OK;
  }
  if (wait_limit_ns == 0 || wait_limit_ns > pa::kWaitLimitNs) return PA_ERR_SHAPE;
  g_debug_wait_limit_ns.store(wait_limit_ns);
  g_debug_skip_copy.store(skip_copy);
  return PA_OK;
}

pa_status pa_get_device_error(uint32_t* code) {
  if (code == nullptr) return PA_ERR_NULL;
  DeviceInfo* dev = nullptr;
  pa_status st = device_info(&dev);
  if (st != PA_OK) return st;
  if (cudaDeviceSynchronize() != cudaSuccess) return PA_ERR_CUDA;
  uint32_t v = 0;
  if (cudaMemcpy(&v, dev->err, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess) return PA_ERR_CUDA;
  const uint32_t zero = 0;
  if (cudaMemcpy(dev->err, &zero, sizeof zero, cudaMemcpyHostToDevice) != cudaSuccess)
    return PA_ERR_CUDA;
  *code = v;
  return PA_OK;
}

}  // extern "C"
