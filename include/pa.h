/*
 * pa.h - C ABI of the GB300 (sm_103a) paged-KV-cache attention library.
 *
 * The operations, as the source pages define them:
 *   pa_store_kv        append new tokens' K/V to their cache slots
 *                      ("tiny-vllm part 05", section "Gathering K/V into a
 *                      batched buffer and scattering into blocks"; the
 *                      store_kvcache step of "Decode Phase Attention Forward
 *                      Pass", section 2).
 *   pa_decode          one query per sequence attending over exactly
 *                      context_len cached keys, read through the block table,
 *                      with GQA head grouping ("Decode Phase Attention Forward
 *                      Pass", sections 2-4 and the zero-padding caveat;
 *                      "Decode Phase" glossary, the q.K^T / softmax / sum-of-V
 *                      steps).
 *   pa_decode_window   pa_decode over a sliding window plus leading sink keys
 *                      ("Decode Phase" glossary, long-context bullets).
 *   pa_decode_append   pa_store_kv of each sequence's new token followed by
 *                      pa_decode, fused into one persistent kernel.
 *   pa_prefill_varlen  packed varlen prefill over a prefix already in the
 *                      paged cache, bottom-right-aligned causal mask
 *                      ("Prefill Forward Prefix Caching Explained", Facts 1-2
 *                      and the mask section).
 * Operators around them, for a decode loop over a bounded cache (the pages have
 * no counterpart beyond the glossary's sliding-window and sink bullets):
 *   pa_norm_rope_store per-head RMS norm of q and k, position rotation, and the
 *                      store of the new K/V rows (quantised for 8-bit caches).
 *   pa_prefill_window  pa_prefill_varlen over a sliding window plus leading
 *                      sink keys.
 *   pa_decode_scored   pa_decode that also adds every key's attention weight to
 *                      a score kept beside the cache.
 *   pa_evict           cut sequences to a budget of keys by those scores and
 *                      move the kept rows to the front.
 *
 * Conventions shared by every call
 *   - Every tensor pointer is a DEVICE pointer owned by the caller. The
 *     library never calls a device allocator: pa_decode's split-K scratch is
 *     passed in as `workspace` (pa_decode_noalloc uses a static buffer).
 *   - All calls are asynchronous on `stream` (a cudaStream_t passed as void*;
 *     NULL = the legacy default stream) and never synchronise the host.
 *     Decode launches may start while the previous launch of this library on
 *     the stream is finishing (programmatic dependent launch): they read
 *     context_lens and block_tables before waiting for it, and everything
 *     else after. No kernel of this library writes those two arrays, except
 *     pa_evict its new_lens: they are complete before its last launch ends,
 *     and that launch lets nothing behind it start before its end, so a decode
 *     may follow it. A caller's own kernel that writes them and lets its
 *     dependents start early must not directly precede a decode call.
 *   - Argument errors are returned before anything is launched. A launch
 *     failure returns PA_ERR_CUDA. Out-of-range indices found on the device
 *     (a slot beyond the pool, a wait that timed out) never fault: the access
 *     is skipped and a bit is set in a per-device error word, read with
 *     pa_get_device_error().
 *   - Layouts (row-major, contiguous):
 *       k_cache, v_cache  (num_blocks, block_size, num_kv_heads, head_dim)
 *                         bf16, FP8-E4M3 bytes (OCP "e4m3fn") or signed INT8
 *                         codes (the "Decode Phase" glossary names FP8 and
 *                         INT8 KV-cache quantisation);
 *       k_scale, v_scale  (num_blocks, num_kv_heads, block_size) fp32, 8-bit
 *                         caches only: element = code value * scale;
 *       block_tables      (batch, max_blocks_per_seq) int32, physical block
 *                         of logical block j of sequence b;
 *       slot              physical_block * block_size + offset (int64).
 *   - Head map (GQA/MQA): query head h reads kv head h / (num_heads /
 *     num_kv_heads), i.e. the repeat_interleave grouping of the decode page.
 *   - Supported: head_dim 64 or 128 (8-bit caches: 128), block_size 16 or 32,
 *     num_heads a multiple of num_kv_heads with at most 8 query heads per kv
 *     head. Anything else returns PA_ERR_UNSUPPORTED.
 */
#ifndef PA_GB300_H
#define PA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PA_ABI_VERSION 1

typedef enum {
  PA_OK = 0,
  PA_ERR_NULL = 1,        /* a required pointer is NULL */
  PA_ERR_SHAPE = 2,       /* a size is negative/zero where it must not be, or inconsistent */
  PA_ERR_DTYPE = 3,       /* cache dtype / scale pointers do not match */
  PA_ERR_UNSUPPORTED = 4, /* valid but not implemented (head_dim, block_size, group size) */
  PA_ERR_CUDA = 5,        /* a CUDA runtime/driver call or a launch failed */
  PA_ERR_WORKSPACE = 6,   /* workspace missing or smaller than pa_decode_workspace_size() */
  PA_ERR_ALIGN = 7,       /* a pointer is not 16-byte aligned */
  PA_ERR_TOO_LARGE = 8    /* pa_decode_noalloc: the shape needs more scratch than the
                             library's static buffer holds */
} pa_status;

typedef enum { PA_KV_BF16 = 0, PA_KV_FP8_E4M3 = 1, PA_KV_INT8 = 2 } pa_kv_dtype;

/* Device error word bits (pa_get_device_error). */
#define PA_DEVERR_SLOT_RANGE 0x1u   /* store_kv: slot >= num_blocks*block_size, skipped */
#define PA_DEVERR_WAIT_TIMEOUT 0x2u /* a kernel's bounded wait on a copy gave up */
#define PA_DEVERR_BLOCK_RANGE 0x4u  /* block table entry outside [0, num_blocks), zero-filled */
#define PA_DEVERR_POSITION_RANGE 0x8u /* norm_rope_store: position outside the table, skipped */

/* A paged KV cache (one layer). Pointers are device pointers; the struct
 * itself is read on the host during the call and may live on the stack. */
typedef struct {
  int32_t num_blocks;   /* physical blocks in the pool */
  int32_t block_size;   /* tokens per block: 16 or 32 */
  int32_t num_kv_heads;
  int32_t head_dim;     /* 64 or 128 */
  int32_t dtype;        /* pa_kv_dtype */
  void* k_cache;        /* (num_blocks, block_size, num_kv_heads, head_dim) */
  void* v_cache;
  float* k_scale;       /* (num_blocks, num_kv_heads, block_size), 8-bit only, else NULL */
  float* v_scale;
} pa_kv_cache;

/* ABI version of the loaded library (PA_ABI_VERSION it was built with). */
int32_t pa_abi_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char* pa_status_string(pa_status status);

/*
 * pa_store_kv - write num_tokens new K/V rows into the cache.
 *   k, v           (num_tokens, num_kv_heads, head_dim), cache dtype (bf16, or
 *                  E4M3 / INT8 bytes for an 8-bit cache), device.
 *   k_scale_new,   (num_tokens, num_kv_heads) fp32, 8-bit caches only (else NULL).
 *   v_scale_new
 *   slot_mapping   (num_tokens) int64: destination slot of token t; a negative
 *                  slot skips the token (padding). Slots within one call must
 *                  be distinct (otherwise which write wins is unspecified).
 *   Bytes are copied unchanged (bit-exact). A slot >= num_blocks*block_size is
 *   skipped and flagged PA_DEVERR_SLOT_RANGE. num_tokens == 0 is a no-op.
 */
pa_status pa_store_kv(const void* k, const void* v, const float* k_scale_new,
                      const float* v_scale_new, const int64_t* slot_mapping, int32_t num_tokens,
                      const pa_kv_cache* cache, void* stream);

/* Norm and rotation parameters of pa_norm_rope_store. Pointers are device
 * pointers; the struct itself is read on the host during the call. */
typedef struct {
  const void* q_weight;  /* (head_dim) bf16 norm weight of the query heads; NULL: no norm */
  const void* k_weight;  /* (head_dim) bf16 norm weight of the key heads; NULL: no norm */
  const float* cos_sin;  /* (max_positions, rotary_dim) fp32: rotary_dim/2 cosines, then the
                            sines; may be NULL when rotary_dim is 0 */
  int32_t max_positions;
  int32_t rotary_dim;    /* leading dims of a head that are rotated: 0, or a multiple of 16 up
                            to head_dim */
  int32_t interleaved;   /* pair i is dims (2i, 2i+1); 0: dims (i, i + rotary_dim/2) */
  float eps;             /* added to the mean square, >= 0 */
} pa_norm_rope;

/*
 * pa_norm_rope_store - what happens to a layer's new q, k and v between the
 * projection and the attention, in one launch: for every query and key head
 *   n(x) = x * rsqrt(mean(x^2) + eps) * weight      (where a weight is given)
 *   (a, b) -> (a cos - b sin, b cos + a sin)        (each pair of rotated dims)
 * in fp32, q rounded once to bf16 into q_out, k (and v as it is) stored in the
 * cache as by pa_store_kv.
 *   q               (num_tokens, num_heads, head_dim) bf16; token t starts
 *                   t * q_stride elements from q (a view of a fused projection's
 *                   output), the heads of a token are contiguous.
 *   k, v            (num_tokens, num_kv_heads, head_dim) bf16, likewise. Strides
 *                   are multiples of 8 elements and at least one token's heads
 *                   (PA_ERR_SHAPE).
 *   positions       (num_tokens) int64: row of cos_sin. A position outside
 *                   [0, max_positions) skips the token (q_out and cache left as
 *                   they were) and sets PA_DEVERR_POSITION_RANGE. May be NULL
 *                   when rotary_dim is 0.
 *   slot_mapping    (num_tokens) int64 as for pa_store_kv. A negative slot is a
 *                   padding token: nothing of it is written. A slot beyond the
 *                   pool is flagged PA_DEVERR_SLOT_RANGE and its K/V skipped.
 *   cache           bf16, or 8-bit: a row is stored as codes round(x / s) with
 *                   s = max|x| / 448 (E4M3) or / 127 (INT8), 1 for a row of
 *                   zeros, from the fp32 row, and s in k_scale / v_scale. A row
 *                   with a NaN or an infinity reads back as NaN.
 *   scores          NULL, or the (num_blocks, num_kv_heads, block_size) fp32
 *                   scores of pa_decode_scored: the stored slots' are set to 0.
 *   q_out           (num_tokens, num_heads, head_dim) bf16, contiguous. May be q
 *                   itself when q is contiguous (else it must not overlap it).
 */
pa_status pa_norm_rope_store(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, const pa_norm_rope* params,
                             const int64_t* positions, const int64_t* slot_mapping,
                             int32_t num_tokens, int32_t num_heads, const pa_kv_cache* cache,
                             float* scores, void* q_out, void* stream);

/*
 * pa_decode_workspace_size - bytes of device scratch pa_decode needs for this
 * shape (split-K partial results). 0 means pa_decode needs no workspace.
 * max_context_len is the same host-side bound that will be passed to
 * pa_decode (<= 0: the block-table capacity max_blocks_per_seq*block_size).
 */
size_t pa_decode_workspace_size(const pa_kv_cache* cache, int32_t batch, int32_t num_heads,
                                int32_t max_blocks_per_seq, int32_t max_context_len);

/*
 * pa_decode - single-query attention over a paged KV cache.
 *   q               (batch, num_heads, head_dim) bf16.
 *   block_tables    (batch, max_blocks_per_seq) int32; only the first
 *                   ceil(context_len/block_size) entries of a row are read.
 *   context_lens    (batch) int32 on the device: keys 0..context_len-1 of each
 *                   sequence are attended (the token stored this step
 *                   included). context_len 0 gives a zero output row.
 *   max_context_len host-side upper bound of every context_len (sizes the
 *                   split-K grid; <= 0 means max_blocks_per_seq*block_size).
 *                   Keys at positions >= this bound are not attended.
 *   scale           softmax scale applied to q.k.
 *   out             (batch, num_heads, head_dim) bf16.
 *   workspace       device scratch of at least pa_decode_workspace_size()
 *                   bytes (may be NULL when that is 0). Contents on entry are
 *                   ignored, up to a 2^-32 chance per stale 64-bit word of
 *                   carrying the call's tag; calls sharing one workspace must
 *                   not overlap.
 *                   The split-K arrival counters in it carry a per-call
 *                   32-bit tag (unrelated from call to call) and each is
 *                   cleared by its last arrival, so a CUDA graph
 *                   that captured the call can be replayed back to back on
 *                   the same workspace (its tag is frozen at capture). After
 *                   a launch that reported PA_DEVERR_WAIT_TIMEOUT, counters
 *                   of unfinished segments stay set: make one uncaptured call
 *                   on the workspace before replaying such a graph again.
 * Arithmetic: bf16 (or E4M3 / INT8 codes widened exactly to f16) operands, fp32 scores,
 * softmax and accumulation, one round to bf16 at the output.
 */
pa_status pa_decode(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                    int32_t max_blocks_per_seq, const int32_t* context_lens,
                    int32_t max_context_len, int32_t batch, int32_t num_heads, float scale,
                    void* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * pa_decode_window - pa_decode restricted to a sliding window with attention
 * sinks ("Decode Phase" glossary, the long-context bullets: sliding window
 * attention over the most recent W tokens; attention sinks as in
 * StreamingLLM, keeping the initial tokens). For a sequence of L =
 * context_len keys the query attends to keys p < sinks and p >= L - window.
 *   window   > 0: window size in keys; <= 0: all keys (same as pa_decode,
 *            sinks ignored).
 *   sinks    >= 0: leading keys always attended (PA_ERR_SHAPE if negative).
 *   other arguments as pa_decode (same workspace size). Blocks that hold no
 *   visible key are not read. Batches above 16384 return PA_ERR_UNSUPPORTED.
 */
pa_status pa_decode_window(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* context_lens,
                           int32_t max_context_len, int32_t batch, int32_t num_heads,
                           float scale, int32_t window, int32_t sinks, void* out, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * pa_decode_scored - pa_decode that also adds every key's softmax weight to a
 * score: for each sequence, kv head g and key position p < context_len,
 *   scores[slot(p), g] += sum over the query heads h of g of softmax_h(p)
 * (fp32). The scores of heavily attended keys grow from step to step; pa_evict
 * keeps the keys with the largest.
 *   scores    (num_blocks, num_kv_heads, block_size) fp32, as the 8-bit scales.
 *             Every visible slot gets one addition per call and sequence: scores
 *             of sequences that share blocks sum over the sequences (in an order
 *             that may change from call to call). Slots at or past context_len
 *             are left as they were. pa_norm_rope_store can set a new slot's
 *             score to zero. A query head whose scores hold a NaN or +infinity
 *             (its out is NaN) adds NaN to those keys' scores and nothing to
 *             the others'. After a launch that reported
 *             PA_DEVERR_WAIT_TIMEOUT they are as invalid as out.
 *   workspace at least pa_decode_scored_workspace_size() bytes (0: the shape is
 *             not supported), contract as for pa_decode. It holds the scores of
 *             every key: 4 bytes per query head and key of the bound batch *
 *             max_context_len, which can be as large as the cache. A tight
 *             max_context_len keeps it small; without one it goes by the width
 *             of the block table.
 *   other arguments as pa_decode; out equals pa_decode's bit for bit. Batches
 *   above 16384 return PA_ERR_UNSUPPORTED.
 */
size_t pa_decode_scored_workspace_size(const pa_kv_cache* cache, int32_t batch, int32_t num_heads,
                                       int32_t max_blocks_per_seq, int32_t max_context_len);
pa_status pa_decode_scored(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* context_lens,
                           int32_t max_context_len, int32_t batch, int32_t num_heads, float scale,
                           float* scores, void* out, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * pa_evict - cut sequences to `budget` keys per kv head. For a sequence of
 * L = min(context_len, bound) > budget keys (bound: max_context_len or the
 * block-table capacity), every kv head keeps the keys p < sinks, the keys
 * p >= L - recent, and of the others the budget - sinks - recent with the
 * largest scores (equal scores: the lowest p; a NaN counts as the largest).
 * The kept rows of K, V, their scales and scores move, in order, to positions
 * 0 .. budget-1 of the sequence's blocks; rows from budget on are left as they
 * were, and the caller may free the blocks past them. A sequence of at most
 * budget keys is left as it is.
 *   scores         (num_blocks, num_kv_heads, block_size) fp32, moved like K.
 *   budget         >= 1; sinks, recent >= 0, sinks + recent <= budget
 *                  (else PA_ERR_SHAPE).
 *   kept           (batch, num_kv_heads, budget) int32 out: the positions the
 *                  rows came from, ascending; 0 .. L-1 and then -1 for a
 *                  sequence left as it is.
 *   max_context_len as pa_decode. It also chooses how many CTAs share the
 *                  selection of a (sequence, kv head): without a bound close to
 *                  the longest sequence, short ones under a wide block table
 *                  are selected from by too many (twice the time of a call).
 *   new_lens       (batch) int32 out: min(L, budget). Not context_lens itself
 *                  (PA_ERR_SHAPE): the lengths are read by several CTAs.
 * Keys carry their rotation, and attention does not depend on the order of the
 * keys, so decode calls over new_lens attend to exactly the kept keys; a later
 * token's position (for the rotation) is the caller's to keep counting. The
 * blocks of a cut sequence must be distinct and not shared with another
 * sequence, and no other call may read or write them (or their scores) at the
 * same time. Length bounds and budgets above 2^30 return PA_ERR_UNSUPPORTED. A physical
 * block id out of range sets PA_DEVERR_BLOCK_RANGE; scores there count as 0 and
 * rows there are not moved.
 */
pa_status pa_evict(const pa_kv_cache* cache, float* scores, const int32_t* block_tables,
                   int32_t max_blocks_per_seq, const int32_t* context_lens,
                   int32_t max_context_len, int32_t batch, int32_t budget, int32_t sinks,
                   int32_t recent, int32_t* kept, int32_t* new_lens, void* stream);

/*
 * pa_decode_append - one decode step's store and attention in one call: the
 * store_kvcache step (each sequence's new K/V row written to the cache) then
 * attention over context_len keys, new token included ("Decode Phase
 * Attention Forward Pass", section 2, the store-then-attend order).
 *   k_new, v_new    (batch, num_kv_heads, head_dim), cache dtype, device,
 *                   16-byte aligned: the new token of sequence b.
 *   k_scale_new,    (batch, num_kv_heads) fp32, 8-bit caches only (else NULL).
 *   v_scale_new
 *   other arguments as pa_decode (same workspace size).
 * The row goes to position p = min(context_len, bound) - 1 of its sequence,
 * i.e. slot block_tables[b][p / block_size] * block_size + p % block_size,
 * where bound is max_context_len (or the block-table capacity); a sequence
 * with context_len 0 appends nothing. Result and cache contents are those of
 * pa_store_kv with that slot mapping followed by pa_decode. The block holding
 * position p must not be read by another sequence of the same call. A
 * physical block id out of range skips the write and sets
 * PA_DEVERR_BLOCK_RANGE. With the persistent kernel (batch <= 16384) the warp
 * that attends to a sequence's last block also writes the row; larger batches
 * use a separate store launch first.
 */
pa_status pa_decode_append(const void* q, const void* k_new, const void* v_new,
                           const float* k_scale_new, const float* v_scale_new,
                           const pa_kv_cache* cache, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* context_lens,
                           int32_t max_context_len, int32_t batch, int32_t num_heads,
                           float scale, void* out, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * pa_decode_window_append - pa_decode_append with the sliding window and
 * attention sinks of pa_decode_window: the new row is written as by
 * pa_decode_append, then each query attends to the keys pa_decode_window
 * selects (the new token, at position context_len - 1, is always among them).
 * Result and cache contents are those of pa_store_kv followed by
 * pa_decode_window; window 0 is pa_decode_append. Same arguments as
 * pa_decode_append plus window and sinks (as pa_decode_window); batches above
 * 16384 return PA_ERR_UNSUPPORTED, as for pa_decode_window.
 */
pa_status pa_decode_window_append(const void* q, const void* k_new, const void* v_new,
                                  const float* k_scale_new, const float* v_scale_new,
                                  const pa_kv_cache* cache, const int32_t* block_tables,
                                  int32_t max_blocks_per_seq, const int32_t* context_lens,
                                  int32_t max_context_len, int32_t batch, int32_t num_heads,
                                  float scale, int32_t window, int32_t sinks, void* out,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * pa_prefill_varlen - prefill attention of packed new tokens over their
 * sequences' paged K/V (cached prefix + the new tokens, which must already be
 * stored with pa_store_kv), with the bottom-right-aligned causal mask: query
 * row i of a sequence (0-based) sees keys j <= i + (kv_len - q_len).
 *   q               (total_q, num_heads, head_dim) bf16, sequences packed.
 *   block_tables    (batch, max_blocks_per_seq) int32.
 *   cu_seqlens_q    (batch+1) int32 on the device, prefix sums of q_len
 *                   (cu_seqlens_q[0] = 0, cu_seqlens_q[batch] = total_q).
 *   cu_seqlens_k    (batch+1) int32 on the device, prefix sums of kv_len.
 *   total_q         packed rows of q/out (host-side).
 *   max_q_len       host-side bound of every q_len (sizes the grid; <= 0 means
 *                   total_q). Of a sequence longer than the bound some rows are
 *                   not computed.
 *   scale           softmax scale, > 0.
 *   out             (total_q, num_heads, head_dim) bf16.
 * A sequence with q_len > kv_len is invalid input: its cached length is taken
 * as 0 and keys are clamped to kv_len. Supported: bf16 cache, head_dim 128,
 * block_size 16 or 32, num_heads/num_kv_heads in {1, 2, 4, 8, 16}.
 * Arithmetic: bf16 operands on the tensor cores, fp32 scores and
 * accumulation, probabilities rounded to bf16 for P.V (as two bf16 terms,
 * bf16(p) + bf16(p - bf16(p)), on the first 128 keys of the query tiles that
 * hold rows seeing fewer than 128 keys), bf16 output. V of every key of a
 * sequence must be finite: a row that does not see a key may give it the weight
 * 0.
 */
pa_status pa_prefill_varlen(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                            int32_t max_blocks_per_seq, const int32_t* cu_seqlens_q,
                            const int32_t* cu_seqlens_k, int32_t batch, int32_t num_heads,
                            int32_t total_q, int32_t max_q_len, float scale, void* out,
                            void* stream);

/*
 * pa_prefill_window - pa_prefill_varlen over a sliding window with attention
 * sinks: query row i, at position p = i + (kv_len - q_len), sees the keys
 * j <= p with j < sinks or j > p - window.
 *   window   >= 1 (PA_ERR_SHAPE otherwise); a window of kv_len keys or more is
 *            pa_prefill_varlen's mask.
 *   sinks    >= 0 (PA_ERR_SHAPE if negative).
 *   max_q_len also chooses the kernel: with a bound of 128 / (heads a kv head)
 *            tokens or fewer, both halves of a CTA share its one query tile.
 *   other arguments, support (bf16 caches, head_dim 128; 8-bit caches return
 *   PA_ERR_UNSUPPORTED) and arithmetic as pa_prefill_varlen, with P as two
 *   bf16 terms also on the first 128-key tile (the sinks') where sinks > 0, and
 *   on every tile where window + sinks < 128.
 * Blocks that hold no key visible to a 128-row query tile pair are not read, nor
 * their table entries, so the blocks of keys no row of the call sees may have
 * been freed. K and V there, and in keys of a partly visible block that no row
 * of the pair sees, may hold anything. V of a key that some row of a pair sees
 * must be finite: a row that does not see it gives it the weight 0.
 */
pa_status pa_prefill_window(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                            int32_t max_blocks_per_seq, const int32_t* cu_seqlens_q,
                            const int32_t* cu_seqlens_k, int32_t batch, int32_t num_heads,
                            int32_t total_q, int32_t max_q_len, float scale, int32_t window,
                            int32_t sinks, void* out, void* stream);

/*
 * pa_decode_noalloc - pa_decode for callers that cannot allocate device memory.
 * The pages have no counterpart: this entry point exists for callers with no
 * device allocator of their own (a plain C host program handed device
 * pointers by another runtime) or whose device memory is fully reserved (a
 * serving engine's KV-block pool), for whom a scratch cudaMalloc is not an
 * option. Same arguments and result as pa_decode, minus the workspace: the
 * split-K scratch is a static device buffer of
 * PA_DECODE_NOALLOC_SCRATCH_BYTES inside the library, held by every GPU that
 * loads it until the process exits. Allocates nothing per call (no cudaMalloc,
 * cudaFree or allocating library routine).
 *   - Shapes whose pa_decode_workspace_size() exceeds the buffer are rejected
 *     with PA_ERR_TOO_LARGE before anything is launched.
 *   - The first call on a device (with it current) looks up the buffer's
 *     device address; make that first call before any stream capture.
 *   - All calls share the buffer and it keeps the last call's contents (the
 *     kernels write every partial they read, so nothing needs clearing). Calls
 *     that may overlap on the GPU race on it: serialise them.
 */
#define PA_DECODE_NOALLOC_SCRATCH_BYTES (32u << 20) /* 32 MiB */
pa_status pa_decode_noalloc(const void* q, const pa_kv_cache* cache, const int32_t* block_tables,
                            int32_t max_blocks_per_seq, const int32_t* context_lens,
                            int32_t max_context_len, int32_t batch, int32_t num_heads,
                            float scale, void* out, void* stream);

/*
 * pa_get_device_error - synchronise the current device, return its error word
 * (PA_DEVERR_* bits, 0 if none) in *code and clear it.
 */
pa_status pa_get_device_error(uint32_t* code);

/*
 * pa_debug_inject_wait_timeout - test hook for the failure-detection path; the
 * pages have no counterpart. Every wait of a decode kernel on a copy is
 * bounded (2 s by default); after the bound it records PA_DEVERR_WAIT_TIMEOUT,
 * lets the copies it has in flight land (each wait bounded again) and returns,
 * so the context stays usable. This hook makes that happen on purpose without
 * faulting anything: while armed (skip_copy >= 0), decode launches of this
 * process (persistent kernel, batch <= 16384; pa_decode, pa_decode_window,
 * pa_decode_append) wait at most wait_limit_ns (1 .. 2e9) per copy, and in
 * each launch the first warp of the first CTA never issues its skip_copy-th
 * block copy (counted from 0 in its own block order), so its wait for that
 * block runs out. Outputs of such a launch are invalid. skip_copy < 0
 * disarms the hook and restores the 2 s bound (wait_limit_ns ignored).
 * Process-wide, not thread-safe against concurrent decode calls: arm, run
 * one call, disarm. Returns PA_ERR_SHAPE for a bound outside 1 .. 2e9.
 */
pa_status pa_debug_inject_wait_timeout(int32_t skip_copy, uint64_t wait_limit_ns);

#ifdef __cplusplus
}
#endif

#endif /* PA_GB300_H */
