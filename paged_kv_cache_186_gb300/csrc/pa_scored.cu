// The second launch of pa_decode_scored: from the scores x (base-2 units) and
// every head's maximum m and 1 / sum r that the decode kernel left in the
// workspace,
//     scores[slot(b, p), g] += sum over query heads h of kv head g of
//                              2^(x[h, p] - m[h]) * r[h],   p < context_len[b].
//
// How: the scores lie in the decode's block order (block i of all (sequence,
// kv head) segments holds (group, block_size) floats), so a warp takes a
// contiguous run of blocks and goes through it segment by segment, 128 keys at
// a time: each lane four keys of one block, read as one 16-byte vector per
// query head, all heads' loads under way at once, summed in the order of the
// heads and added with two vector reductions. The adds are reductions, not
// read-modify-writes by the lane, so that sequences that share physical blocks
// (a common prefix) may add to them in one call; a slot of one sequence gets
// one add per call. Bound by the reads of the scores, 4 bytes per key and query
// head, and by memory as far as L2 does not hold them any more: on one GB300 (ncu,
// one pass) 8-9 us for the 17 MB of batch 64 (contexts 512-4096, 32/8 heads; none
// from memory), 15-17 us for 70 MB (8 contexts of 32768-131072; 11-15 MB from
// memory), 23-24 us for 122 MB (E4M3, 64/8 heads; 72 MB from memory).
#include <algorithm>

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kAsWarps = 8;
constexpr int kAsCtas = 4;  // per SM: all of them resident (at most 64 registers a thread)
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void red_add_v2(float* p, float x, float y) {
  asm volatile("red.relaxed.gpu.global.add.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(x), "f"(y)
               : "memory");
}

template <int BS, int GP>
__global__ void __launch_bounds__(kAsWarps * 32, kAsCtas) add_scores_kernel(const DecodeArgs a,
                                                                   float* scores) {
  constexpr int KB = 128 / BS;   // blocks of a warp's step
  constexpr int LPB = BS / 4;    // lanes per block
  // (no early start for the next launch: a decode's would bring its first tiles
  // into L2 over the scores that are still to be read here)
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int B = a.batch, Hkv = a.num_kv_heads, G = a.group;
  const int* const prefix = a.prefix_out;
  const long long N = static_cast<long long>(prefix[B]) * Hkv;
  const long long W = static_cast<long long>(gridDim.x) * kAsWarps;
  const long long w = static_cast<long long>(blockIdx.x) * kAsWarps + (threadIdx.x >> 5);
  const long long r0 = w * N / W, r1 = (w + 1) * N / W;  // the warp's blocks
  if (r0 >= r1) return;
  // last sequence whose blocks start at or before the warp's first one: 32
  // candidates a round
  int b = 0;
  {
    int lo = 0, hi = B;  // invariant: prefix[lo] * Hkv <= r0 < prefix[hi] * Hkv
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int at = min(lo + (lane + 1) * step, hi);
      const unsigned m = __ballot_sync(kAll, static_cast<long long>(prefix[at]) * Hkv <= r0);
      const int n = __popc(m);  // candidates at or before r0: the first n
      const int nlo = n == 0 ? lo : min(lo + n * step, hi);
      hi = min(lo + (n + 1) * step, hi);
      lo = nlo;
    }
    b = lo;
  }
  int nblk = prefix[b + 1] - prefix[b];
  const long long off = r0 - static_cast<long long>(prefix[b]) * Hkv;
  int kvh = static_cast<int>(off / nblk), blk0 = static_cast<int>(off % nblk);
  // a block's scores are whole lines (the workspace is only sure to be 16-byte aligned)
  const bool drop = ((reinterpret_cast<uintptr_t>(a.raw_scores) | (G * BS * 4)) & 127) == 0;
  // the lane's keys in its block: t0, t0 + 1, t0 + 8, t0 + 9
  const int s4 = lane % LPB, t0 = BS == 16 ? 2 * s4 : 16 * (s4 & 1) + 2 * (s4 >> 1);
  for (long long g = r0; g < r1;) {  // segment (b, kvh) from block blk0 on
    const int n = static_cast<int>(min(static_cast<long long>(nblk - blk0), r1 - g));
    const int L = min(max(a.context_lens[b], 0), a.len_cap);
    const int32_t* const table = a.block_tables + static_cast<long long>(b) * a.max_blocks + blk0;
    const float2* const ml = a.head_ml + static_cast<long long>(b) * a.num_heads + kvh * G;
    const float* const x0 = a.raw_scores + g * (G * BS) + 4 * s4;
    float2 c[GP];
#pragma unroll
    for (int h = 0; h < GP; ++h) c[h] = h < G ? __ldcg(ml + h) : make_float2(0.f, 0.f);
#pragma unroll 1
    for (int i = lane / LPB; i < n; i += KB) {
      const int phys = table[i];
      float4 v[GP];
#pragma unroll
      for (int h = 0; h < GP; ++h)
        v[h] = h < G ? __ldcs(reinterpret_cast<const float4*>(
                           x0 + static_cast<long long>(i) * (G * BS) + h * BS))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        sum.x += fast_exp2(v[h].x - c[h].x) * c[h].y;
        sum.y += fast_exp2(v[h].y - c[h].x) * c[h].y;
        sum.z += fast_exp2(v[h].z - c[h].x) * c[h].y;
        sum.w += fast_exp2(v[h].w - c[h].x) * c[h].y;
      }
      const int left = L - (blk0 + i) * BS - t0;  // the lane's keys below `left` exist
      if (phys >= 0 && phys < a.num_blocks) {  // (others: reported by the decode launch)
        float* const dst = scores + (static_cast<long long>(phys) * Hkv + kvh) * BS + t0;
        if (left >= 10) {
          red_add_v2(dst, sum.x, sum.y);
          red_add_v2(dst + 8, sum.z, sum.w);
        } else {
          if (left > 0) atomicAdd(dst, sum.x);
          if (left > 1) atomicAdd(dst + 1, sum.y);
          if (left > 8) atomicAdd(dst + 8, sum.z);
          if (left > 9) atomicAdd(dst + 9, sum.w);
        }
      }
      // the block's lanes have all used their scores: drop the lines from L2,
      // which would otherwise write them to memory some time; a line that is
      // shared with the next block only loses the priority it was stored with
      __syncwarp(((1u << LPB) - 1u) << (lane / LPB * LPB));
      const uintptr_t first = reinterpret_cast<uintptr_t>(a.raw_scores + (g + i) * (G * BS));
      for (uintptr_t line = (first & ~static_cast<uintptr_t>(127)) + s4 * 128;
           line < first + G * BS * 4; line += LPB * 128) {
        if (drop) asm volatile("discard.global.L2 [%0], 128;" ::"l"(line) : "memory");
        else asm volatile("applypriority.global.L2::evict_normal [%0], 128;" ::"l"(line) : "memory");
      }
    }
    g += n;
    blk0 = 0;
    if (g < r1 && ++kvh == Hkv) {
      kvh = 0;
      do {
        ++b;
      } while (prefix[b + 1] == prefix[b]);
      nblk = prefix[b + 1] - prefix[b];
    }
  }
}

template <int BS>
cudaError_t launch_bs(const cudaLaunchConfig_t& cfg, const DecodeArgs& a, float* scores) {
  if (a.group <= 1) return cudaLaunchKernelEx(&cfg, add_scores_kernel<BS, 1>, a, scores);
  if (a.group <= 2) return cudaLaunchKernelEx(&cfg, add_scores_kernel<BS, 2>, a, scores);
  if (a.group <= 4) return cudaLaunchKernelEx(&cfg, add_scores_kernel<BS, 4>, a, scores);
  return cudaLaunchKernelEx(&cfg, add_scores_kernel<BS, 8>, a, scores);
}

}  // namespace

cudaError_t launch_add_scores(const DecodeArgs& a, float* scores, int num_sms,
                              cudaStream_t stream) {
  const long long nblk = (static_cast<long long>(a.len_cap) + a.block_size - 1) / a.block_size;
  const long long steps = (nblk * a.batch * a.num_kv_heads * a.block_size + 127) / 128;
  const long long ctas = std::max(1LL, std::min<long long>((steps + kAsWarps - 1) / kAsWarps,
                                                           static_cast<long long>(num_sms) * kAsCtas));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kAsWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.block_size == 16 ? launch_bs<16>(cfg, a, scores) : launch_bs<32>(cfg, a, scores);
}

}  // namespace pa
