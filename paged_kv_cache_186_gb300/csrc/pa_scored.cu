// The second launch of pa_decode_scored: from the scores x (base-2 units) and
// every head's maximum m and 1 / sum r that the decode kernel left in the
// workspace,
//     scores[slot(b, p), g] += sum over query heads h of kv head g of
//                              2^(x[h, p] - m[h]) * r[h],   p < context_len[b].
//
// How: the scores lie in the decode's block order (block i of all (sequence,
// kv head) segments holds (group, block_size) floats), so a warp takes a
// contiguous run of blocks, 128 keys at a time: each lane four consecutive
// keys of one block, read as one 16-byte vector per query head, summed in the
// order of the heads and added with one vector reduction. The adds are
// reductions, not read-modify-writes by the lane, so that sequences that share
// physical blocks (a common prefix) may add to them in one call; a slot of one
// sequence gets one add per call.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kAsWarps = 8;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void red_add_v4(float* p, float4 v) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v.x),
               "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

template <int BS>
__global__ void __launch_bounds__(kAsWarps * 32) add_scores_kernel(const DecodeArgs a,
                                                                   float* scores) {
  constexpr int KB = 128 / BS;   // blocks of a warp's step
  constexpr int LPB = BS / 4;    // lanes per block
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int B = a.batch, Hkv = a.num_kv_heads, G = a.group;
  const int* const prefix = a.prefix_out;
  const long long N = static_cast<long long>(prefix[B]) * Hkv;
  const long long steps = (N + KB - 1) / KB;
  const long long W = static_cast<long long>(gridDim.x) * kAsWarps;
  const long long w = static_cast<long long>(blockIdx.x) * kAsWarps + (threadIdx.x >> 5);
  const long long s0 = w * steps / W, s1 = (w + 1) * steps / W;
  if (s0 >= s1) return;
  // last sequence whose blocks start at or before the warp's first one: 32
  // candidates a round
  int b = 0;
  {
    const long long g0 = s0 * KB;
    int lo = 0, hi = B;  // invariant: prefix[lo] * Hkv <= g0 < prefix[hi] * Hkv
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int at = min(lo + (lane + 1) * step, hi);
      const unsigned m = __ballot_sync(kAll, static_cast<long long>(prefix[at]) * Hkv <= g0);
      const int n = __popc(m);  // candidates at or before g0: the first n
      const int nlo = n == 0 ? lo : min(lo + n * step, hi);
      hi = min(lo + (n + 1) * step, hi);
      lo = nlo;
    }
    b = lo;
  }
  const int t4 = (lane % LPB) * 4;  // the lane's first key in its block
  for (long long s = s0; s < s1; ++s) {
    const long long g = s * KB + lane / LPB;
    if (g >= N) break;  // no warp-wide step below
    while (static_cast<long long>(prefix[b + 1]) * Hkv <= g) ++b;
    const int nblk = prefix[b + 1] - prefix[b];
    const long long off = g - static_cast<long long>(prefix[b]) * Hkv;
    const int kvh = static_cast<int>(off / nblk), blk = static_cast<int>(off % nblk);
    const int left = min(max(a.context_lens[b], 0), a.len_cap) - blk * BS - t4;
    if (left <= 0) continue;
    const int phys = a.block_tables[static_cast<long long>(b) * a.max_blocks + blk];
    if (phys < 0 || phys >= a.num_blocks) continue;  // reported by the decode launch
    const float* x = a.raw_scores + g * (G * BS) + t4;
    const float2* ml = a.head_ml + static_cast<long long>(b) * a.num_heads + kvh * G;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int h = 0; h < G; ++h) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(x + h * BS));
      const float2 c = __ldcg(ml + h);
      sum.x += fast_exp2(v.x - c.x) * c.y;
      sum.y += fast_exp2(v.y - c.x) * c.y;
      sum.z += fast_exp2(v.z - c.x) * c.y;
      sum.w += fast_exp2(v.w - c.x) * c.y;
    }
    float* dst = scores + (static_cast<long long>(phys) * Hkv + kvh) * BS + t4;
    if (left >= 4) {
      red_add_v4(dst, sum);
    } else {
      atomicAdd(dst, sum.x);
      if (left > 1) atomicAdd(dst + 1, sum.y);
      if (left > 2) atomicAdd(dst + 2, sum.z);
    }
  }
}

}  // namespace

cudaError_t launch_add_scores(const DecodeArgs& a, float* scores, int num_sms,
                              cudaStream_t stream) {
  const long long nblk = (static_cast<long long>(a.len_cap) + a.block_size - 1) / a.block_size;
  const long long steps = (nblk * a.batch * a.num_kv_heads * a.block_size + 127) / 128;
  const long long ctas = std::max(1LL, std::min<long long>((steps + kAsWarps - 1) / kAsWarps,
                                                           static_cast<long long>(num_sms) * 8));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kAsWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.block_size == 16 ? cudaLaunchKernelEx(&cfg, add_scores_kernel<16>, a, scores)
                            : cudaLaunchKernelEx(&cfg, add_scores_kernel<32>, a, scores);
}

}  // namespace pa
