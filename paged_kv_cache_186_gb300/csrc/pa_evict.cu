// evict: cut sequences to a budget of keys per kv head by their scores, and
// move the kept rows to the front of the sequence's blocks.
//
// What is computed, for sequence b of L = min(context_len, bound) > budget keys
// and kv head g: kept = keys 0 .. sinks-1, keys L-recent .. L-1, and of the keys
// between them the budget - sinks - recent with the largest scores (equal
// scores: the lowest position; NaN above every number; -0 equals 0), in
// ascending order. Then row i of (b, g) - K, V, their scales, the score -
// becomes row kept[i]. A sequence of L <= budget keys is left as it is.
//
// How: two launches.
//   * select: one CTA per (sequence, kv head). Scores map to 32-bit integers of
//     the same order; three rounds of an 11-bit histogram (11 + 11 + 10 bits,
//     the third over the lowest ones) find the value T of the last key kept and
//     how many keys equal to T are. A pass over the positions in order then
//     writes the kept ones, placed by a CTA-wide prefix count.
//   * move: one CTA per (sequence, kv head, 128-byte column of K or of V), and
//     one per (sequence, kv head) for the scores and scales. Since kept ascends,
//     kept[j] >= j: writing rows [a, c) cannot touch a source of rows >= c, so a
//     CTA that reads a tile of rows, waits for its threads, writes the tile and
//     goes on to the next moves the rows in place without a copy.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_evict.h"

namespace pa {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

// A score as an unsigned integer of the same order: NaN highest, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum of v over the CTA's threads before this one; *total: over all.
__device__ __forceinline__ int cta_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(kAll, incl, o);
    if (lane >= o) incl += t;
  }
  __syncthreads();  // warp_sums of the call before are read
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int base = 0, sum = 0;
  for (int w = 0; w < kSelWarps; ++w) {
    if (w < warp) base += warp_sums[w];
    sum += warp_sums[w];
  }
  *total = sum;
  return base + incl - v;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictArgs a) {
  __shared__ int hist[kBins];
  __shared__ int warp_sums[kSelWarps];
  __shared__ int sel_bin, sel_above;
  grid_dependency_wait();
  const int b = blockIdx.x / a.num_kv_heads, kvh = blockIdx.x % a.num_kv_heads;
  const int L = min(max(a.context_lens[b], 0), a.len_cap);
  int32_t* const kept = a.kept + static_cast<long long>(blockIdx.x) * a.budget;
  if (kvh == 0 && threadIdx.x == 0) a.new_lens[b] = min(L, a.budget);
  if (L <= a.budget) {
    for (int i = threadIdx.x; i < a.budget; i += kSelThreads) kept[i] = i < L ? i : -1;
    return;
  }
  const int32_t* const table = a.block_tables + static_cast<long long>(b) * a.max_blocks;
  auto key_at = [&](int p) {
    const int phys = table[p / a.block_size];
    if (phys < 0 || phys >= a.num_blocks) {
      report_error(a.err, PA_DEVERR_BLOCK_RANGE);
      return order_key(0.f);
    }
    return order_key(
        a.scores[(static_cast<long long>(phys) * a.num_kv_heads + kvh) * a.block_size +
                 p % a.block_size]);
  };
  const int m0 = a.sinks, m1 = L - a.recent;      // keys chosen by score: [m0, m1)
  int want = a.budget - a.sinks - a.recent;       // how many of them (< m1 - m0)
  uint32_t prefix = 0u;                           // bits of T found so far
  int shift = 32;
  if (want > 0) {
    for (int round = 0; round < 3; ++round) {
      const int bits = round < 2 ? 11 : 10;
      const uint32_t known = shift == 32 ? 0u : ~0u << shift;
      shift -= bits;
      for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int p = m0 + threadIdx.x; p < m1; p += kSelThreads) {
        const uint32_t u = key_at(p);
        if ((u & known) == prefix) atomicAdd(&hist[(u >> shift) & ((1 << bits) - 1)], 1);
      }
      __syncthreads();
      // bin of the want-th largest: threads hold 4 bins each, highest first
      constexpr int PT = kBins / kSelThreads;
      int c[PT], sum = 0, total;
#pragma unroll
      for (int j = 0; j < PT; ++j) {
        c[j] = hist[kBins - 1 - (threadIdx.x * PT + j)];
        sum += c[j];
      }
      int above = cta_scan(sum, warp_sums, &total);
#pragma unroll
      for (int j = 0; j < PT; ++j) {
        if (above < want && above + c[j] >= want) {
          sel_bin = kBins - 1 - (threadIdx.x * PT + j);
          sel_above = above;
        }
        above += c[j];
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(sel_bin) << shift;
      want -= sel_above;
      __syncthreads();
    }
  }
  // keys above `prefix` (= T) are kept, and the first `want` equal to it
  const bool any = a.budget > a.sinks + a.recent;
  int out = 0, equal = 0;
  for (int p0 = 0; p0 < L; p0 += kSelThreads) {
    const int p = p0 + threadIdx.x;
    const bool mid = p >= m0 && p < m1;
    bool keep = p < L && !mid, tie = false;
    if (mid && any) {
      const uint32_t u = key_at(p);
      keep = u > prefix;
      tie = u == prefix;
    }
    int ties, n;
    const int rank = equal + cta_scan(tie, warp_sums, &ties);
    equal += ties;
    keep = keep || (tie && rank < want);
    const int at = out + cta_scan(keep, warp_sums, &n);
    out += n;
    if (keep && at < a.budget) kept[at] = p;
  }
}

// ---------------------------------------------------------------- move
constexpr int kMvThreads = 256;
constexpr int kMvVec = 8;  // 16-byte chunks in flight per thread

__global__ void __launch_bounds__(kMvThreads) move_kernel(const EvictArgs a) {
  const int cols = a.row_bytes / 128;     // 128-byte columns of a row
  const int parts = 2 * cols + 1;
  const int seg = blockIdx.x / parts, part = blockIdx.x % parts;
  const int b = seg / a.num_kv_heads, kvh = seg % a.num_kv_heads;
  if (min(max(a.context_lens[b], 0), a.len_cap) <= a.budget) return;
  const int32_t* const kept = a.kept + static_cast<long long>(seg) * a.budget;
  const int32_t* const table = a.block_tables + static_cast<long long>(b) * a.max_blocks;
  // pool block of logical position p; -1: outside the pool
  auto block_of = [&](int p) {
    const int phys = table[p / a.block_size];
    return phys >= 0 && phys < a.num_blocks ? phys : -1;
  };
  if (part < 2 * cols) {
    uint8_t* const base = static_cast<uint8_t*>(part < cols ? a.k_cache : a.v_cache) +
                          static_cast<long long>(kvh) * a.row_bytes + (part % cols) * 128;
    const long long stride = static_cast<long long>(a.num_kv_heads) * a.row_bytes;
    const int c = threadIdx.x & 7, r = threadIdx.x >> 3;  // 16-byte chunk, row of a group
    constexpr int RG = kMvThreads / 8;
    for (int t0 = 0; t0 < a.budget; t0 += RG * kMvVec) {
      uint4 x[kMvVec];
      long long to[kMvVec];
#pragma unroll
      for (int i = 0; i < kMvVec; ++i) {
        const int row = t0 + i * RG + r;
        to[i] = -1;
        if (row >= a.budget) continue;
        const int p = kept[row];
        if (p == row) continue;
        const long long sb = block_of(p), db = block_of(row);
        if (sb < 0 || db < 0) continue;
        to[i] = (db * a.block_size + row % a.block_size) * stride;
        x[i] = *reinterpret_cast<const uint4*>(
            base + (sb * a.block_size + p % a.block_size) * stride + c * 16);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kMvVec; ++i)
        if (to[i] >= 0) *reinterpret_cast<uint4*>(base + to[i] + c * 16) = x[i];
      __syncthreads();
    }
    return;
  }
  float* const arr[3] = {a.scores, a.k_scale, a.v_scale};
  const int n = a.k_scale != nullptr ? 3 : 1;
  for (int t0 = 0; t0 < a.budget; t0 += kMvThreads) {
    const int row = t0 + threadIdx.x;
    float x[3];
    long long to = -1;
    if (row < a.budget) {
      const int p = kept[row];
      const long long sb = block_of(p), db = block_of(row);
      if (p != row && sb >= 0 && db >= 0) {
        to = (db * a.num_kv_heads + kvh) * a.block_size + row % a.block_size;
        const long long from = (sb * a.num_kv_heads + kvh) * a.block_size + p % a.block_size;
        for (int i = 0; i < n; ++i) x[i] = arr[i][from];
      }
    }
    __syncthreads();
    if (to >= 0)
      for (int i = 0; i < n; ++i) arr[i][to] = x[i];
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const long long segs = static_cast<long long>(a.batch) * a.num_kv_heads;
  const long long parts = 2 * (a.row_bytes / 128) + 1;
  if (segs * parts > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(segs));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, select_kernel, a);
  if (e != cudaSuccess) return e;
  // A plain launch: it starts when new_lens is written and visible, so a decode
  // that follows, and reads the lengths before its own dependency wait, sees
  // them. The kept list is in place for the same reason.
  move_kernel<<<static_cast<unsigned>(segs * parts), kMvThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pa
