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
//   * select: a cluster of 1 to 8 CTAs per (sequence, kv head), each with a
//     contiguous share of the positions. Scores map to 32-bit integers of the
//     same order, read once into shared memory. The value T of the last key kept
//     is found digit by digit (11 + 7 + 7 + 7 bits from the top): a histogram of
//     the digit over the keys that match the digits found so far, counted in
//     shared memory and summed over the cluster through distributed shared
//     memory. The first digit's bin holds a few percent of the keys (its 11 bits
//     are sign, exponent and two mantissa bits): one pass over the keys then
//     counts those above it and lists those in it, and the other digits are
//     found on the lists. Every warp counts its positions' keys above and equal
//     to T, and writes its kept positions behind those of the warps and CTAs
//     before it: three passes over the keys in all.
//   * move: one CTA per (sequence, kv head, 128-byte column of K or of V), and
//     one per (sequence, kv head) for the scores and scales. Since kept ascends,
//     kept[j] >= j: writing rows [a, c) cannot touch a source of rows >= c, so a
//     CTA that has read a tile of rows may write it while later tiles are still
//     on their way, and moves the rows in place without a copy: a ring of tiles
//     in shared memory filled by 16-byte asynchronous copies, with the pool rows
//     of source and destination in a second ring, looked up two tiles ahead by
//     one thread per row.
// On one GB300, first calls on inputs that L2 does not hold (ncu, one pass): 64
// sequences of 2176 keys to 2048 (8 heads, E4M3) 14 us of selection and 94 us of
// moving 536 MB (HBM-bound, 5.7 TB/s); 8 contexts of 32768-131072 keys to 4096 (8
// heads, bf16) 46 and 52 us, the selection bound by the latency of its three
// passes over 4.4 M keys and of the cluster's barriers. 8 short segments 9 and 8
// us: two launches, since a sequence's scores and scales and all columns of K and
// V move in parallel CTAs, which can start only when its selection is complete.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_evict.h"

namespace pa {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kBins0 = 2048;  // bins of the first digit's histogram
constexpr int kBins = 128;    // of the others'
constexpr int kDigits = 3;    // digits after the first
constexpr int kListed = 2048; // keys a CTA can list
constexpr int kMaxCluster = 8;
// Keys a CTA of select holds in shared memory (36 KB: four CTAs to an SM); keys
// past them are read again, through L2, in every pass.
constexpr int kMaxHeld = 9 * 1024;

// A score as an unsigned integer of the same order. Adding +0 makes -0 a +0 and
// any NaN the canonical one (positive, all mantissa bits set: the largest).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.f));
  return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();  // the aligned forms want whole warps
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
// This CTA's shared-memory address `p` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(uint32_t p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(p), "r"(rank));
  return r;
}
__device__ __forceinline__ int4 peer_load4(uint32_t a) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ int2 peer_load2(uint32_t a) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

template <int NT>
__global__ void __launch_bounds__(NT, 4) select_kernel(const EvictArgs a, int held_max) {
  constexpr int NW = NT / 32;
  constexpr int CAP = kListed / NW;  // keys a warp can list
  extern __shared__ __align__(16) uint32_t held[];  // order keys of the CTA's first positions
  __shared__ __align__(16) int hist0[kBins0];
  __shared__ __align__(16) int hist[kDigits][kBins];
  __shared__ __align__(16) int total[kDigits][kBins];  // hist summed over the cluster
  __shared__ uint32_t listed[NW][CAP];
  __shared__ int nlisted[NW], seg_sum[NW];
  __shared__ int2 warp_counts[NW];
  __shared__ __align__(8) int2 cta_counts;
  __shared__ int sel[kDigits + 1][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int seg = blockIdx.x / C, b = seg / a.num_kv_heads, kvh = seg % a.num_kv_heads;
  for (int i = tid; i < kBins0; i += NT) hist0[i] = 0;
  for (int i = tid; i < kDigits * kBins; i += NT) (&hist[0][0])[i] = (&total[0][0])[i] = 0;
  if (tid < NW) nlisted[tid] = 0;
  if (tid <= kDigits) sel[tid][0] = sel[tid][1] = 0;
  grid_dependency_wait();
  grid_launch_dependents();  // move waits for this grid before it reads anything
  const int L = min(max(a.context_lens[b], 0), a.len_cap);
  int32_t* const kept = a.kept + static_cast<long long>(seg) * a.budget;
  if (kvh == 0 && rank == 0 && tid == 0) a.new_lens[b] = min(L, a.budget);
  if (L <= a.budget) {  // the same for the whole cluster
    for (int i = rank * NT + tid; i < a.budget; i += C * NT)
      kept[i] = i < L ? i : -1;
    return;
  }
  const int32_t* const table = a.block_tables + static_cast<long long>(b) * a.max_blocks;
  const int bs_shift = a.block_size == 16 ? 4 : 5;
  // Four keys from position p (a multiple of 4: within one block) as order keys.
  auto load4 = [&](int p) {
    const int phys = table[p >> bs_shift];
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (phys < 0 || phys >= a.num_blocks)
      report_error(a.err, PA_DEVERR_BLOCK_RANGE);
    else
      x = *reinterpret_cast<const float4*>(
          a.scores + (((static_cast<long long>(phys) * a.num_kv_heads + kvh) << bs_shift) +
                      (p & (a.block_size - 1))));
    return make_uint4(order_key(x.x), order_key(x.y), order_key(x.z), order_key(x.w));
  };
  // this CTA's positions [c0, c1); the first held_max of them are held
  const int share = ((L + C - 1) / C + 127) & ~127;
  const int c0 = min(rank * share, L), c1 = min(c0 + share, L);
  const int m0 = a.sinks, m1 = L - a.recent;  // keys chosen by score: [m0, m1)
  int want = a.budget - a.sinks - a.recent;   // how many of them (< m1 - m0)
  __syncthreads();  // histograms are zero
  uint32_t prefix = 0u;  // bits of T found so far
  const bool any = want > 0;
  // Warp w owns the CTA's positions [w0, w1), 128 at a time, four to a lane.
  const int wshare = ((c1 - c0 + NW - 1) / NW + 127) & ~127;
  const int w0 = min(c0 + warp * wshare, c1), w1 = min(w0 + wshare, c1);
  // A lane's four keys from position p on, and which of them (bit j: p + j) lie
  // in the middle.
  auto keys = [&](int p) {
    if (!any || p >= w1) return make_uint4(0u, 0u, 0u, 0u);
    return p - c0 < held_max ? *reinterpret_cast<const uint4*>(held + (p - c0)) : load4(p);
  };
  auto mid_bits = [&](int p) {
    const int lo = min(max(m0 - p, 0), 4), hi = min(max(min(m1, w1) - p, 0), 4);
    return hi > lo ? ((1u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
  };
  int nabove = 0;  // the lane's keys above the first digit's bin
  if (any) {
#pragma unroll 4
    for (int p0 = w0; p0 < w1; p0 += 128) {
      const int p = p0 + 4 * lane;
      if (p < w1) {
        const uint4 u = load4(p);
        if (p - c0 < held_max) *reinterpret_cast<uint4*>(held + (p - c0)) = u;
        const uint32_t m = mid_bits(p);
        if (m & 1u) atomicAdd(&hist0[u.x >> 21], 1);
        if (m & 2u) atomicAdd(&hist0[u.y >> 21], 1);
        if (m & 4u) atomicAdd(&hist0[u.z >> 21], 1);
        if (m & 8u) atomicAdd(&hist0[u.w >> 21], 1);
      }
    }
    if (C > 1) cluster_sync(); else __syncthreads();
    // the bin of the want-th largest: warps hold segments of the bins, highest
    // first, each lane PB of them summed over the cluster
    {
      constexpr int PB = kBins0 / NT;
      const int bin0 = kBins0 - PB * (tid + 1);
      int c[PB];
#pragma unroll
      for (int j = 0; j < PB; ++j) c[j] = 0;
      // four CTAs' loads under way at once, each CTA starting at another
      for (int r0 = 0; r0 < C; r0 += 4) {
#pragma unroll
        for (int j = 0; j < PB; j += 4) {
          int4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = make_int4(0, 0, 0, 0);
            if (r0 + i < C)
              v[i] = peer_load4(peer_addr(smem_addr(&hist0[bin0 + j]), (r0 + i + rank) & (C - 1)));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            c[PB - 1 - j] += v[i].x;
            c[PB - 2 - j] += v[i].y;
            c[PB - 3 - j] += v[i].z;
            c[PB - 4 - j] += v[i].w;
          }
        }
      }
      int sum = 0;
#pragma unroll
      for (int j = 0; j < PB; ++j) sum += c[j];
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) seg_sum[warp] = incl;
      __syncthreads();
      int above = __reduce_add_sync(kAll, lane < warp ? seg_sum[lane] : 0) + incl - sum;
#pragma unroll
      for (int j = 0; j < PB; ++j) {
        if (above < want && above + c[j] >= want) {
          sel[0][0] = kBins0 - 1 - (tid * PB + j);
          sel[0][1] = above;
        }
        above += c[j];
      }
      __syncthreads();
      prefix = static_cast<uint32_t>(sel[0][0]) << 21;
      want -= sel[0][1];
    }
    // the keys above the bin counted, those in it listed
    for (int p0 = w0; p0 < w1; p0 += 128) {
      const int p = p0 + 4 * lane;
      const uint4 q = keys(p);
      const uint32_t u[4] = {q.x, q.y, q.z, q.w}, m = mid_bits(p);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t d = (u[j] >> 21) - (prefix >> 21);  // 0: in the bin
        const bool mid = (m >> j) & 1u;
        nabove += mid && d != 0u && static_cast<int>(d) > 0 ? 1 : 0;
        if (mid && d == 0u) {
          const int at = atomicAdd(&nlisted[warp], 1);
          if (at < CAP) listed[warp][at] = u[j];
        }
      }
    }
    __syncwarp();
    const bool fits = nlisted[warp] <= CAP;  // else the warp goes over its positions again
    // Every key of this warp in the first digit's bin, to f.
    auto each_listed = [&](auto&& f) {
      if (fits) {
        const int n = nlisted[warp];
        for (int i = lane; i < n; i += 32) f(listed[warp][i]);
      } else {
        for (int p0 = w0; p0 < w1; p0 += 128) {
          const int p = p0 + 4 * lane;
          const uint4 q = keys(p);
          const uint32_t u[4] = {q.x, q.y, q.z, q.w}, m = mid_bits(p);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (((m >> j) & 1u) && (u[j] >> 21) == (prefix >> 21)) f(u[j]);
        }
      }
    };
#pragma unroll 1
    for (int round = 0; round < kDigits; ++round) {
      const int shift = 14 - 7 * round;
      int* const h = hist[round];
      each_listed([&](uint32_t u) {
        if (((u ^ prefix) >> (shift + 7)) == 0u) atomicAdd(&h[(u >> shift) & (kBins - 1)], 1);
      });
      if (C > 1) {  // one warp per CTA of the cluster adds its bins
        cluster_sync();
        if (warp < C) {
          const int4 v = peer_load4(peer_addr(smem_addr(&h[4 * lane]), warp));
          int* const s = total[round] + 4 * lane;
          if (v.x) atomicAdd(s, v.x);
          if (v.y) atomicAdd(s + 1, v.y);
          if (v.z) atomicAdd(s + 2, v.z);
          if (v.w) atomicAdd(s + 3, v.w);
        }
      }
      __syncthreads();
      if (warp == 0) {  // four bins a lane, highest first
        const int4 v = *reinterpret_cast<const int4*>((C > 1 ? total[round] : h) + kBins -
                                                      4 * (lane + 1));
        const int c[4] = {v.w, v.z, v.y, v.x};
        const int sum = v.x + v.y + v.z + v.w;
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(kAll, incl, o);
          if (lane >= o) incl += x;
        }
        int above = incl - sum;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (above < want && above + c[j] >= want) {
            sel[round + 1][0] = kBins - 1 - (lane * 4 + j);
            sel[round + 1][1] = above;
          }
          above += c[j];
        }
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(sel[round + 1][0]) << shift;
      want -= sel[round + 1][1];
    }
    // prefix is T: keys above it are kept, and the first `want` equal to it
    int nk = nabove, nt = 0;
    each_listed([&](uint32_t u) {
      nk += u > prefix ? 1 : 0;
      nt += u == prefix ? 1 : 0;
    });
    nk = __reduce_add_sync(kAll, nk);
    nt = __reduce_add_sync(kAll, nt);
    if (lane == 0) warp_counts[warp] = make_int2(nk, nt);
  } else if (lane == 0) {
    warp_counts[warp] = make_int2(0, 0);
  }
  // the positions outside the middle are kept as well
  if (lane == 0)
    warp_counts[warp].x += max(0, min(w1, m0) - w0) + max(0, w1 - max(w0, m1));
  __syncthreads();
  if (warp == 0) {
    const int2 s = lane < NW ? warp_counts[lane] : make_int2(0, 0);
    const int sx = __reduce_add_sync(kAll, s.x), sy = __reduce_add_sync(kAll, s.y);
    if (lane == 0) cta_counts = make_int2(sx, sy);
  }
  if (C > 1) cluster_sync(); else __syncthreads();
  // kept above T, and equal to T, before this warp: in the CTAs before (their
  // counts read by lanes 16..) and in the warps before
  int2 v = make_int2(0, 0);
  if (lane < warp) v = warp_counts[lane];
  if (lane >= 16 && lane - 16 < rank)
    v = peer_load2(peer_addr(smem_addr(&cta_counts), lane - 16));
  const int before = __reduce_add_sync(kAll, v.x);
  int ties = __reduce_add_sync(kAll, v.y);
  int out = before + min(ties, want);
  const unsigned lt = (1u << lane) - 1u;
  // sum over the lanes before this one, and over all, of a number of 0 to 4
  auto scan4 = [&](int n, int& all) {
    const unsigned b0 = __ballot_sync(kAll, n & 1), b1 = __ballot_sync(kAll, n & 2),
                   b2 = __ballot_sync(kAll, n & 4);
    all = __popc(b0) + 2 * __popc(b1) + 4 * __popc(b2);
    return __popc(b0 & lt) + 2 * __popc(b1 & lt) + 4 * __popc(b2 & lt);
  };
  for (int p0 = w0; p0 < w1; p0 += 128) {
    const int p = p0 + 4 * lane;
    const uint4 q = keys(p);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w}, m = mid_bits(p);
    const int in = min(max(w1 - p, 0), 4);
    uint32_t keep = ((1u << in) - 1u) & ~m, tie = 0u;  // bit j: position p + j
    if (any) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        keep |= u[j] > prefix ? m & (1u << j) : 0u;
        tie |= u[j] == prefix ? m & (1u << j) : 0u;
      }
    }
    if (__any_sync(kAll, tie != 0u)) {
      int n;
      int rank_of = ties + scan4(__popc(tie), n);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if ((tie >> j & 1u) && rank_of++ < want) keep |= 1u << j;
      }
      ties += n;
    }
    int n;
    int at = out + scan4(__popc(keep), n);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (keep >> j & 1u) {
        if (at < a.budget) kept[at] = p + j;
        ++at;
      }
    }
    out += n;
  }
  if (C > 1) cluster_sync();  // no CTA's shared memory goes while another reads it
}

// ---------------------------------------------------------------- move
constexpr int kMvThreads = 256;
constexpr int kMvRows = 128;                       // rows of a tile
constexpr int kMvStages = 4;
constexpr int kMvIndex = 8;                        // tiles of the index ring (> kMvStages)
constexpr int kMvVec = kMvRows * 8 / kMvThreads;   // 16-byte chunks per thread and tile
constexpr int kMvSmem = kMvStages * kMvRows * 128 + kMvIndex * kMvRows * 8;

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__global__ void __launch_bounds__(kMvThreads) move_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  grid_dependency_wait();
  const int cols = a.row_bytes / 128;     // 128-byte columns of a row
  const int parts = 2 * cols + 1;
  const int seg = blockIdx.x / parts, part = blockIdx.x % parts;
  const int b = seg / a.num_kv_heads, kvh = seg % a.num_kv_heads;
  const int L = min(max(a.context_lens[b], 0), a.len_cap);
  if (L <= a.budget) return;
  const int32_t* const kept = a.kept + static_cast<long long>(seg) * a.budget;
  const int32_t* const table = a.block_tables + static_cast<long long>(b) * a.max_blocks;
  const int bs_shift = a.block_size == 16 ? 4 : 5, bs_mask = a.block_size - 1;
  // A kept entry; -1 should scores that changed under select (a call on another
  // stream) have left no position of the sequence there.
  auto checked = [&](int p) { return p >= 0 && p < L ? p : -1; };
  auto in_pool = [&](int phys) {
    if (phys >= 0 && phys < a.num_blocks) return true;
    report_error(a.err, PA_DEVERR_BLOCK_RANGE);
    return false;
  };
  if (part < 2 * cols) {
    uint8_t* const base = static_cast<uint8_t*>(part < cols ? a.k_cache : a.v_cache) +
                          static_cast<long long>(kvh) * a.row_bytes + (part % cols) * 128 +
                          (threadIdx.x & 7) * 16;
    const long long stride = static_cast<long long>(a.num_kv_heads) * a.row_bytes;
    const uint32_t slot0 = smem_addr(ring) + threadIdx.x * 16;
    int2* const index = reinterpret_cast<int2*>(ring + kMvStages * kMvRows * 128);
    const int r = threadIdx.x >> 3;  // row of a group of kMvThreads / 8
    const int tiles = (a.budget + kMvRows - 1) / kMvRows;
    // Index of a tile: thread i < kMvRows looks up row i, one step (kept, then
    // the block table) per call, each a tile behind the other.
    const bool indexer = threadIdx.x < kMvRows;
    // (used only a step after they are read, so that no lookup is waited for)
    int p1 = -1, p2 = -1, sb = -1, db = -1;  // kept entries of two tiles, blocks of the second
    auto row_of = [&](int tile) { return tile * kMvRows + static_cast<int>(threadIdx.x); };
    auto read_kept = [&](int tile) {
      p1 = indexer && row_of(tile) < a.budget ? kept[row_of(tile)] : -1;
    };
    auto read_blocks = [&](int tile) {  // of the tile read_kept was last called for
      p2 = checked(p1);
      if (p2 > row_of(tile)) {
        sb = table[p2 >> bs_shift];
        db = table[row_of(tile) >> bs_shift];
      }
    };
    auto write_index = [&](int tile) {
      if (indexer)
        index[(tile % kMvIndex) * kMvRows + threadIdx.x] =
            p2 > row_of(tile) && in_pool(sb) && in_pool(db)
                ? make_int2((sb << bs_shift) + (p2 & bs_mask),
                            (db << bs_shift) + (row_of(tile) & bs_mask))
                : make_int2(-1, -1);
    };
    auto issue = [&](int tile) {
      const int2* ix = index + (tile % kMvIndex) * kMvRows + r;
#pragma unroll
      for (int i = 0; i < kMvVec; ++i) {
        const int src = ix[i * (kMvThreads / 8)].x;
        if (src >= 0)
          cp_async_16(slot0 + ((tile % kMvStages) * kMvVec + i) * (kMvThreads * 16),
                      base + src * stride);
      }
    };
    // the first tiles' indexes at once, the next one's lookups under way
    for (int t = 0; t < kMvStages; ++t) {
      read_kept(t);
      read_blocks(t);
      write_index(t);
    }
    read_kept(kMvStages);
    __syncthreads();
    for (int t = 0; t < kMvStages - 1; ++t) {
      if (t < tiles) issue(t);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    read_blocks(kMvStages);
    read_kept(kMvStages + 1);
    for (int t = 0; t < tiles; ++t) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kMvStages - 2) : "memory");
      // every thread's copies of tile t have been read from the cache, and the
      // index of tile t + kMvStages - 1 is written
      __syncthreads();
      const int2* ix = index + (t % kMvIndex) * kMvRows + r;
#pragma unroll
      for (int i = 0; i < kMvVec; ++i) {
        const int dst = ix[i * (kMvThreads / 8)].y;
        if (dst >= 0)
          *reinterpret_cast<uint4*>(base + dst * stride) = *reinterpret_cast<const uint4*>(
              ring + ((t % kMvStages) * kMvVec + i) * (kMvThreads * 16) + threadIdx.x * 16);
      }
      if (t + kMvStages - 1 < tiles) issue(t + kMvStages - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      write_index(t + kMvStages);
      read_blocks(t + kMvStages + 1);
      read_kept(t + kMvStages + 2);
    }
    return;
  }
  float* const arr[3] = {a.scores, a.k_scale, a.v_scale};
  const int n = a.k_scale != nullptr ? 3 : 1;
  constexpr int RT = 4;  // rows per thread and tile
  for (int t0 = 0; t0 < a.budget; t0 += kMvThreads * RT) {
    float x[RT][3];
    long long to[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int row = t0 + i * kMvThreads + threadIdx.x;
      to[i] = -1;
      if (row >= a.budget) continue;
      const int p = checked(kept[row]);
      if (p <= row) continue;
      const int sb = table[p >> bs_shift], db = table[row >> bs_shift];
      if (!in_pool(sb) || !in_pool(db)) continue;
      to[i] = ((static_cast<long long>(db) * a.num_kv_heads + kvh) << bs_shift) + (row & bs_mask);
      const long long from =
          ((static_cast<long long>(sb) * a.num_kv_heads + kvh) << bs_shift) + (p & bs_mask);
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (j < n) x[i][j] = arr[j][from];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i)
      if (to[i] >= 0)
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (j < n) arr[j][to[i]] = x[i][j];
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const long long segs = static_cast<long long>(a.batch) * a.num_kv_heads;
  const long long parts = 2 * (a.row_bytes / 128) + 1;
  // CTAs per (sequence, kv head): one per 8192 keys of the length bound. Whole
  // calls on restored inputs, CUDA events, one GB300: 8 long contexts (bound
  // 131072) with 8 / 4 / 2 / 1 CTAs a head 100 / 104 / 129 / 195 us; 64 sequences
  // of 2176 keys with 1 / 2 CTAs 106 / 119. The bound decides, the lengths are on
  // the device: the same 64 sequences with a bound of 131072 take 221 us.
  int C = 1;
  while (C < kMaxCluster && (a.len_cap + C - 1) / C > 8192) C *= 2;
  if (segs * std::max<long long>(parts, C) > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int share = ((a.len_cap + C - 1) / C + 127) / 128 * 128;
  const int held = std::min(share, kMaxHeld);
  // (the 8 long contexts with 256 threads a CTA: 117 us instead of 100)
  auto* const select = share <= 4096 ? select_kernel<256> : select_kernel<512>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(select_kernel<512>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxHeld * 4);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMvSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(segs * C));
  cfg.blockDim = dim3(share <= 4096 ? 256 : 512);
  cfg.dynamicSmemBytes = static_cast<size_t>(held) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, select, a, held);
  if (e != cudaSuccess) return e;
  // Every CTA of move waits for select to be complete and visible, and lets no
  // launch behind it start before its own end: a decode that follows, and reads
  // the lengths before its own dependency wait, sees new_lens.
  cfg.gridDim = dim3(static_cast<unsigned>(segs * parts));
  cfg.blockDim = dim3(kMvThreads);
  cfg.dynamicSmemBytes = kMvSmem;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, move_kernel, a);
}

}  // namespace pa
