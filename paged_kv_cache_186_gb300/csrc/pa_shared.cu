// Attention of groups of sequences that share their first keys.
//
// What is computed: for row t (a sequence's query) and head h, with the keys
// p < vis(t) that the row sees,
//     out[t,h] = sum_p softmax_p(scale * q[t,h] . K[p]) V[p].
// The rows of a group share the keys p < P (whole blocks, one copy in the
// cache). A softmax over a union of key sets is an exact merge of the sets'
// (max m, sum l, unnormalised o): with M = max_j m_j
//     out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j    (scores in base 2)
// so the shared keys are attended to once for all rows of the group, as a dense
// product of 128-row query tiles with 128-key tiles, and every sequence's own
// keys p >= P by the decode or prefill kernel, which here leave (m, l, o) too.
//
// Four launches:
//   plan    (one CTA) the groups' shared keys, rows, segments and work units.
//   own     pa_decode.cu / pa_prefill.cu over the keys from P on.
//   shared  below: persistent CTAs over the units of all segments.
//   merge   below: each row's parts and its own keys' result -> bf16.
//
// The shared launch. A segment is one kv head of one group and up to row_tiles
// tiles of 128 rows (128/G tokens x the G query heads of the kv head); a unit is
// one 128-key tile of it. Every CTA takes an equal run of units, so one long
// prefix is spread over all SMs and short ones are not, and leaves one partial
// per segment it meets. The CTA is organised as the prefill kernel: K, V and Q
// arrive by TMA through their own rings (warps 8, 10, 11), warp 9 issues the
// tcgen05 MMAs, two softmax warpgroups own one TMEM lane (row) a thread. With
// two row tiles each warpgroup has its own (a K/V tile serves 256 rows); with
// one, both take its key tiles in turn and merge at the end of the segment.
// P goes into P.V as two bf16 terms, bf16(p) and bf16(p - bf16(p)): rounded
// once, a row whose weight lies on few keys misses the library's tolerance
// (1.28e-2 measured on rows with four dominant keys), and shared prompts begin
// with such keys.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_launch.h"
#include "pa_shared.h"
#include "pa_tcgen05.cuh"

namespace pa {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBM = 128;  // rows per query tile
constexpr int kBN = 128;  // keys per tile
constexpr int kSub = 128 * kBM;  // bytes of a 64-dim (128-byte-wide) column of a 128-row tile

// ============================================================ plan
constexpr int kPlanThreads = 1024;

// Inclusive scan of one value per thread of the CTA (op associative).
template <typename T, typename Op>
__device__ __forceinline__ T block_scan(T v, T* warp_part, Op op) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v = op(v, t);
  }
  if (lane == 31) warp_part[warp] = v;
  __syncthreads();
  if (warp == 0) {
    T w = warp_part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T t = __shfl_up_sync(kFull, w, o);
      if (lane >= o) w = op(w, t);
    }
    warp_part[lane] = w;
  }
  __syncthreads();
  if (warp > 0) v = op(v, warp_part[warp - 1]);
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedArgs a) {
  __shared__ long long part[32];
  // everything this launch writes may still be read by the call before it
  grid_dependency_wait();
  grid_launch_dependents();
  const SharedPlan& p = a.plan;
  const int G = a.num_groups, B = a.batch, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const bool decode = a.context_lens != nullptr;
  auto kv_len = [&](int b) {
    return decode ? min(max(a.context_lens[b], 0), a.len_cap)
                  : min(max(a.cu_k[b + 1] - a.cu_k[b], 0), a.len_cap);
  };

  // ---- group bounds, made to ascend
  long long carry = 0;
  for (int base = 0; base <= G; base += kPlanThreads) {
    const int i = base + tid;
    long long v = i <= G ? min(max(a.cu_groups[i], 0), B) : 0;
    v = block_scan<long long>(v, part, [](long long x, long long y) { return max(x, y); });
    v = max(v, carry);
    if (i <= G) p.cu[i] = static_cast<int>(v);
    carry = max(carry, part[31]);
    __syncthreads();
  }

  // ---- shared keys of each group, and the first of its sequences that has them all
  for (int g = warp; g < G; g += kPlanThreads / 32) {
    const int b0 = p.cu[g], b1 = p.cu[g + 1];
    const int want = min(max(a.prefix_lens[g], 0), a.len_cap) / a.block_size * a.block_size;
    int owner = -1;
    for (int base = b0; want > 0 && base < b1 && owner < 0; base += 32) {
      const int b = base + lane;
      const unsigned has = __ballot_sync(kFull, b < b1 && kv_len(b) >= want);
      if (has) owner = base + __ffs(has) - 1;
    }
    if (lane == 0) {
      int t0 = b0, t1 = b1;
      if (!decode) {
        t0 = min(max(a.cu_q[b0], 0), a.rows);
        t1 = min(max(a.cu_q[b1], t0), a.rows);
      }
      p.tok[2 * g] = t0;
      p.tok[2 * g + 1] = t1;
      p.owner[g] = max(owner, 0);
      p.keys[g] = owner >= 0 && t1 > t0 ? want : 0;
    }
  }
  __syncthreads();

  // ---- segments and units before each group
  const int per_seg = a.tokens_per_tile * a.row_tiles;
  long long segs = 0, units = 0;
  for (int base = 0; base < G; base += kPlanThreads) {
    const int g = base + tid;
    long long s = 0, u = 0;
    if (g < G && p.keys[g] > 0) {
      s = static_cast<long long>((p.tok[2 * g + 1] - p.tok[2 * g] + per_seg - 1) / per_seg) *
          a.num_kv_heads;
      u = s * ((p.keys[g] + kBN - 1) / kBN);
    }
    auto add = [](long long x, long long y) { return x + y; };
    const long long si = block_scan<long long>(s, part, add);
    const long long s_all = part[31];
    __syncthreads();
    const long long ui = block_scan<long long>(u, part, add);
    if (g < G) {
      p.seg[g] = static_cast<int>(segs + si - s);
      p.unit[g] = units + ui - u;
    }
    segs += s_all;
    units += part[31];
    __syncthreads();
  }
  // (only row bounds that do not ascend could need more segments than there is
  // room for: nothing is shared then)
  const bool fits = segs <= a.max_segments;
  if (tid == 0) {
    p.seg[G] = fits ? static_cast<int>(segs) : 0;
    p.unit[G] = fits ? units : 0;
  }

  // ---- rows
  auto group_of = [&](int b) {  // the group that holds sequence b, if it shares keys
    int lo = 0, hi = G;  // last g with cu[g] <= b
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] <= b) lo = mid; else hi = mid;
    }
    return fits && p.cu[lo] <= b && b < p.cu[lo + 1] && p.keys[lo] > 0 ? lo : -1;
  };
  if (decode) {
    for (int b = tid; b < B; b += kPlanThreads) {
      const int g = group_of(b);
      p.row_vis[b] = kv_len(b);
      p.row_grp[b] = g;
      p.row_start[b] = g >= 0 ? p.keys[g] : 0;
    }
    return;
  }
  const int t_lo = a.cu_q[0], t_hi = a.cu_q[B];
  for (int t = tid; t < a.rows; t += kPlanThreads)
    if (t < t_lo || t >= t_hi) p.row_vis[t] = -1, p.row_grp[t] = -1, p.row_start[t] = 0;
  for (int b = warp; b < B; b += kPlanThreads / 32) {
    const int q0 = a.cu_q[b], q1 = min(a.cu_q[b + 1], a.rows);
    const int kv = kv_len(b), cached = max(kv - (a.cu_q[b + 1] - q0), 0);
    const int g = group_of(b), start = g >= 0 ? p.keys[g] : 0;
    for (int t = max(q0, 0) + lane; t < q1; t += 32) {
      p.row_vis[t] = min(cached + (t - q0) + 1, kv);
      p.row_grp[t] = g;
      p.row_start[t] = start;
    }
  }
}

// ============================================================ shared keys
// CTA c of the W that work owns units [c N / W, (c+1) N / W). A unit is dearer
// than a CTA's start only where there are very few of them, so as many CTAs as
// there are units work.
__device__ __forceinline__ long long working_ctas(long long units, int ctas) {
  return max(1LL, min(units, static_cast<long long>(ctas)));
}

// One CTA's run of key tiles within one segment.
struct Piece {
  int kvh, tok0, tok1;  // kv head; rows: first of the segment, past the group's last
  int t0, t1;           // key tiles
  int keys, owner;      // of the group
  long long slot;       // of the partial: segment + CTA (unique: either grows from piece to piece)
};

// (The plan is read past L1: this launch may overlap others on its SM.)
struct PieceWalk {
  long long u, u1;
  int g, cta;
  __device__ __forceinline__ PieceWalk(const SharedArgs& a) {
    const long long N = __ldcg(a.plan.unit + a.num_groups), W = working_ctas(N, a.ctas);
    cta = blockIdx.x;
    u = cta < W ? cta * N / W : N;
    u1 = cta < W ? (cta + 1) * N / W : N;
    g = 0;
    int hi = a.num_groups;  // last g with unit[g] <= u
    while (u < u1 && hi - g > 1) {
      const int mid = (g + hi) >> 1;
      if (__ldcg(a.plan.unit + mid) <= u) g = mid; else hi = mid;
    }
  }
  // The next piece, or false.
  __device__ __forceinline__ bool next(const SharedArgs& a, Piece& p) {
    if (u >= u1) return false;
    while (__ldcg(a.plan.unit + g + 1) <= u) ++g;
    p.keys = __ldcg(a.plan.keys + g);
    p.owner = __ldcg(a.plan.owner + g);
    const int first = __ldcg(a.plan.tok + 2 * g);
    p.tok1 = __ldcg(a.plan.tok + 2 * g + 1);
    const int per_seg = a.tokens_per_tile * a.row_tiles;
    const int R = (p.tok1 - first + per_seg - 1) / per_seg, KT = (p.keys + kBN - 1) / kBN;
    const long long off = u - __ldcg(a.plan.unit + g);
    const int s = static_cast<int>(off / KT);
    p.t0 = static_cast<int>(off % KT);
    p.t1 = static_cast<int>(min(static_cast<long long>(KT), p.t0 + (u1 - u)));
    p.kvh = s / R;
    p.tok0 = first + (s % R) * per_seg;
    p.slot = static_cast<long long>(__ldcg(a.plan.seg + g)) + s + cta;
    u += p.t1 - p.t0;
    return true;
  }
};

constexpr int kThreads = 384;  // 2 x 4 softmax warps, K, MMA, V and Q warps
// Register split (setmaxnreg), as the prefill kernel's: 2*128*208 + 128*88 = 384*168.
constexpr int kSoftmaxRegs = 208;
constexpr int kControlRegs = 88;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kControlRegs <= kThreads * 168,
              "register split exceeds the launch allocation");
constexpr float kRescaleThreshold = 8.0f;  // log2 units

// K (and V) stages: what shared memory holds beside the query tiles.
template <int D, bool PAIR>
struct Ring {
  static constexpr int kTile = (D / 64) * kSub;
  static constexpr int kQTiles = PAIR ? 2 : 1;
  static constexpr int kStages = D == 64 ? (PAIR ? 4 : 6) : (PAIR ? 2 : 3);
  static constexpr int kBytes = 1024 + (kQTiles + 2 * kStages) * kTile;
  // (the static part: barriers and 1 KB of row sums)
  static_assert(kBytes <= 225 * 1024 + 512, "shared memory over the per-CTA limit");
};
constexpr int kMaxStages = 6;

enum {
  BAR_QF = 0,                    // Q tiles landed
  BAR_QE,                        // the last S of the segment is done
  BAR_KF,                        // + stage
  BAR_KE = BAR_KF + kMaxStages,
  BAR_VF = BAR_KE + kMaxStages,
  BAR_VE = BAR_VF + kMaxStages,
  BAR_S = BAR_VE + kMaxStages,   // + half: S ready
  BAR_P = BAR_S + 2,             // + half: P written (4 warps)
  BAR_O = BAR_P + 2,             // + half: P.V done
  BAR_E = BAR_O + 2,             // + half: O of the piece has been read (4 warps)
  BAR_ML = BAR_E + 2,            // second half's (max, sum) written (4 warps)
  BAR_DRAIN,
  NBAR
};

// Bounded wait that also gives up when another role of the CTA has aborted.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          uint32_t* err) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const unsigned long long t0 = global_timer_ns();
    while (!ok) {
#pragma unroll 1
      for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, parity);
      if (ok || *abort_flag) break;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        report_error(err, PA_DEVERR_WAIT_TIMEOUT);
        break;
      }
    }
  }
  return __all_sync(kFull, ok);
}

template <int D, int BS, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    shared_keys_kernel(const __grid_constant__ CUtensorMap qmap,
                       const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const SharedArgs a) {
  using R = Ring<D, PAIR>;
  constexpr int ST = R::kStages, kTile = R::kTile, kBlocks = kBN / BS;
  constexpr int kCols = D / 32;  // 32-column chunks of O
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[NBAR];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ float2 half_ml[PAIR ? 1 : kBM];  // the second half's (max, sum) of each row

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.group, TPT = a.tokens_per_tile;
  // The launch before this one (each sequence's own keys) let it start only
  // after the plan was complete, and works beside it: its results are waited
  // for at the end, on behalf of the merge.
  PieceWalk walk(a);
  if (walk.u >= walk.u1) {
    grid_dependency_wait();
    return;
  }

  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  auto q_s = [&](int i) { return base + i * kTile; };
  auto k_s = [&](int s) { return base + (R::kQTiles + s) * kTile; };
  auto v_s = [&](int s) { return base + (R::kQTiles + ST + s) * kTile; };
  const uint32_t bar0 = smem_addr(&bars[0]);
  auto bar = [&](int i) { return bar0 + 8u * i; };
  if (threadIdx.x == 0) {
    for (int i = 0; i < NBAR; ++i) {
      const bool warps4 = i == BAR_P || i == BAR_P + 1 || i == BAR_E || i == BAR_E + 1 || i == BAR_ML;
      mbar_init(bar(i), warps4 ? 4 : 1);
    }
    abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 9) {
    tc::tmem_alloc(smem_addr(&tmem_slot), 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  auto tS = [&](int i) { return tmem + 128u * i; };  // S, then P (terms in columns 0-63, 64-127)
  auto tO = [&](int i) { return tmem + 256u + 128u * i; };
  auto wait = [&](int b, uint32_t parity) { return warp_wait(bar(b), parity, &abort_flag, a.err); };

  Piece p;
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp == 11) {
      // ---------------------------------------------------------- Q producer
      uint32_t n = 0;
      bool pending = false;
      for (; walk.next(a, p); ++n) {
        if (n > 0 && !wait(BAR_QE, (n - 1) & 1)) break;
        const int tiles = PAIR && p.tok0 + TPT < p.tok1 ? 2 : 1;
        if (lane == 0) {
          // a box is G heads of TPT tokens: TPT * G rows of 128 bytes
          mbar_arrive_expect_tx(bar(BAR_QF), tiles * (D / 64) * TPT * G * 128);
          for (int i = 0; i < tiles; ++i)
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(q_s(i) + c * kSub, &qmap, bar(BAR_QF), 64 * c, p.kvh * G,
                          p.tok0 + i * TPT);
        }
        __syncwarp();
        pending = true;
      }
      if (abort_flag && pending) (void)mbar_wait(bar(BAR_QF), (n - 1) & 1);
    } else if (warp == 8 || warp == 10) {
      // ---------------------------------------------------------- K, V producers
      const bool is_k = warp == 8;
      const CUtensorMap* map = is_k ? &kmap : &vmap;
      const int full0 = is_k ? BAR_KF : BAR_VF, empty0 = is_k ? BAR_KE : BAR_VE;
      const int oob = a.num_blocks * BS;  // first row past the pool: TMA fills zeros
      uint32_t c = 0;
      bool ok = true;
      while (ok && walk.next(a, p)) {
        const long long bt_row = static_cast<long long>(p.owner) * a.max_blocks;
        const int nblk = p.keys / BS;
        // block ids 32 at a time (lane l: block wb + l, as the pool row of its
        // first key), the next ones' reads under way while these are used
        auto load_ids = [&](int wb) {
          const int lb = wb + lane;
          int rc = oob;
          if (lb < nblk) {
            const int phys = a.block_tables[bt_row + lb];
            if (phys >= 0 && phys < a.num_blocks) rc = phys * BS;
            else if (is_k) report_error(a.err, PA_DEVERR_BLOCK_RANGE);
          }
          return rc;
        };
        int wb = p.t0 * kBlocks;
        int ids = load_ids(wb), nxt = load_ids(wb + 32);
        for (int t = p.t0; t < p.t1; ++t, ++c) {
          if (t * kBlocks - wb == 32) {  // (whole tiles fit a window)
            wb += 32;
            ids = nxt;
            nxt = load_ids(wb + 32);
          }
          const int s = c % ST;
          if (c >= ST && !wait(empty0 + s, (c / ST - 1) & 1)) {
            ok = false;
            break;
          }
          const uint32_t dst = is_k ? k_s(s) : v_s(s);
          if (lane == 0) mbar_arrive_expect_tx(bar(full0 + s), kTile);
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) {
            const int rc = __shfl_sync(kFull, ids, t * kBlocks - wb + i);
            if (lane == 0) {
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_load_3d(dst + h * kSub + i * BS * 128, map, bar(full0 + s), 64 * h, p.kvh, rc);
            }
          }
        }
      }
      if (abort_flag) {
        // let the copies already in flight land before shared memory is released
        for (uint32_t n = c > ST ? c - ST : 0; n < c; ++n)
          (void)mbar_wait(bar(full0 + n % ST), (n / ST) & 1);
      }
    } else {
      // ---------------------------------------------------------- MMA issue
      constexpr uint32_t kIdescQK = tc::idesc_bf16_f32(kBM, kBN, false, false);
      constexpr uint32_t kIdescPV = tc::idesc_bf16_f32(kBM, D, false, true);
      auto issue_s = [&](int i, uint32_t c) {  // S_i = Q K(c)^T
        const uint32_t q = q_s(PAIR ? i : 0), k = k_s(c % ST);
        tc::fence_after_sync();
        if (lane == 0) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kSub + (kk & 3) * 32;
            tc::mma_ss(tS(i), tc::smem_desc_sw128(q + off, 16, 1024),
                       tc::smem_desc_sw128(k + off, 16, 1024), kIdescQK, kk > 0 ? 1u : 0u);
          }
          tc::commit(bar(BAR_S + i));
        }
        __syncwarp();
      };
      auto issue_pv = [&](int i, uint32_t c, bool first) {  // O_i (+)= P_i V(c), both terms
        const uint32_t v = v_s(c % ST);
        tc::fence_after_sync();
        if (lane == 0) {
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int kk = 0; kk < kBN / 16; ++kk)
              tc::mma_ts(tO(i), tS(i) + 64 * t + kk * 8,
                         tc::smem_desc_sw128(v + kk * 16 * 128, kSub, 1024), kIdescPV,
                         !first || kk > 0 || t > 0 ? 1u : 0u);
          }
          tc::commit(bar(BAR_O + i));
        }
        __syncwarp();
      };
      auto commit = [&](int b) {
        if (lane == 0) tc::commit(bar(b));
        __syncwarp();
      };
      uint32_t c = 0;                // key tiles before the piece
      uint32_t done0 = 0, done1 = 0;  // tiles of each half so far
      uint32_t ends0 = 0, ends1 = 0;  // pieces of each half so far
      auto done = [&](int i) -> uint32_t& { return i ? done1 : done0; };
      auto ends = [&](int i) -> uint32_t& { return i ? ends1 : ends0; };
      bool ok = true;
      for (uint32_t n = 0; ok && walk.next(a, p); ++n) {
        const int T = p.t1 - p.t0;
        // halves: the two row tiles (each takes every key tile), or the two
        // takers of one row tile's key tiles (half i: tiles i, i + 2, ...)
        const int halves = PAIR ? (p.tok0 + TPT < p.tok1 ? 2 : 1) : min(T, 2);
        constexpr int kStep = PAIR ? 1 : 2;
        ok = wait(BAR_QF, n & 1);
        // the first S of each half: its P of the piece before has been read
        for (int i = 0; ok && i < halves; ++i) {
          const int t = PAIR ? 0 : i;
          ok = (t > 0 || i == 0 ? wait(BAR_KF + (c + t) % ST, ((c + t) / ST) & 1) : true) &&
               (done(i) == 0 || wait(BAR_O + i, (done(i) - 1) & 1));
          if (!ok) break;
          issue_s(i, c + t);
          if (!PAIR || i == halves - 1) commit(BAR_KE + (c + t) % ST);
        }
        if (ok && T <= kStep) commit(BAR_QE);
        for (int t = 0; ok && t < T; ++t) {
          const uint32_t ct = c + t, cn = ct + kStep;
          const bool more = t + kStep < T;
          ok = wait(BAR_VF + ct % ST, (ct / ST) & 1) &&
               (!more || wait(BAR_KF + cn % ST, (cn / ST) & 1));
          for (int i = PAIR ? 0 : t & 1; ok && i < (PAIR ? halves : (t & 1) + 1); ++i) {
            ok = wait(BAR_P + i, done(i) & 1) &&
                 (t >= kStep || ends(i) == 0 || wait(BAR_E + i, (ends(i) - 1) & 1));
            if (!ok) break;
            issue_pv(i, ct, t < kStep);
            if (more) {
              ok = wait(BAR_O + i, done(i) & 1);
              if (!ok) break;
              issue_s(i, cn);
            }
            ++done(i);
          }
          if (!ok) break;
          commit(BAR_VE + ct % ST);
          if (more) commit(BAR_KE + cn % ST);
          if (more && t + kStep == T - 1) commit(BAR_QE);
        }
        c += T;
        for (int i = 0; i < halves; ++i) ++ends(i);
      }
      if (abort_flag) {  // no MMA may still run when TMEM is freed
        commit(BAR_DRAIN);
        (void)mbar_wait(bar(BAR_DRAIN), 0);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------------------ softmax
    const int hf = warp / 4;  // half: row tile (PAIR) or taker of every other key tile
    const int r = 32 * (warp & 3) + lane;  // row of the tile = TMEM lane
    const uint32_t trow = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const float sl2 = a.scale_log2;
    constexpr int kStep = PAIR ? 1 : 2;
    uint32_t done = 0;    // tiles of this half so far
    uint32_t other = 0;   // first half, one row tile: tiles of the second half so far
    uint32_t merged = 0;  // pieces in which the second half had tiles
    bool ok = true;
    for (uint32_t n = 0; ok && walk.next(a, p); ++n) {
      const int T = p.t1 - p.t0;
      if (PAIR && hf == 1 && p.tok0 + TPT >= p.tok1) continue;  // one row tile in this segment
      const int tok = p.tok0 + (PAIR ? hf * TPT : 0) + r / G;
      const bool valid = r < TPT * G && tok < p.tok1;
      const int lim = valid ? min(p.keys, __ldcg(a.plan.row_vis + tok)) : p.keys;  // keys the row sees
      float m_used = -INFINITY, l = 0.f;
      const int first = PAIR ? 0 : hf;
      for (int t = first; t < T; t += kStep) {
        ok = wait(BAR_S + hf, done & 1);
        if (!ok) break;
        tc::fence_after_sync();
        uint32_t u[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_ld32(tS(hf) + trow + 32 * c, u[c]);
        tc::tmem_wait_ld();
        const int left = lim - (p.t0 + t) * kBN;  // keys of this tile the row sees
        if (!__all_sync(kFull, left >= kBN)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * c + j >= left) u[c][j] = __float_as_uint(-INFINITY);
        }
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          mx = fmaxf(mx, fmaxf(fmaxf(__uint_as_float(u[0][j]), __uint_as_float(u[1][j])),
                               fmaxf(__uint_as_float(u[2][j]), __uint_as_float(u[3][j]))));
        // (scores in base 2 grow with the raw ones, or fall where the scale is negative)
        const float m_tile = mx * sl2;
        if (t == first) {
          m_used = m_tile;
        } else if (__any_sync(kFull, m_tile > m_used + kRescaleThreshold)) {
          // raise the maximum and rescale O: its last product must be done
          ok = wait(BAR_O + hf, (done - 1) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          const float m_new = fmaxf(m_used, m_tile);
          // (a row that has seen no key yet has nothing to rescale)
          const float alpha = m_new == -INFINITY ? 1.f : fast_exp2(m_used - m_new);
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            tc::tmem_ld32(tO(hf) + trow + 32 * c, w);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) * alpha);
            tc::tmem_st32(tO(hf) + trow + 32 * c, w);
          }
          tc::tmem_wait_st();
          l *= alpha;
          m_used = m_new;
        }
        // P = 2^(s * scale * log2(e) - m_used) as two bf16 terms; pairs of keys
        // share one packed FMA and one packed add
        const float nm = m_used == -INFINITY ? 0.f : -m_used;
        const uint64_t sl2x2 = tc::f32x2(sl2, sl2), nmx2 = tc::f32x2(nm, nm);
        uint64_t lsum = tc::f32x2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint64_t x = tc::fma_f32x2(
                tc::f32x2(__uint_as_float(u[c][2 * j]), __uint_as_float(u[c][2 * j + 1])), sl2x2,
                nmx2);
            float x0, x1;
            tc::f32x2_split(x, x0, x1);
            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
            lsum = tc::add_f32x2(lsum, tc::f32x2(p0, p1));
            hi[j] = pack_bf16x2(p0, p1);
            lo[j] = pack_bf16x2(p0 - __uint_as_float(hi[j] << 16),
                                p1 - __uint_as_float(hi[j] & 0xffff0000u));
          }
          tc::tmem_st16(tS(hf) + trow + 16 * c, hi);
          tc::tmem_st16(tS(hf) + trow + 64 + 16 * c, lo);
        }
        float la, lb;
        tc::f32x2_split(lsum, la, lb);
        l += la + lb;
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_P + hf));
        ++done;
      }
      if (!ok) break;
      // ---- the piece's partial: (max, sum) and O, unnormalised
      float f0 = 1.f, f1 = 0.f;
      const bool both = !PAIR && T > 1;
      if constexpr (!PAIR) {
        if (both) {
          if (hf == 1) {
            // (the first half has read the piece before's once that O is released)
            ok = merged == 0 || wait(BAR_E + 1, (merged - 1) & 1);
            if (!ok) break;
            half_ml[r] = make_float2(m_used, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(BAR_ML));
            ++merged;
            continue;  // the first half reads this half's O, in the same TMEM lanes
          }
          other += T / 2;
          ok = wait(BAR_ML, merged & 1) && wait(BAR_O + 1, (other - 1) & 1);
          if (!ok) break;
          const float2 o = half_ml[r];
          ++merged;
          const float m = fmaxf(m_used, o.x);
          f0 = m_used == -INFINITY ? 0.f : fast_exp2(m_used - m);
          f1 = o.x == -INFINITY ? 0.f : fast_exp2(o.x - m);
          l = l * f0 + o.y * f1;
          m_used = m;
        } else if (hf == 1) {
          continue;
        }
      }
      ok = wait(BAR_O + hf, (done - 1) & 1);
      if (!ok) break;
      tc::fence_after_sync();
      const long long row = p.slot * (kBM * a.row_tiles) + (PAIR ? hf * kBM : 0) + r;
      float4* const dst = reinterpret_cast<float4*>(a.part_o + row * D);
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        uint32_t w[32];
        tc::tmem_ld32(tO(hf) + trow + 32 * c, w);
        tc::tmem_wait_ld();
        if (both) {
          uint32_t v[32];
          tc::tmem_ld32(tO(1) + trow + 32 * c, v);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j)
            w[j] = __float_as_uint(__uint_as_float(w[j]) * f0 + __uint_as_float(v[j]) * f1);
        }
        if (valid) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[8 * c + j] = make_float4(__uint_as_float(w[4 * j]), __uint_as_float(w[4 * j + 1]),
                                         __uint_as_float(w[4 * j + 2]), __uint_as_float(w[4 * j + 3]));
        }
      }
      if (valid) a.part_ml[row] = make_float2(m_used, l);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(BAR_E + hf));
        if (both) mbar_arrive(bar(BAR_E + 1));
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
  grid_dependency_wait();
}

// ============================================================ merge
constexpr int kMergeWarps = 4;

// One row and head on D/4 lanes, 16 bytes of O each: its parts of the shared
// keys in order, then its own keys' result.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) shared_merge_kernel(const SharedArgs a) {
  constexpr int LPR = D / 4, RPW = 32 / LPR;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, sub = lane % LPR;
  const long long rh = (static_cast<long long>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5)) * RPW +
                       lane / LPR;
  const bool in = rh < static_cast<long long>(a.rows) * a.num_heads;
  const int t = in ? static_cast<int>(rh / a.num_heads) : 0;
  const int h = in ? static_cast<int>(rh % a.num_heads) : 0;
  const int vis = in ? a.plan.row_vis[t] : -1;
  const int g = in ? a.plan.row_grp[t] : -1;
  const bool own = vis > (in ? a.plan.row_start[t] : 0);

  // ---- the row's parts: slots seg + c of the CTAs c that own units of its segment
  long long first = 0;
  int n = 0, r = 0;
  if (g >= 0) {
    const int per_seg = a.tokens_per_tile * a.row_tiles, kvh = h / a.group;
    const int i = t - a.plan.tok[2 * g], rows = a.plan.tok[2 * g + 1] - a.plan.tok[2 * g];
    const int R = (rows + per_seg - 1) / per_seg, KT = (a.plan.keys[g] + kBN - 1) / kBN;
    const int s = kvh * R + i / per_seg, q = i % per_seg;
    r = q / a.tokens_per_tile * kBM + q % a.tokens_per_tile * a.group + h % a.group;
    const long long N = a.plan.unit[a.num_groups], W = working_ctas(N, a.ctas);
    const long long u0 = a.plan.unit[g] + static_cast<long long>(s) * KT;
    const long long c0 = ((u0 + 1) * W - 1) / N, c1 = ((u0 + KT) * W - 1) / N;
    first = a.plan.seg[g] + s + c0;
    n = static_cast<int>(c1 - c0 + 1);
  }
  auto part = [&](int j) { return (first + j) * (kBM * a.row_tiles) + r; };

  // ---- (max, sum): a lane takes every LPR-th part, then the row's lanes combine
  float M = -INFINITY, L = 0.f;
  auto fold = [&](float m, float l) {
    const float m2 = fmaxf(M, m);
    if (m2 != -INFINITY) {
      L = L * fast_exp2(M - m2) + l * fast_exp2(m - m2);
      M = m2;
    }
  };
  for (int j = sub; j < n; j += LPR) {
    const float2 ml = __ldcg(a.part_ml + part(j));
    fold(ml.x, ml.y);
  }
  float2 mine = make_float2(-INFINITY, 0.f);
  if (own) mine = __ldcg(a.own_ml + rh);
  if (own && sub == 0) fold(mine.x, mine.y);
#pragma unroll
  for (int o = LPR / 2; o >= 1; o >>= 1) {
    const float m = __shfl_xor_sync(kFull, M, o), l = __shfl_xor_sync(kFull, L, o);
    fold(m, l);
  }

  // ---- O
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float m, const float4& x) {
    const float f = m == -INFINITY ? 0.f : fast_exp2(m - M);
    acc.x += f * x.x;
    acc.y += f * x.y;
    acc.z += f * x.z;
    acc.w += f * x.w;
  };
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const long long row = part(j);
    const float m = __ldcg(&a.part_ml[row].x);
    add(m, __ldcg(reinterpret_cast<const float4*>(a.part_o + row * D) + sub));
  }
  if (own) add(mine.x, __ldcg(reinterpret_cast<const float4*>(a.own_o + rh * D) + sub));
  if (vis < 0) return;
  const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // no keys: zeros; NaN stays
  uint2 w;
  w.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  w.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + rh * D)[sub] = w;
}

// ============================================================ host side
cudaLaunchConfig_t config(dim3 grid, int threads, size_t smem, cudaStream_t stream,
                          cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int D, int BS, bool PAIR>
cudaError_t launch_keys(const SharedArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                        const CUtensorMap& vmap, cudaStream_t stream) {
  auto* k = shared_keys_kernel<D, BS, PAIR>;
  constexpr int smem = Ring<D, PAIR>::kBytes;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(dim3(a.ctas), kThreads, smem, stream, attr);
  return cudaLaunchKernelEx(&cfg, k, qmap, kmap, vmap, a);
}

}  // namespace

SharedLayout shared_layout(size_t base, int rows, int num_heads, int num_kv_heads, int head_dim,
                           int num_groups, int num_sms) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  SharedLayout l{};
  l.tokens_per_tile = kBM / (num_heads / num_kv_heads);
  // Two row tiles a segment where the groups have the rows for them on average:
  // a K/V tile then serves twice the rows. Smaller groups leave the second tile
  // empty, and are bound by reading the keys.
  const long long tiles = (rows + static_cast<long long>(l.tokens_per_tile) - 1) / l.tokens_per_tile;
  l.row_tiles = tiles > std::max(num_groups, 1) ? 2 : 1;
  const long long per_seg = static_cast<long long>(l.tokens_per_tile) * l.row_tiles;
  // every group may end in a segment that is not full
  const long long segs = (rows / per_seg + std::min(num_groups, rows)) * num_kv_heads;
  l.max_segments = static_cast<int>(std::min<long long>(segs, 0x7fffffff));
  l.ctas = num_sms;
  const size_t slots = static_cast<size_t>(segs) + l.ctas;
  const size_t part_rows = slots * kBM * l.row_tiles;
  const size_t rh = static_cast<size_t>(rows) * num_heads;
  l.plan = up(base);
  const size_t plan_bytes = (static_cast<size_t>(num_groups) + 1) * (sizeof(long long) + 6 * sizeof(int)) +
                            3 * static_cast<size_t>(rows) * sizeof(int);
  l.part_ml = up(l.plan + plan_bytes);
  l.part_o = up(l.part_ml + part_rows * sizeof(float2));
  l.own_ml = up(l.part_o + part_rows * head_dim * sizeof(float));
  l.own_o = up(l.own_ml + rh * sizeof(float2));
  l.bytes = l.own_o + rh * head_dim * sizeof(float);
  return l;
}

void shared_pointers(SharedArgs& a, const SharedLayout& l, void* workspace) {
  char* const ws = static_cast<char*>(workspace);
  const int g1 = a.num_groups + 1;
  a.plan.unit = reinterpret_cast<long long*>(ws + l.plan);
  a.plan.cu = reinterpret_cast<int*>(a.plan.unit + g1);
  a.plan.keys = a.plan.cu + g1;
  a.plan.owner = a.plan.keys + g1;
  a.plan.seg = a.plan.owner + g1;
  a.plan.tok = a.plan.seg + g1;
  a.plan.row_vis = a.plan.tok + 2 * g1;
  a.plan.row_grp = a.plan.row_vis + a.rows;
  a.plan.row_start = a.plan.row_grp + a.rows;
  a.part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
  a.part_o = reinterpret_cast<float*>(ws + l.part_o);
  a.own_ml = reinterpret_cast<float2*>(ws + l.own_ml);
  a.own_o = reinterpret_cast<float*>(ws + l.own_o);
  a.tokens_per_tile = l.tokens_per_tile;
  a.row_tiles = l.row_tiles;
  a.max_segments = l.max_segments;
  a.ctas = l.ctas;
}

cudaError_t launch_shared_plan(const SharedArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(dim3(1), kPlanThreads, 0, stream, attr);
  return cudaLaunchKernelEx(&cfg, shared_plan_kernel, a);
}

cudaError_t launch_shared_keys(const SharedArgs& a, const CUtensorMap& qmap,
                               const CUtensorMap& kmap, const CUtensorMap& vmap,
                               cudaStream_t stream) {
  const bool pair = a.row_tiles == 2;
  if (a.head_dim == 128 && a.block_size == 16)
    return pair ? launch_keys<128, 16, true>(a, qmap, kmap, vmap, stream)
                : launch_keys<128, 16, false>(a, qmap, kmap, vmap, stream);
  if (a.head_dim == 128 && a.block_size == 32)
    return pair ? launch_keys<128, 32, true>(a, qmap, kmap, vmap, stream)
                : launch_keys<128, 32, false>(a, qmap, kmap, vmap, stream);
  if (a.head_dim == 64 && a.block_size == 16)
    return pair ? launch_keys<64, 16, true>(a, qmap, kmap, vmap, stream)
                : launch_keys<64, 16, false>(a, qmap, kmap, vmap, stream);
  if (a.head_dim == 64 && a.block_size == 32)
    return pair ? launch_keys<64, 32, true>(a, qmap, kmap, vmap, stream)
                : launch_keys<64, 32, false>(a, qmap, kmap, vmap, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_shared_merge(const SharedArgs& a, cudaStream_t stream) {
  const long long rh = static_cast<long long>(a.rows) * a.num_heads;
  const long long per_cta = kMergeWarps * (128 / a.head_dim);
  const long long grid = (rh + per_cta - 1) / per_cta;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      config(dim3(static_cast<unsigned>(grid)), kMergeWarps * 32, 0, stream, attr);
  return a.head_dim == 64 ? cudaLaunchKernelEx(&cfg, shared_merge_kernel<64>, a)
                          : cudaLaunchKernelEx(&cfg, shared_merge_kernel<128>, a);
}

}  // namespace pa
