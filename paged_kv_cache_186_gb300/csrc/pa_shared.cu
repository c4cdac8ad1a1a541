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
// per segment it meets. Sixteen warps:
//   * warp 8 brings Q and K, warp 10 V, by TMA (one box per physical block and 64
//     dims), each through its own ring, block ids read 32 ahead. One elected lane
//     issues all copies of a tile: behind elect.sync their operands are taken from
//     uniform registers, behind a comparison of the lane number a 16-copy tile took
//     1300-1600 clocks instead of 400-480.
//   * warps 12-15 turn V into f16 times a power of two (moved when a tile's largest
//     value leaves its range, O being rescaled with it), and widen 8-bit codes, K
//     to bf16 and V to f16, exactly; their scales go to the scores and the weights.
//     P then goes into P.V as one f16 term (11 bits, at most 2^-11 of a weight off).
//     In bf16 a row whose weight lies on few keys misses the library's tolerance
//     (1.28e-2 measured on rows with four dominant keys, and shared prompts begin
//     with such keys), and a second bf16 term costs as much tensor time again.
//   * warps 9 and 11 issue the MMAs of one half each, one thread of each from end
//     to end. A half is one of two row tiles (PAIR: a K/V tile serves 256 rows), or
//     one of the two takers of a single row tile's key tiles, in turn, whose
//     results meet at the end of a segment.
//   * warps 0-7: a softmax warpgroup a half, one TMEM lane (row) a thread, 64 keys a
//     step. S is read into registers at once and its columns given back, so that
//     the next S is made during the step; P has two buffers of its own. TMEM, 512
//     columns: per half S 64, P 2 x 32, O 128.
// What it measured, per 128-key tile of a CTA with two row tiles (questions of 16-256
// tokens over four documents, 32/8 heads of 128, one GB300):
// S of 128 keys with P stored over it 6000 clocks; two S buffers of 64 keys, MMAs
// issued by lane 0 8900, by one elected thread 4900; f16 P 4800; S given back once
// read, an MMA warp a half 3850; fewer waits in a step 3600. 2.0 us a tile now, 0.66
// of the measured bf16 rate. The bound is the softmax step (about 1400 clocks, of
// which 440 are the exponentials) next to shared memory, busy 3250 clocks of a tile
// at 128 bytes a clock (192 KB of operands of Q.K, 64 of P.V, 64 of copies, 64-96 of
// conversion): a satisfied wait on an mbarrier takes 200 clocks there. With one row
// tile a call is bound by reading the keys: 32 sequences behind 131067 keys take 82
// us in the CTAs, 6.5 TB/s. 8-bit codes 4700 clocks a tile (scales and widening).
#include <algorithm>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_launch.h"
#include "pa_shared.h"
#include "pa_tcgen05.cuh"

namespace pa {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBM = 128;  // rows per query tile
constexpr int kBN = 128;  // keys per tile
constexpr int kSN = 64;   // keys per step: half a tile
constexpr int kSub = 128 * kBM;  // bytes of a 64-dim (128-byte-wide) column of a 128-row tile

// ============================================================ plan
// CTA c of the W that work owns units [c N / W, (c+1) N / W). A unit is dearer
// than a CTA's start only where there are very few of them, so as many CTAs as
// there are units work.
__device__ __forceinline__ long long working_ctas(long long units, int ctas) {
  return max(1LL, min(units, static_cast<long long>(ctas)));
}

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

// Groups whose bounds and keys the plan keeps in shared memory; more are read
// back from the workspace.
constexpr int kPlanGroups = 512;

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedArgs a) {
  __shared__ long long part[32];
  __shared__ int s_cu[kPlanGroups + 1], s_keys[kPlanGroups];
  __shared__ float sums[4][kPlanThreads / 32];
  const SharedPlan& p = a.plan;
  const int G = a.num_groups, B = a.batch, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const bool decode = a.context_lens != nullptr;
  const bool few = G <= kPlanGroups;
  int* const cu = few ? s_cu : p.cu;
  int* const keys = few ? s_keys : p.keys;
  // what this launch writes may still be read by the call before it, and its
  // inputs written by the launch before it
  grid_dependency_wait();
  grid_launch_dependents();
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
    if (i <= G) cu[i] = static_cast<int>(v);
    carry = max(carry, part[31]);
    __syncthreads();
  }

  // ---- shared keys of each group, and the first of its sequences that has them all
  for (int g = warp; g < G; g += kPlanThreads / 32) {
    const int b0 = cu[g], b1 = cu[g + 1];
    const int want = min(max(a.prefix_lens[g], 0), a.len_cap) / a.block_size * a.block_size;
    int t0 = b0, t1 = b1;
    if (!decode) {
      t0 = min(max(a.cu_q[b0], 0), a.rows);
      t1 = min(max(a.cu_q[b1], t0), a.rows);
    }
    int owner = -1;
    for (int base = b0; want > 0 && base < b1 && owner < 0; base += 32) {
      const int b = base + lane;
      const unsigned has = __ballot_sync(kFull, b < b1 && kv_len(b) >= want);
      if (has) owner = base + __ffs(has) - 1;
    }
    if (lane == 0) {
      const int k = owner >= 0 && t1 > t0 ? want : 0;
      keys[g] = k;
      if (few) p.keys[g] = k;
      p.tok[2 * g] = t0;
      p.tok[2 * g + 1] = t1;
      p.owner[g] = max(owner, 0);
    }
  }
  __syncthreads();

  // ---- prefill: does sharing pay? Unshared, CTA after CTA of the prefill kernel
  // walks the prefix: waves of them, each as long as its key tiles; shared, the
  // same products are spread evenly and full, but the call has a fixed cost, one
  // for each wave of the CTAs over the sequences' own keys, and one for each row
  // merged. In us, fitted on one GB300 over 2-64 sequences of 4-256 new tokens
  // behind 512-16384 keys (always shared / pa_prefill_varlen measured: 64 drafts of 4-8
  // tokens behind 4096 91 / 216, 32 questions of 1-64 behind 8000 147 / 219, 32 of 128
  // behind 8192 568 / 502, 8 of 32 behind 2048 48 / 30, 2 of 128 behind 8192 72 /
  // 129. (A decode step is chosen for on the host: its kernel's own cost is small.)
  if (!decode && !a.always) {
    const int span = a.own_tokens;  // new tokens of a sequence that one CTA takes
    float v[4] = {0.f, 0.f, 0.f, 0.f};  // CTAs, their key tiles, shared units, rows
    for (int g = warp; g < G; g += kPlanThreads / 32) {
      const int KT = (keys[g] + kBN - 1) / kBN, b0 = cu[g], b1 = cu[g + 1];
      if (KT == 0) continue;
      for (int b = b0 + lane; b < b1; b += 32) {
        const int n = (max(a.cu_q[b + 1] - a.cu_q[b], 0) + span - 1) / span;
        v[0] += n;
        v[1] += static_cast<float>(n) * KT;
      }
      if (lane == 0) {
        const int t = p.tok[2 * g + 1] - p.tok[2 * g], per = a.tokens_per_tile * a.row_tiles;
        v[2] += static_cast<float>((t + per - 1) / per) * KT;
        v[3] += t;
      }
    }
    // the CTA's sums, the same bits in every thread
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(kFull, v[i], o);
      if (lane == 0) sums[i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = sums[i][lane];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(kFull, v[i], o);
    }
    const float n = v[0] * a.num_kv_heads, tiles = v[1] / fmaxf(v[0], 1.f);
    const float u = v[2] * a.num_kv_heads, r = v[3] * a.num_heads;
    const float waves = ceilf(n / a.ctas);
    const float unshared = waves * tiles * 1.8f;
    const float shared = ceilf(u / a.ctas) * (a.row_tiles == 2 ? 2.f : 1.6f) + 14.f + 6.f * waves +
                         r * 4e-4f;
    if (shared >= unshared) {  // (the same in every thread)
      for (int g = tid; g < G; g += kPlanThreads) keys[g] = p.keys[g] = 0;
      __syncthreads();
    }
  }

  // ---- segments and units before each group
  const int per_seg = a.tokens_per_tile * a.row_tiles;
  long long segs = 0, units = 0;
  for (int base = 0; base < G; base += kPlanThreads) {
    const int g = base + tid;
    long long s = 0, u = 0;
    if (g < G && keys[g] > 0) {
      s = static_cast<long long>((p.tok[2 * g + 1] - p.tok[2 * g] + per_seg - 1) / per_seg) *
          a.num_kv_heads;
      u = s * ((keys[g] + kBN - 1) / kBN);
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

  __syncthreads();

  // ---- the partials of each segment: one of every CTA that owns units of it
  const long long W = working_ctas(units, a.ctas);
  for (int i = tid; fits && i < segs; i += kPlanThreads) {
    int lo = 0, hi = G;  // last g with seg[g] <= i (groups without segments come before it)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.seg[mid] <= i) lo = mid; else hi = mid;
    }
    const long long KT = (keys[lo] + kBN - 1) / kBN;
    const long long u0 = p.unit[lo] + (i - p.seg[lo]) * KT;
    const long long c0 = ((u0 + 1) * W - 1) / units, c1 = ((u0 + KT) * W - 1) / units;
    p.parts[i] = make_int2(static_cast<int>(i + c0), static_cast<int>(c1 - c0 + 1));
  }

  // ---- rows
  auto group_of = [&](int b) {  // the group that holds sequence b, if it shares keys
    int lo = 0, hi = G;  // last g with cu[g] <= b
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= b) lo = mid; else hi = mid;
    }
    return fits && cu[lo] <= b && b < cu[lo + 1] && keys[lo] > 0 ? lo : -1;
  };
  if (decode) {
    // (-1, 0): no own parts, until the decode kernel has finished the segment that
    // leaves some. One whose wait runs out names none: the merge must not take what
    // another call left here for slots and counts. (128 coalesced stores a thread at
    // 16384 sequences of 8 kv heads.)
    for (long long i = tid; i < static_cast<long long>(B) * a.num_kv_heads; i += kPlanThreads)
      a.own_parts[i] = make_int2(-1, 0);
    for (int b = tid; b < B; b += kPlanThreads) {
      const int g = group_of(b);
      p.row_vis[b] = kv_len(b);
      p.row_grp[b] = g;
      p.row_start[b] = g >= 0 ? keys[g] : 0;
    }
    return;
  }
  const int t_lo = a.cu_q[0], t_hi = a.cu_q[B];
  for (int t = tid; t < a.rows; t += kPlanThreads)
    if (t < t_lo || t >= t_hi) p.row_vis[t] = -1, p.row_grp[t] = -1, p.row_start[t] = 0;
  for (int b = warp; b < B; b += kPlanThreads / 32) {
    const int q0 = a.cu_q[b], q1 = min(a.cu_q[b + 1], a.rows);
    const int kv = kv_len(b), cached = max(kv - (a.cu_q[b + 1] - q0), 0);
    const int g = group_of(b), start = g >= 0 ? keys[g] : 0;
    for (int t = max(q0, 0) + lane; t < q1; t += 32) {
      p.row_vis[t] = min(cached + (t - q0) + 1, kv);
      p.row_grp[t] = g;
      p.row_start[t] = start;
    }
  }
}

// ============================================================ shared keys
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

constexpr int kThreads = 512;  // 8 softmax warps, Q and K, MMA, V, MMA, 4 converting warps
// Register split (setmaxnreg) of the launch's 512 x 128.
constexpr int kSoftmaxRegs = 160;
constexpr int kControlRegs = 96;
constexpr int kConvertRegs = 96;
static_assert(2 * kSoftmaxRegs + kControlRegs + kConvertRegs <= 4 * 128,
              "register split exceeds the launch allocation");
constexpr float kRescaleThreshold = 8.0f;  // log2 units: P stays below 2^8 of its row's scale

// Shared memory of a CTA. 8-bit codes (Q8) land as they are in raw stages of 128
// keys and are widened into the 16-bit ones; with one row tile the room of the
// second goes to deeper rings, since such calls are bound by the loads.
template <int D, bool Q8, bool PAIR>
struct Ring {
  static constexpr int kTile = (D / 64) * kSub;
  static constexpr int kRawTile = kBN * 128;
  static constexpr int kQTiles = PAIR ? 2 : 1;
  static constexpr int kK = Q8 ? 1 : D == 64 ? (PAIR ? 4 : 6) : PAIR ? 2 : 3;
  static constexpr int kV = Q8 ? 2 : D == 64 ? (PAIR ? 4 : 6) : 3;
  static constexpr int kRaw = Q8 ? 2 : 0;  // of K and of V each
  static constexpr int kQ0 = 0;
  static constexpr int kK0 = kQ0 + kQTiles * kTile;
  static constexpr int kV0 = kK0 + kK * kTile;
  static constexpr int kRawK0 = kV0 + kV * kTile;
  static constexpr int kRawV0 = kRawK0 + kRaw * kRawTile;
  static constexpr int kScale0 = kRawV0 + kRaw * kRawTile;   // (kV, 2, 128) fp32: K, V scales
  static constexpr int kHalf0 = kScale0 + (Q8 ? kV * 2 * kBN * 4 : 0);  // (128) float2
  static constexpr int kSmall0 = kHalf0 + (PAIR ? 0 : kBM * 8);
  static constexpr int kBytes = kSmall0 + 640;
  static_assert(kBytes <= 227 * 1024, "shared memory over the per-CTA limit");
  static_assert(kScale0 % 16 == 0 && kHalf0 % 16 == 0 && kSmall0 % 16 == 0, "16-byte accesses");
};
constexpr int kMaxStages = 6;
constexpr int kMaxRaw = 2;

enum {
  BAR_QF = 0,                    // Q tiles landed
  BAR_QE,                        // each half's last S of the segment is done (2 arrivals)
  BAR_KF,                        // + K stage: ready for the MMAs (landed, or widened by 4 warps)
  BAR_KE = BAR_KF + kMaxStages,  // + K stage: free (both halves' MMA threads)
  BAR_VL = BAR_KE + kMaxStages,  // + V stage: landed (bf16)
  BAR_VF = BAR_VL + kMaxStages,  // + V stage: in f16 (4 warps)
  BAR_VE = BAR_VF + kMaxStages,  // + V stage: free (PAIR: 2 arrivals)
  BAR_RKF = BAR_VE + kMaxStages,  // + raw stage: K codes landed
  BAR_RKE = BAR_RKF + kMaxRaw,    // + raw stage: K codes read (4 warps)
  BAR_RVF = BAR_RKE + kMaxRaw,
  BAR_RVE = BAR_RVF + kMaxRaw,
  BAR_S = BAR_RVE + kMaxRaw,     // + half: S ready
  BAR_SR = BAR_S + 2,            // + half: S read (4 warps)
  BAR_P = BAR_SR + 2,            // + 2 half + buffer: P written (4 warps)
  BAR_O = BAR_P + 4,             // + 2 half + buffer: P.V done
  BAR_E = BAR_O + 4,             // + half: O of the piece has been read (4 warps)
  BAR_ML = BAR_E + 2,            // second half's (max, sum) written (4 warps)
  BAR_X,                         // converting warps' maxima written (4 warps)
  BAR_DRAIN,                     // + half
  NBAR = BAR_DRAIN + 2
};
static_assert(NBAR * 8 + kMaxStages * 4 + 8 * 4 + 12 <= 640, "barriers and small arrays");

// Bounded waits that also give up when another role of the CTA has aborted: by
// one thread, and by a warp. (The timer is read and the flag looked at every 64
// tries, each of which suspends the warp for a while.)
__device__ __forceinline__ bool give_up(uint32_t i, unsigned long long& t0, volatile int* abort_flag,
                                        uint32_t* err) {
  if (i % 64 != 0) return false;
  if (*abort_flag) return true;
  const unsigned long long now = global_timer_ns();
  if (t0 == 0) t0 = now;
  if (now - t0 <= kWaitLimitNs) return false;
  *abort_flag = 1;
  report_error(err, PA_DEVERR_WAIT_TIMEOUT);
  return true;
}
__device__ __forceinline__ bool thread_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                            uint32_t* err) {
  unsigned long long t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i)
    if (give_up(i, t0, abort_flag, err)) return false;
  return true;
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          uint32_t* err) {
  unsigned long long t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1; !__all_sync(kFull, mbar_try_wait(bar, parity)); ++i)
    if (__any_sync(kFull, give_up(i, t0, abort_flag, err))) return false;
  return true;
}

__device__ __forceinline__ float pow2i(int k) {  // 2^k, k in [-126, 127]
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// Two f16 -> two bf16 (of 8-bit codes: exact).
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack_bf16x2(f.x, f.y);
}

template <int D, int BS, int KV, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    shared_keys_kernel(const __grid_constant__ CUtensorMap qmap,
                       const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const SharedArgs a) {
  constexpr bool Q8 = KV != kKvBf16;
  using R = Ring<D, Q8, PAIR>;
  constexpr int kTile = R::kTile, kBlocks = kBN / BS;
  constexpr int kCols = D / 32;  // 32-column chunks of O
  constexpr int kStep = PAIR ? 1 : 2;  // key tiles from one of a half's to its next
  extern __shared__ __align__(1024) uint8_t smem_raw[];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.group, TPT = a.tokens_per_tile;
  // The launch before this one (each sequence's own keys) let it start only
  // after the plan was complete, and works beside it: its results are waited
  // for at the end, on behalf of the merge.
  // (The merge waits for all of this launch: it may be launched at any time.)
  grid_launch_dependents();
  PieceWalk walk(a);
  const uint32_t base = smem_addr(smem_raw);
  if (walk.u >= walk.u1 || (base & 1023u) != 0) {  // (swizzled tiles need the alignment asked for)
    if (walk.u < walk.u1 && threadIdx.x == 0) report_error(a.err, PA_DEVERR_WAIT_TIMEOUT);
    grid_dependency_wait();
    return;
  }
  auto q_s = [&](int i) { return base + R::kQ0 + i * kTile; };
  auto k_s = [&](int s) { return base + R::kK0 + s * kTile; };
  auto v_s = [&](int s) { return base + R::kV0 + s * kTile; };
  float* const scales = reinterpret_cast<float*>(smem_raw + R::kScale0);
  float2* const half_ml = reinterpret_cast<float2*>(smem_raw + R::kHalf0);
  uint32_t* const cmax = reinterpret_cast<uint32_t*>(smem_raw + R::kSmall0);  // (2, 4), read by fours
  uint64_t* const bars = reinterpret_cast<uint64_t*>(cmax + 8);
  int* const fac = reinterpret_cast<int*>(bars + NBAR);  // (kV) V's factor is 2^fac
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(fac + kMaxStages);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* const half_k = reinterpret_cast<int*>(tmem_slot + 2);  // the second half's factor
  const uint32_t bar0 = smem_addr(bars);
  auto bar = [&](int i) { return bar0 + 8u * i; };
  if (threadIdx.x == 0) {
    for (int i = 0; i < NBAR; ++i) {
      const bool warps4 = (i >= BAR_VF && i < BAR_VE) || (i >= BAR_SR && i < BAR_O) ||
                          (i >= BAR_E && i <= BAR_X) || (i >= BAR_RKE && i < BAR_RVF) ||
                          (i >= BAR_RVE && i < BAR_S) || (Q8 && i >= BAR_KF && i < BAR_KE);
      const bool both = i == BAR_QE || (i >= BAR_KE && i < BAR_VL) ||
                        (PAIR && i >= BAR_VE && i < BAR_RKF);
      mbar_init(bar(i), warps4 ? 4 : both ? 2 : 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 9) {
    tc::tmem_alloc(smem_addr(tmem_slot), 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // of half i: S (64 columns), two buffers of P (32 each), O. S is free as soon as
  // the softmax warps have read it, so the next S is made while they work on it.
  auto tS = [&](int i) { return tmem + 128u * i; };
  auto tP = [&](int i, uint32_t b) { return tmem + 128u * i + 64u + 32u * b; };
  auto tO = [&](int i) { return tmem + 256u + 128u * i; };
  auto wait = [&](int b, uint32_t parity) { return warp_wait(bar(b), parity, abort_flag, a.err); };

  Piece p;
  if (warp >= 12) {
    // ------------------------------------------------------------ conversion
    // V into f16 (times a power of two), where P as one f16 term is precise
    // enough; 8-bit codes into bf16 (K) and f16 (V), exactly.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
    const int tid = threadIdx.x - 384;  // and, of 8-bit codes, the thread's key of the tile
    uint32_t c = 0;  // key tiles so far
    int k = 0;       // log2 of V's factor, or of the V scales'
    uint32_t xc = 0;  // maxima taken so far
    bool ok = true;
    // the largest of the four warps' values
    auto all_max = [&](uint32_t v) {
      v = __reduce_max_sync(kFull, v);
      const uint32_t b = xc++ & 1;
      if (lane == 0) {
        cmax[b * 4 + (warp - 12)] = v;
        mbar_arrive(bar(BAR_X));
      }
      ok = wait(BAR_X, b);
      const uint4 m = *reinterpret_cast<const uint4*>(cmax + b * 4);
      return max(max(m.x, m.y), max(m.z, m.w));
    };
    // keep the factor while it puts the tile's largest value (bits of a positive
    // float) at 2^lo .. 2^(hi + 1), else move the value to 2^mid. Within a piece it
    // rises to no more than 2^70 times its smallest: O, below 2^47 in f16 products of
    // at most 2^30, is multiplied by that and stays finite. (What is then lost is
    // below 2^-90 of the piece's largest value.)
    constexpr int kRise = 70;
    int k_min = 1 << 20;
    auto move_factor = [&](uint32_t bits, int lo, int hi, int mid) {
      if (bits != 0) {
        const int e = static_cast<int>(bits >> 23) - 127;
        if (e + k < lo || e + k > hi) k = min(max(mid - e, -120), 80);
      }
      k = min(k, k_min + kRise);
      k_min = min(k_min, k);
    };
    auto publish = [&](int b) {  // this warp's writes to a stage, to the MMAs
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
    };
    while (ok && walk.next(a, p)) {
      k_min = 1 << 20;
      float ks = 0.f, vs = 0.f;  // Q8: scales of this thread's key
      int phys1 = -1;            // its block in the next tile
      const long long bt_row = static_cast<long long>(p.owner) * a.max_blocks;
      auto block_of = [&](int t) {
        const int key = t * kBN + tid;
        return t < p.t1 && key < p.keys ? __ldg(a.block_tables + bt_row + key / BS) : -1;
      };
      auto load_scales = [&](int phys) {
        ks = vs = 0.f;
        if (phys >= 0 && phys < a.num_blocks) {
          const long long i = (static_cast<long long>(phys) * a.num_kv_heads + p.kvh) * BS + tid % BS;
          ks = a.k_scale[i];
          vs = a.v_scale[i];
        }
      };
      if constexpr (Q8) {
        load_scales(block_of(p.t0));
        phys1 = block_of(p.t0 + 1);
      }
      for (int t = p.t0; ok && t < p.t1; ++t, ++c) {
        const int sv = c % R::kV;
        if constexpr (!Q8) {
          constexpr int N = kTile / 16 / 128;
          ok = wait(BAR_VL + sv, (c / R::kV) & 1);
          if (!ok) break;
          uint4* const tile = reinterpret_cast<uint4*>(smem_raw + R::kV0 + sv * kTile) + tid;
          // (read once: the MMAs leave shared memory little room, see above)
          uint4 x[N];
          uint32_t m = 0;  // largest |V| so far, two bf16 side by side
#pragma unroll
          for (int i = 0; i < N; ++i) {
            x[i] = tile[128 * i];
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                     __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
          }
          m = all_max(max(m >> 16, m & 0xffffu));
          if (ok && m >= 0x7f80u) {  // some V is not finite: the largest of the others
            m = 0;
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
              const uint4 y = tile[128 * i];
              const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t a0 = w[j] & 0x7fffu, a1 = (w[j] >> 16) & 0x7fffu;
                m = max(m, max(a0 < 0x7f80u ? a0 : 0u, a1 < 0x7f80u ? a1 : 0u));
              }
            }
            m = all_max(m);
          }
          if (!ok) break;
          move_factor(m << 16, 6, 14, 11);
          const uint64_t f2 = tc::f32x2(pow2i(k), pow2i(k));
          auto widen = [&](uint32_t w) {
            float lo, hi;
            tc::f32x2_split(tc::mul_f32x2(tc::f32x2(__uint_as_float(w << 16),
                                                    __uint_as_float(w & 0xffff0000u)), f2), lo, hi);
            return pack_f16x2(lo, hi);
          };
#pragma unroll
          for (int i = 0; i < N; ++i)
            tile[128 * i] = make_uint4(widen(x[i].x), widen(x[i].y), widen(x[i].z), widen(x[i].w));
          if (tid == 0) fac[sv] = k;
          publish(BAR_VF + sv);
        } else {
          // a thread's key: 128 codes, 16-byte chunk j of row tid at j ^ (tid & 7)
          const int rs = c % R::kRaw, sk = c % R::kK;
          auto read_raw = [&](int raw0, int full, int empty, uint4 (&x)[8]) {
            ok = wait(full + rs, (c / R::kRaw) & 1);
            const uint8_t* row = smem_raw + raw0 + rs * R::kRawTile + tid * 128;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              x[j] = *reinterpret_cast<const uint4*>(row + ((j ^ (tid & 7)) << 4));
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(empty + rs));
          };
          auto write_row = [&](uint8_t* tile, const uint4 (&x)[8], auto&& widen) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // 16 dims: chunks 2 j, 2 j + 1 of the 16-bit row
              uint8_t* row = tile + (j >> 2) * kSub + tid * 128;
              uint4 lo, hi;
              widen(x[j].x, lo.x, lo.y);
              widen(x[j].y, lo.z, lo.w);
              widen(x[j].z, hi.x, hi.y);
              widen(x[j].w, hi.z, hi.w);
              const int ch = 2 * (j & 3);
              *reinterpret_cast<uint4*>(row + ((ch ^ (tid & 7)) << 4)) = lo;
              *reinterpret_cast<uint4*>(row + (((ch + 1) ^ (tid & 7)) << 4)) = hi;
            }
          };
          uint4 x[8];
          read_raw(R::kRawK0, BAR_RKF, BAR_RKE, x);
          ok = ok && (c < R::kK || wait(BAR_KE + sk, (c / R::kK - 1) & 1));
          if (!ok) break;
          write_row(smem_raw + R::kK0 + sk * kTile, x, [](uint32_t w, uint32_t& lo, uint32_t& hi) {
            codes8x4_to_f16x2x2<KV>(w, lo, hi);
            lo = f16x2_to_bf16x2(lo);
            hi = f16x2_to_bf16x2(hi);
          });
          publish(BAR_KF + sk);
          read_raw(R::kRawV0, BAR_RVF, BAR_RVE, x);
          ok = ok && (c < R::kV || wait(BAR_VE + sv, (c / R::kV - 1) & 1));
          if (!ok) break;
          write_row(smem_raw + R::kV0 + sv * kTile, x, [](uint32_t w, uint32_t& lo, uint32_t& hi) {
            codes8x4_to_f16x2x2<KV>(w, lo, hi);
          });
          // (a scale that is not finite spoils its rows, not the factor)
          const uint32_t vb = __float_as_uint(vs) & 0x7fffffffu;
          const uint32_t m = all_max(vb < 0x7f800000u ? vb : 0u);
          if (!ok) break;
          move_factor(m, 2, 6, 5);
          scales[(2 * sv) * kBN + tid] = ks;
          scales[(2 * sv + 1) * kBN + tid] = vs * pow2i(k);
          if (tid == 0) fac[sv] = k;
          publish(BAR_VF + sv);
          load_scales(phys1);
          phys1 = block_of(t + 2);
        }
      }
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
    if (warp == 8 || warp == 10) {
      // ---------------------------------------------------------- Q and K, V producers
      const bool is_k = warp == 8;
      const CUtensorMap* map = is_k ? &kmap : &vmap;
      const int ST = Q8 ? R::kRaw : is_k ? R::kK : R::kV;
      const int full0 = Q8 ? (is_k ? BAR_RKF : BAR_RVF) : is_k ? BAR_KF : BAR_VL;
      const int empty0 = Q8 ? (is_k ? BAR_RKE : BAR_RVE) : is_k ? BAR_KE : BAR_VE;
      const uint32_t dst0 = base + (Q8 ? (is_k ? R::kRawK0 : R::kRawV0) : is_k ? R::kK0 : R::kV0);
      constexpr int kBytes = Q8 ? R::kRawTile : kTile;
      constexpr int kSubs = Q8 ? 1 : D / 64;  // 128-byte columns of a row
      const int oob = a.num_blocks * BS;  // first row past the pool: TMA fills zeros
      uint32_t c = 0, s = 0, round = 0;   // tiles so far; stage and use of it
      uint32_t n = 0;                     // Q loads so far
      bool ok = true;
      while (ok && walk.next(a, p)) {
        if (is_k) {
          if (n > 0 && !wait(BAR_QE, (n - 1) & 1)) break;
          const int tiles = PAIR && p.tok0 + TPT < p.tok1 ? 2 : 1;
          if (tc::elect_one()) {
            // a box is G heads of TPT tokens: TPT * G rows of 128 bytes
            mbar_arrive_expect_tx(bar(BAR_QF), tiles * (D / 64) * TPT * G * 128);
            for (int i = 0; i < tiles; ++i)
              for (int h = 0; h < D / 64; ++h)
                tma_load_3d(q_s(i) + h * kSub, &qmap, bar(BAR_QF), 64 * h, p.kvh * G,
                            p.tok0 + i * TPT);
          }
          __syncwarp();
          ++n;
        }
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
          if (round > 0 && !wait(empty0 + s, (round - 1) & 1)) {
            ok = false;
            break;
          }
          const uint32_t dst = dst0 + s * kBytes, full = bar(full0 + s);
          int rc[kBlocks];
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) rc[i] = __shfl_sync(kFull, ids, t * kBlocks - wb + i);
          if (tc::elect_one()) {
            mbar_arrive_expect_tx(full, kBytes);
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
#pragma unroll
              for (int h = 0; h < kSubs; ++h)
                tma_load_3d(dst + h * kSub + i * BS * 128, map, full, 64 * h, p.kvh, rc[i]);
          }
          __syncwarp();
          if (++s == ST) {
            s = 0;
            ++round;
          }
        }
      }
      if (*abort_flag) {
        // let the copies already in flight land before shared memory is released
        if (n > 0) (void)mbar_wait(bar(BAR_QF), (n - 1) & 1);
        for (uint32_t j = c > ST ? c - ST : 0; j < c; ++j)
          (void)mbar_wait(bar(full0 + j % ST), (j / ST) & 1);
      }
    } else {
      // ---------------------------------------------------------- MMA issue
      // One warp a half, one thread of it from end to end: between two MMAs the
      // tensor pipe only has what is queued, and every warp-wide step in between,
      // or a wait for the other half, costs some of that.
      if (tc::elect_one()) {
        const int i = warp == 9 ? 0 : 1;
        auto wait = [&](int b, uint32_t parity) {
          return thread_wait(bar(b), parity, abort_flag, a.err);
        };
        constexpr uint32_t kIdescQK = tc::idesc_f32(kBM, kSN, tc::kBf16, false, false);
        constexpr uint32_t kIdescPV = tc::idesc_f32(kBM, D, tc::kF16, false, true);
        constexpr int kStepDesc = kSN * 128 >> 4;  // from a tile's first 64 keys to its others
        const uint64_t q = tc::smem_desc_sw128(q_s(PAIR ? i : 0), 16, 1024);
        uint32_t xs = 0, xp = 0;  // steps of this half so far: S issued, P.V issued
        uint32_t pieces = 0;      // of this half, so far
        uint32_t c = 0;           // key tiles before the piece
        // A barrier is asked for its phases one after the other, and none may pass
        // unseen (the parity would be that of another). So K tiles are waited for in
        // turn, also those the other half takes (the copies may land in any order),
        // and every stage is given back by both threads. V tiles are converted in
        // turn, and a half's own are never more than three apart; with two V stages
        // (8-bit codes) S of a tile implies that V of the tile before is there.
        uint32_t kw = 0;
        auto wait_k = [&](uint32_t tile) {
          for (; kw <= tile; ++kw) {
            const uint32_t s = kw % R::kK;
            if (!wait(BAR_KF + s, (kw / R::kK) & 1)) return false;
            if (kw < tile) mbar_arrive(bar(BAR_KE + s));  // the other half's
          }
          return true;
        };
        bool ok = true;
        for (uint32_t n = 0; ok && walk.next(a, p); ++n) {
          const int T = p.t1 - p.t0;
          const bool mine = i == 0 || (PAIR ? p.tok0 + TPT < p.tok1 : T > 1);
          auto steps_of = [&](int t) { return p.keys - (p.t0 + t) * kBN > kSN ? 2 : 1; };
          ok = wait(BAR_QF, n & 1);
          if (!mine) {  // stages need this half's arrivals all the same
            for (int t = 0; ok && t < T; ++t) {
              const uint32_t vs = (c + t) % R::kV;
              ok = wait_k(c + t);
              if (ok) mbar_arrive(bar(BAR_KE + (c + t) % R::kK));
              ok = ok && wait(BAR_VF + vs, ((c + t) / R::kV) & 1);
              if (ok && PAIR) mbar_arrive(bar(BAR_VE + vs));
            }
            if (ok) mbar_arrive(bar(BAR_QE));
            c += T;
            continue;
          }
          // The next S in the order of this half's key tiles t (PAIR: all; else i,
          // i + 2, ...) and their steps h, once the one before has been read.
          int st = PAIR ? 0 : i, sh = 0;
          auto issue_s = [&]() {
            const uint32_t cs = c + st, s = cs % R::kK;
            if (!wait_k(cs)) return false;
            if (xs > 0 && !wait(BAR_SR + i, (xs - 1) & 1)) return false;
            ++xs;
            const uint64_t k = tc::smem_desc_sw128(k_s(s), 16, 1024) + sh * kStepDesc;
            const uint32_t d = tS(i);
            tc::fence_after_sync();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              // (a descriptor's low bits are the address in units of 16 bytes)
              const int off = ((kk >> 2) * kSub + (kk & 3) * 32) >> 4;
              tc::mma_ss(d, q + off, k + off, kIdescQK, kk > 0 ? 1u : 0u);
            }
            tc::commit(bar(BAR_S + i));
            if (++sh == steps_of(st)) {
              tc::commit(bar(BAR_KE + s));
              sh = 0;
              st += kStep;
              if (st >= T) tc::commit(bar(BAR_QE));
            }
            return true;
          };
          ok = ok && issue_s();
          for (int t = PAIR ? 0 : i; ok && t < T; t += kStep) {
            const uint32_t cv = c + t, s = cv % R::kV;
            const int steps = steps_of(t);
#pragma unroll 1
            for (int h = 0; ok && h < steps; ++h) {
              if (st < T) ok = issue_s();
              ok = ok && (h > 0 || wait(BAR_VF + s, (cv / R::kV) & 1));
              // O (+)= P V for 64 keys
              const uint32_t b = 2 * i + (xp & 1);
              const bool first = t < kStep && h == 0;
              ok = ok && wait(BAR_P + b, (xp >> 1) & 1) &&
                   (!first || pieces == 0 || wait(BAR_E + i, (pieces - 1) & 1));
              if (!ok) break;
              const uint64_t v = tc::smem_desc_sw128(v_s(s), kSub, 1024) + h * kStepDesc;
              const uint32_t d = tO(i), pa = tP(i, xp & 1);
              ++xp;
              tc::fence_after_sync();
#pragma unroll
              for (int kk = 0; kk < kSN / 16; ++kk)
                tc::mma_ts(d, pa + kk * 8, v + kk * (16 * 128 >> 4), kIdescPV,
                           !first || kk > 0 ? 1u : 0u);
              tc::commit(bar(BAR_O + b));
            }
            if (ok) tc::commit(bar(BAR_VE + s));
          }
          c += T;
          ++pieces;
        }
        if (*abort_flag) {  // no MMA may still run when TMEM is freed
          tc::commit(bar(BAR_DRAIN + i));
          (void)mbar_wait(bar(BAR_DRAIN + i), 0);
        }
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------------------ softmax
    const int hf = warp / 4;  // half: row tile (PAIR) or taker of every other key tile
    const int r = 32 * (warp & 3) + lane;  // row of the tile = TMEM lane
    const uint32_t trow = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const float sl2 = a.scale_log2;
    // P's f16 holds 2^(score - max) times 2^7 (bf16) or times the V scale at up to
    // 2^7: at most 2^15 with the threshold above, and nothing below 2^-31 of the
    // row's largest is lost. The sum l takes the same 2^7.
    constexpr float kLift = Q8 ? 0.f : 7.f;
    uint32_t x = 0;       // steps of this half so far: P buffer x & 1 for the (x >> 1)-th time
    uint32_t other = 0;   // first half, one row tile: steps of the second half so far
    uint32_t merged = 0;  // pieces in which the second half had tiles
    uint32_t c0 = 0;      // key tiles before the piece
    bool ok = true;
    for (int T; ok && walk.next(a, p); c0 += T) {
      T = p.t1 - p.t0;
      if (PAIR && hf == 1 && p.tok0 + TPT >= p.tok1) continue;  // one row tile in this segment
      const int tok = p.tok0 + (PAIR ? hf * TPT : 0) + r / G;
      const bool valid = r < TPT * G && tok < p.tok1;
      const int lim = valid ? min(p.keys, __ldcg(a.plan.row_vis + tok)) : p.keys;  // keys the row sees
      float m_used = -INFINITY, l = 0.f;
      int k = 0;  // O holds the sum times 2^k
      // steps (64 keys) of the piece; this half's: with one row tile, both of every other tile's
      const int steps = (min(p.t1 * kBN, p.keys) - p.t0 * kBN + kSN - 1) / kSN;
      const uint32_t x0 = x;
      for (int st = PAIR ? 0 : 2 * hf; st < steps; st += !PAIR && (st & 1) ? 3 : 1, ++x) {
        const uint32_t S = tS(hf) + trow;
        const bool begin = x == x0;
        const uint32_t ct = c0 + (st >> 1);
        const int sv = ct % R::kV;
        ok = wait(BAR_S + hf, x & 1);
        if (!ok) break;
        tc::fence_after_sync();
        uint32_t u[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tc::tmem_ld32(S + 32 * c, u[c]);
        // (S on its way) the tile's V is converted: its factor and scales are there
        // (asked for only after S: V of the tiles before is then known to be)
        if ((st & 1) == 0) ok = wait(BAR_VF + sv, (ct / R::kV) & 1);
        const int k_new = fac[sv];
        const float* const sc = scales + (2 * sv) * kBN + (st & 1) * kSN;
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (!ok) break;
        if (lane == 0) mbar_arrive(bar(BAR_SR + hf));
        if constexpr (Q8) {  // K scales
#pragma unroll
          for (int j = 0; j < kSN; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(sc + j);
            uint32_t* w = &u[j >> 5][j & 31];
            auto mul2 = [&](int e, float f0, float f1) {
              float x0, x1;
              tc::f32x2_split(tc::mul_f32x2(tc::f32x2(__uint_as_float(w[e]), __uint_as_float(w[e + 1])),
                                            tc::f32x2(f0, f1)), x0, x1);
              w[e] = __float_as_uint(x0);
              w[e + 1] = __float_as_uint(x1);
            };
            mul2(0, f.x, f.y);
            mul2(2, f.z, f.w);
          }
        }
        const int left = lim - p.t0 * kBN - st * kSN;  // keys of this step the row sees
        if (!__all_sync(kFull, left >= kSN)) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * c + j >= left) u[c][j] = __float_as_uint(-INFINITY);
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 32; ++j)
          mx[j & 3] = fmaxf(mx[j & 3], fmaxf(__uint_as_float(u[0][j]), __uint_as_float(u[1][j])));
        // (the scale is positive)
        const float m_step = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
        if (begin) {
          m_used = m_step;
          k = k_new;
        } else if (k_new != k || __any_sync(kFull, valid && m_step > m_used + kRescaleThreshold)) {
          // raise the maximum, or follow V's factor: rescale O once its last product is done
          // (for rows of the group only: where 128 is no multiple of G, the tile's last rows
          // of Q hold what another CTA left there, which must not decide how these round)
          ok = wait(BAR_O + 2 * hf + ((x - 1) & 1), ((x - 1) >> 1) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          const float m_new = fmaxf(m_used, m_step);
          // (a row that has seen no key yet has nothing to rescale)
          const float alpha = m_new == -INFINITY ? 1.f : fast_exp2(m_used - m_new);
          const float beta = alpha * pow2i(min(max(k_new - k, -126), 126));
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            tc::tmem_ld32(tO(hf) + trow + 32 * c, w);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) * beta);
            tc::tmem_st32(tO(hf) + trow + 32 * c, w);
          }
          tc::tmem_wait_st();
          l *= alpha;
          m_used = m_new;
          k = k_new;
        }
        // P = 2^(s * scale * log2(e) - m_used) in f16; pairs of keys share one
        // packed FMA and one packed add
        const float nm = m_used == -INFINITY ? 0.f : kLift - m_used;
        const uint64_t sl2x2 = tc::f32x2(sl2, sl2), nmx2 = tc::f32x2(nm, nm);
        uint64_t lsum[2] = {tc::f32x2(0.f, 0.f), tc::f32x2(0.f, 0.f)};
        uint32_t w[32];
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          float4 f;
          if constexpr (Q8) f = *reinterpret_cast<const float4*>(sc + kBN + 2 * j);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t* e = &u[j >> 4][2 * ((j + i) & 15)];
            const uint64_t y = tc::fma_f32x2(
                tc::f32x2(__uint_as_float(e[0]), __uint_as_float(e[1])), sl2x2, nmx2);
            float p0, p1;
            tc::f32x2_split(y, p0, p1);
            p0 = fast_exp2(p0);
            p1 = fast_exp2(p1);
            const uint64_t pp = tc::f32x2(p0, p1);
            lsum[i] = tc::add_f32x2(lsum[i], pp);
            if constexpr (Q8)  // V scales, times 2^k
              tc::f32x2_split(tc::mul_f32x2(pp, i ? tc::f32x2(f.z, f.w) : tc::f32x2(f.x, f.y)), p0, p1);
            w[j + i] = pack_f16x2(p0, p1);
          }
        }
        // (The buffer's P of two steps ago has been used: its product was issued
        // before this step's S by the same thread, whose commit of S covers it.)
        tc::tmem_st32(tP(hf, x & 1) + trow, w);
        float la, lb;
        tc::f32x2_split(tc::add_f32x2(lsum[0], lsum[1]), la, lb);
        l += la + lb;
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_P + 2 * hf + (x & 1)));
      }
      if (!ok) break;
      // ---- the piece's partial: (max, sum) and O, unnormalised, without P's lift
      // and V's factor (powers of two)
      const int lift = static_cast<int>(kLift);
      l *= pow2i(-lift);
      float f0 = pow2i(-k - lift), f1 = 0.f;
      const bool both = !PAIR && T > 1;
      if constexpr (!PAIR) {
        if (both) {
          if (hf == 1) {
            // (the first half has read the piece before's once that O is released)
            ok = merged == 0 || wait(BAR_E + 1, (merged - 1) & 1);
            if (!ok) break;
            half_ml[r] = make_float2(m_used, l);
            if (r == 0) *half_k = k;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(BAR_ML));
            ++merged;
            continue;  // the first half reads this half's O, in the same TMEM lanes
          }
          other += steps - static_cast<int>(x - x0);
          ok = wait(BAR_ML, merged & 1) &&
               wait(BAR_O + 2 + ((other - 1) & 1), ((other - 1) >> 1) & 1);
          if (!ok) break;
          const float2 o = half_ml[r];
          ++merged;
          const float m = fmaxf(m_used, o.x);
          const float e0 = m_used == -INFINITY ? 0.f : fast_exp2(m_used - m);
          const float e1 = o.x == -INFINITY ? 0.f : fast_exp2(o.x - m);
          f0 *= e0;
          f1 = e1 * pow2i(-*half_k - lift);
          l = l * e0 + o.y * e1;
          m_used = m;
        } else if (hf == 1) {
          continue;
        }
      }
      ok = wait(BAR_O + 2 * hf + ((x - 1) & 1), ((x - 1) >> 1) & 1);
      if (!ok) break;
      tc::fence_after_sync();
      const long long row = p.slot * (kBM * a.row_tiles) + (PAIR ? hf * kBM : 0) + r;
      float* const dst = a.part_o + row * D;
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
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) * f0);
        }
        if (valid) {
#pragma unroll
          for (int j = 0; j < 4; ++j) st_global_32(dst + 32 * c + 8 * j, w + 8 * j);
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

// Every query head of a row and kv head: the parts of the shared keys and the
// row's own keys' result, folded into a running (max, sum, O). O of a head is on
// D/4 lanes, 16 bytes each; such a team of lanes takes some heads at a time, so
// that the look-up of the parts is shared and their reads are under way together.
// WIDE: all teams of the CTA share a row's parts, team s taking the parts s, s +
// teams, ..., and fold each other's results through shared memory; otherwise
// every team has a row of its own.
template <int D, bool WIDE>
__global__ void __launch_bounds__(kMergeWarps * 32, WIDE ? 4 : 8)
    shared_merge_kernel(const SharedArgs a) {
  constexpr int LPR = D / 4, kTeams = kMergeWarps * 32 / LPR;
  constexpr int kHeads = WIDE ? 4 : 2;  // at a time
  __shared__ float2 team_ml[WIDE ? kTeams : 1][kHeads];
  __shared__ float4 team_o[WIDE ? kTeams : 1][kHeads][WIDE ? LPR : 1];
  grid_dependency_wait();
  grid_launch_dependents();
  const int team = threadIdx.x / LPR, sub = threadIdx.x % LPR;
  const long long w = WIDE ? blockIdx.x : static_cast<long long>(blockIdx.x) * kTeams + team;
  if (w >= static_cast<long long>(a.rows) * a.num_kv_heads) return;
  const int t = static_cast<int>(w / a.num_kv_heads), kvh = static_cast<int>(w % a.num_kv_heads);
  const int vis = a.plan.row_vis[t], g = a.plan.row_grp[t], start = a.plan.row_start[t];
  // (no own keys: what is left here from another call is not used)
  int2 mine = make_int2(-1, 1);
  if (a.own_parts != nullptr) mine = a.own_parts[w];
  // (a row that shares nothing is written by the prefill kernel)
  if (vis < 0 || (a.own_parts == nullptr && g < 0)) return;
  const bool own = vis > start;

  // ---- the row's parts of the shared keys, then those of its own
  long long first = 0;  // row of the first
  int n = 0;
  const long long step = kBM * a.row_tiles;
  if (g >= 0) {
    const int per_seg = a.tokens_per_tile * a.row_tiles;
    const int i = t - a.plan.tok[2 * g], rows = a.plan.tok[2 * g + 1] - a.plan.tok[2 * g];
    const int R = (rows + per_seg - 1) / per_seg, q = i % per_seg;
    const int2 parts = a.plan.parts[a.plan.seg[g] + kvh * R + i / per_seg];
    first = parts.x * step + q / a.tokens_per_tile * kBM + q % a.tokens_per_tile * a.group;
    n = parts.y;
  }
  const long long rh = static_cast<long long>(t) * a.num_heads + kvh * a.group;
  // own part j: in own_o, or in the decode kernel's slots (the segment's first
  // part is in its warp's odd one)
  const float2* own_ml = a.own_ml + rh;
  const float* own_o = a.own_o + rh * D;
  if (own && mine.x >= 0) {
    own_ml = a.slot_ml + (2LL * mine.x + 1) * a.slot_rows;
    own_o = a.slot_o + (2LL * mine.x + 1) * a.slot_rows * D;
  }
  const int n_own = own ? mine.y : 0;
  // Part 0 is read ahead of the shared keys' parts (WIDE: by the team that has the
  // fewest of those); parts j > 0 lie 2 j - 1 slots further.
  const int own_team = WIDE ? n % kTeams : 0;
  for (int h0 = 0; h0 < a.group; h0 += kHeads) {
    float M[kHeads], L[kHeads];
    float4 acc[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      M[h] = -INFINITY;
      L[h] = 0.f;
      acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    auto fold = [&](int h, const float2& ml, const float4& x) {
      const float m = fmaxf(M[h], ml.x);
      // (nothing so far, or nothing in this part: a factor of 0, not of 2^(inf - inf))
      const float f0 = M[h] == -INFINITY ? 0.f : fast_exp2(M[h] - m);
      const float f1 = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - m);
      M[h] = m;
      L[h] = L[h] * f0 + ml.y * f1;
      acc[h].x = acc[h].x * f0 + x.x * f1;
      acc[h].y = acc[h].y * f0 + x.y * f1;
      acc[h].z = acc[h].z * f0 + x.z * f1;
      acc[h].w = acc[h].w * f0 + x.w * f1;
    };
    auto read = [&](const float2* ml, const float* o, float2 (&m)[kHeads], float4 (&x)[kHeads]) {
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
        if (h0 + h < a.group) {
          m[h] = __ldcg(ml + h0 + h);
          x[h] = __ldcg(reinterpret_cast<const float4*>(o + static_cast<long long>(h0 + h) * D) + sub);
        }
    };
    auto fold_all = [&](const float2 (&m)[kHeads], const float4 (&x)[kHeads]) {
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
        if (h0 + h < a.group) fold(h, m[h], x[h]);
    };
    const bool have_own = n_own > 0 && (!WIDE || team == own_team);
    float2 om[kHeads];
    float4 ox[kHeads];
    if (have_own) read(own_ml, own_o, om, ox);
#pragma unroll 2
    for (int j = WIDE ? team : 0; j < n; j += WIDE ? kTeams : 1) {
      const long long row = first + j * step;
      float2 m[kHeads];
      float4 x[kHeads];
      read(a.part_ml + row, a.part_o + row * D, m, x);
      fold_all(m, x);
    }
    if (have_own) fold_all(om, ox);
#pragma unroll 1
    for (int j = 1; j < n_own; ++j) {
      if (WIDE && (j + own_team) % kTeams != team) continue;
      const long long row = (2LL * j - 1) * a.slot_rows;
      float2 m[kHeads];
      float4 x[kHeads];
      read(own_ml + row, own_o + row * D, m, x);
      fold_all(m, x);
    }
    if constexpr (WIDE) {
      if (h0 > 0) __syncthreads();  // the heads before have been read
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        if (sub == 0) team_ml[team][h] = make_float2(M[h], L[h]);
        team_o[team][h][sub] = acc[h];
      }
      __syncthreads();
    }
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      if (h0 + h >= a.group) break;
      if (WIDE && h != team) continue;  // (there are at least four teams)
      if constexpr (WIDE) {
        for (int s = 0; s < kTeams; ++s)
          if (s != team) fold(h, team_ml[s][h], team_o[s][h][sub]);
      }
      // no keys: zeros; a NaN stays
      const float inv = L[h] > 0.f ? 1.f / L[h] : L[h];
      uint2 o;
      o.x = pack_bf16x2(acc[h].x * inv, acc[h].y * inv);
      o.y = pack_bf16x2(acc[h].z * inv, acc[h].w * inv);
      reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (rh + h0 + h) * D)[sub] = o;
    }
  }
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

template <int D, int BS, int KV, bool PAIR>
cudaError_t launch_keys_inst(const SharedArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                        const CUtensorMap& vmap, cudaStream_t stream) {
  auto* k = shared_keys_kernel<D, BS, KV, PAIR>;
  constexpr int smem = Ring<D, KV != kKvBf16, PAIR>::kBytes;
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

template <int D, int KV>
cudaError_t launch_keys(const SharedArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                        const CUtensorMap& vmap, cudaStream_t stream) {
  const bool pair = a.row_tiles == 2;
  if (a.block_size == 16)
    return pair ? launch_keys_inst<D, 16, KV, true>(a, qmap, kmap, vmap, stream)
                : launch_keys_inst<D, 16, KV, false>(a, qmap, kmap, vmap, stream);
  return pair ? launch_keys_inst<D, 32, KV, true>(a, qmap, kmap, vmap, stream)
              : launch_keys_inst<D, 32, KV, false>(a, qmap, kmap, vmap, stream);
}

long long query_tiles(int rows, int tokens_per_tile) {
  return (rows + static_cast<long long>(tokens_per_tile) - 1) / tokens_per_tile;
}

// The layout of a call with `row_tiles` tiles a segment.
SharedLayout layout_of(size_t base, int rows, int num_heads, int num_kv_heads, int head_dim,
                       int num_groups, int num_sms, int row_tiles) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  SharedLayout l{};
  l.tokens_per_tile = kBM / (num_heads / num_kv_heads);
  l.row_tiles = row_tiles;
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
                            static_cast<size_t>(l.max_segments) * sizeof(int2) +
                            3 * static_cast<size_t>(rows) * sizeof(int);
  l.part_ml = up(l.plan + plan_bytes);
  l.part_o = up(l.part_ml + part_rows * sizeof(float2));
  l.own_parts = up(l.part_o + part_rows * head_dim * sizeof(float));
  l.own_ml = up(l.own_parts + static_cast<size_t>(rows) * num_kv_heads * sizeof(int2));
  l.own_o = up(l.own_ml + rh * sizeof(float2));
  l.bytes = l.own_o + rh * head_dim * sizeof(float) + 256;  // (to align the address)
  return l;
}

}  // namespace

SharedLayout shared_layout(size_t base, int rows, int num_heads, int num_kv_heads, int head_dim,
                           int num_groups, int num_sms) {
  // Two row tiles a segment where the groups have the rows for them on average:
  // a K/V tile then serves twice the rows. Smaller groups leave the second tile
  // empty, and are bound by reading the keys.
  const bool two = query_tiles(rows, kBM / (num_heads / num_kv_heads)) > std::max(num_groups, 1);
  return layout_of(base, rows, num_heads, num_kv_heads, head_dim, num_groups, num_sms, two ? 2 : 1);
}

// Either form takes more with more rows and with more groups, but a call of fewer
// groups may have two row tiles where one of more has one, and then twice the rows
// a partial: the larger of the two, with as many groups as each can have.
size_t shared_workspace_bytes(size_t base, int rows, int num_heads, int num_kv_heads, int head_dim,
                              int num_groups, int num_sms) {
  auto bytes = [&](int groups, int row_tiles) {
    return layout_of(base, rows, num_heads, num_kv_heads, head_dim, groups, num_sms, row_tiles).bytes;
  };
  const long long tiles = query_tiles(rows, kBM / (num_heads / num_kv_heads));
  const size_t one = bytes(num_groups, 1);
  if (tiles <= 1) return one;
  return std::max(one, bytes(static_cast<int>(std::min<long long>(num_groups, tiles - 1)), 2));
}

void shared_pointers(SharedArgs& a, const SharedLayout& l, void* workspace) {
  // the parts are at multiples of 256 bytes of the address (stores of 32)
  char* const ws = reinterpret_cast<char*>(
      (reinterpret_cast<uintptr_t>(workspace) + 255) & ~static_cast<uintptr_t>(255));
  const int g1 = a.num_groups + 1;
  a.plan.unit = reinterpret_cast<long long*>(ws + l.plan);
  a.plan.parts = reinterpret_cast<int2*>(a.plan.unit + g1);
  a.plan.cu = reinterpret_cast<int*>(a.plan.parts + l.max_segments);
  a.plan.keys = a.plan.cu + g1;
  a.plan.owner = a.plan.keys + g1;
  a.plan.seg = a.plan.owner + g1;
  a.plan.tok = a.plan.seg + g1;
  a.plan.row_vis = a.plan.tok + 2 * g1;
  a.plan.row_grp = a.plan.row_vis + a.rows;
  a.plan.row_start = a.plan.row_grp + a.rows;
  a.part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
  a.part_o = reinterpret_cast<float*>(ws + l.part_o);
  a.own_parts = a.context_lens != nullptr ? reinterpret_cast<int2*>(ws + l.own_parts) : nullptr;
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
  if (a.block_size != 16 && a.block_size != 32) return cudaErrorInvalidValue;
  if (a.kv == kKvE4m3) return launch_keys<128, kKvE4m3>(a, qmap, kmap, vmap, stream);
  if (a.kv == kKvInt8) return launch_keys<128, kKvInt8>(a, qmap, kmap, vmap, stream);
  return a.head_dim == 64 ? launch_keys<64, kKvBf16>(a, qmap, kmap, vmap, stream)
                          : launch_keys<128, kKvBf16>(a, qmap, kmap, vmap, stream);
}

// A row to a team needs enough rows to hide the chain of look-ups and reads of
// one: below 16 warps an SM, a row to a CTA.
cudaError_t launch_shared_merge(const SharedArgs& a, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.rows) * a.num_kv_heads;
  const long long teams = kMergeWarps * (128 / a.head_dim);
  const bool wide = rows < 16LL * a.ctas * (128 / a.head_dim);
  const long long grid = wide ? rows : (rows + teams - 1) / teams;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      config(dim3(static_cast<unsigned>(grid)), kMergeWarps * 32, 0, stream, attr);
  if (a.head_dim == 64)
    return wide ? cudaLaunchKernelEx(&cfg, shared_merge_kernel<64, true>, a)
                : cudaLaunchKernelEx(&cfg, shared_merge_kernel<64, false>, a);
  return wide ? cudaLaunchKernelEx(&cfg, shared_merge_kernel<128, true>, a)
              : cudaLaunchKernelEx(&cfg, shared_merge_kernel<128, false>, a);
}

}  // namespace pa
