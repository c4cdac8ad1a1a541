// norm_rope_store: per-head RMS norm of q and k, position rotation of both, and
// the store of the new K and V rows in their cache slots.
//
// What is computed, for token t at position p = positions[t], slot s =
// slot_mapping[t], in fp32 from the bf16 inputs:
//     n(x)_i = x_i * rsqrt(mean_j x_j^2 + eps) * weight_i      (weight given)
//     (a, b) -> (a cos - b sin, b cos + a sin)                 (dims < rotary_dim)
// with (cos, sin) of pair i from row p of the caller's table, and pair i either
// dims (i, i + rotary_dim/2) or (2i, 2i+1). q rows go to q_out (one rounding to
// bf16), k and v rows to the cache: bf16, or 8-bit codes c = round(x / sc) with
// sc = max|x| / 448 (E4M3) or / 127 (INT8) taken from the unrounded row.
//
// How: a row of head_dim elements belongs to head_dim/8 lanes with one 16-byte
// chunk each, so every load and store is a 16-byte vector and a warp holds 2
// (head_dim 128) or 4 rows at once. A warp's rows are of one kind (q, k or v).
// The norm is a shuffle sum over the row's lanes. The weight and the table
// entries are folded once per warp into two factors per element,
//     y_i = rstd * (x_i * A_i + x_partner(i) * B_i),
// A_i = w_i cos, B_i = -+ w_partner sin, so a row costs two multiply-adds per
// element and a half-split partner chunk is fetched from its lane as raw bf16
// (four shuffles). A warp's first row loads are issued before the table's, and a
// large call's warps read the next rows while they work on these.
//
// Bound by HBM for large calls: 16383 tokens of 32 + 8 + 8 rows of 128 (bf16, 407
// MB in and out) take 77 us on one GB300, 5.3 TB/s; about 140 instructions per
// 16-byte chunk (unpacking, norm, rotation, packing) keep more reads from being
// under way. Small calls are launch latency: 64 tokens 2.6 us in a CUDA graph.
#include "pa_device.cuh"
#include "pa_launch.h"
#include "pa_norm_rope.h"
#include "pa_tcgen05.cuh"

namespace pa {

namespace {

constexpr int kNrWarps = 4;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Two bf16 (one word) -> a packed pair of fp32.
__device__ __forceinline__ uint64_t unpack2(uint32_t w) {
  return tc::f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// max that keeps a NaN of either operand
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight fp32 -> eight 8-bit codes of kind KV (in order, low byte first).
// E4M3: round to nearest even, saturating at 448, NaN stays NaN. INT8: round
// to nearest even, clamped to +-127 (a NaN gives 0: its row's scale is NaN).
template <int KV>
__device__ __forceinline__ uint2 codes8(const float (&x)[8]) {
  if constexpr (KV == kKvE4m3) {
    uint16_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    return make_uint2(c[0] | (static_cast<uint32_t>(c[1]) << 16),
                      c[2] | (static_cast<uint32_t>(c[3]) << 16));
  } else {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = min(127, max(-127, __float2int_rn(x[i])));
      w[i >> 2] |= (static_cast<uint32_t>(c) & 0xffu) << (8 * (i & 3));
    }
    return make_uint2(w[0], w[1]);
  }
}

// One warp: rows_per_warp rows of one kind of one token, in batches of NIT
// rounds of 256/D rows; a batch's rows are read while the one before is worked
// on.
template <int D, int KV, bool INTER, int NIT>
__global__ void __launch_bounds__(kNrWarps * 32, NIT == 2 ? 8 : 1)
    norm_rope_kernel(const NormRopeArgs a) {
  constexpr int LPR = D / 8;     // lanes per row
  constexpr int RPW = 32 / LPR;  // rows of a round
  constexpr int RW = NIT * RPW;  // rows of a batch
  // launched as a programmatic dependent: everything is read after the wait,
  // and the next launch may start only then (a decode reads the lengths and
  // the block tables before its own wait; what wrote them is complete here)
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, c = lane % LPR;
  const int H = a.num_heads, Hkv = a.num_kv_heads;
  const int RPT = a.rows_per_warp;
  const int nq = (H + RPT - 1) / RPT, nk = (Hkv + RPT - 1) / RPT;
  const unsigned wpt = nq + 2 * nk;  // warps per token
  const unsigned w = blockIdx.x * kNrWarps + (threadIdx.x >> 5);
  const long long t = w / wpt;
  if (t >= a.num_tokens) return;
  int part = static_cast<int>(w % wpt);
  const int kind = part < nq ? 0 : part < nq + nk ? 1 : 2;  // q, k, v
  part -= kind == 0 ? 0 : kind == 1 ? nq : nq + nk;
  const int row0 = part * RPT + sub;
  const int rows = min(kind == 0 ? H : Hkv, part * RPT + RPT);

  const __nv_bfloat16* src =
      static_cast<const __nv_bfloat16*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
      t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + c * 8;
  uint4 raw[NIT], nxt[NIT];
  auto load = [&](uint4 (&x)[NIT], int r0) {
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
      const int r = r0 + i * RPW;
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) x[i] = *reinterpret_cast<const uint4*>(src + r * D);
    }
  };
  load(raw, row0);
  const long long slot = a.slot_mapping[t];
  if (slot < 0) return;  // padding token
  const int rot = a.rotary_dim;
  long long pos = 0;
  if (rot > 0) {
    pos = a.positions[t];
    if (pos < 0 || pos >= a.max_positions) {
      if (lane == 0) report_error(a.err, PA_DEVERR_POSITION_RANGE);
      return;
    }
  }
  if (kind != 0 && slot >= a.num_slots) {
    if (lane == 0) report_error(a.err, PA_DEVERR_SLOT_RANGE);
    return;
  }

  // ---- factors of this lane's eight elements: y_i = rstd * (x_i A_i + partner_i B_i)
  // (a lane that is not rotated adds 0 * -0 = -0: x * A unchanged, zeros too)
  float A[8], B[8];
  const void* const wt = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
  const bool norm = wt != nullptr;
  int pc = c;  // chunk that holds the partners of a half-split pair
  float wf[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) wf[i] = 1.f;
  if (norm) unpack8(__ldg(static_cast<const uint4*>(wt) + c), wf);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    A[i] = wf[i];
    B[i] = -0.f;
  }
  if (kind != 2) {
    if (c * 8 < rot) {
      const float* cs = a.cos_sin + pos * rot;
      if constexpr (INTER) {
        // pairs (2i, 2i+1): four of them in this chunk
        const float4 co = __ldg(reinterpret_cast<const float4*>(cs + c * 4));
        const float4 si = __ldg(reinterpret_cast<const float4*>(cs + rot / 2 + c * 4));
        const float cv[4] = {co.x, co.y, co.z, co.w}, sv[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          A[2 * i] = wf[2 * i] * cv[i];
          B[2 * i] = -wf[2 * i + 1] * sv[i];
          A[2 * i + 1] = wf[2 * i + 1] * cv[i];
          B[2 * i + 1] = wf[2 * i] * sv[i];
        }
      } else {
        const int hc = rot / 16;  // chunks of half the rotated part
        const bool second = c >= hc;
        pc = second ? c - hc : c + hc;
        float pw[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) pw[i] = 1.f;
        if (norm) unpack8(__ldg(static_cast<const uint4*>(wt) + pc), pw);
        const float4* cp = reinterpret_cast<const float4*>(cs + 8 * (second ? pc : c));
        const float4* sp = reinterpret_cast<const float4*>(cs + rot / 2 + 8 * (second ? pc : c));
        const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
        const float cv[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          A[i] = wf[i] * cv[i];
          B[i] = second ? pw[i] * sv[i] : -pw[i] * sv[i];
        }
      }
    }
  }
  const int plane = (lane - c) + pc;  // lane of the partner chunk

  const long long blk = kind == 0 ? 0 : slot / a.block_size;
  const int off = kind == 0 ? 0 : static_cast<int>(slot - blk * a.block_size);
  const uint32_t pmask = kind != 2 && c * 8 < rot ? 0xffffffffu : 0u;  // not rotated: no partner
  uint64_t A2[4], B2[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    A2[j] = tc::f32x2(A[2 * j], A[2 * j + 1]);
    B2[j] = tc::f32x2(B[2 * j], B[2 * j + 1]);
  }
#pragma unroll 1
  for (int r0 = row0; r0 - sub < rows; r0 += RW) {
    if (r0 - sub + RW < rows) load(nxt, r0 + RW);
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
      const int r = r0 + i * RPW;
      float x[8];
      if (kind != 2) {
        const uint32_t xw[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint64_t x2[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x2[j] = unpack2(xw[j]);
        float rstd = 1.f;
        if (norm) {
          uint64_t s2 = tc::fma_f32x2(x2[0], x2[0], tc::f32x2(0.f, 0.f));
#pragma unroll
          for (int j = 1; j < 4; ++j) s2 = tc::fma_f32x2(x2[j], x2[j], s2);
          float s0, s1;
          tc::f32x2_split(s2, s0, s1);
          float ss = s0 + s1;
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
          rstd = rsqrtf(ss * (1.f / D) + a.eps);
        }
        const uint64_t r2 = tc::f32x2(rstd, rstd);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t pw = INTER ? prmt(xw[j], 0u, 0x1032u) : __shfl_sync(kAll, xw[j], plane);
          const uint64_t y2 = tc::mul_f32x2(unpack2(pw & pmask), B2[j]);
          tc::f32x2_split(tc::mul_f32x2(tc::fma_f32x2(x2[j], A2[j], y2), r2), x[2 * j], x[2 * j + 1]);
        }
      } else if (KV != kKvBf16) {
        unpack8(raw[i], x);
      }
      if (kind == 0) {
        if (r < rows)
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.q_out) +
                                    (t * H + r) * D + c * 8) = pack8(x);
        continue;
      }
      void* const cache = kind == 1 ? a.k_cache : a.v_cache;
      const long long row = slot * Hkv + r;  // (slot, head) row of the cache
      if constexpr (KV == kKvBf16) {
        if (r < rows)
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cache) + row * D + c * 8) =
              kind == 2 ? raw[i] : pack8(x);
      } else {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(x[j]));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(kAll, amax, o));
        float sc = amax / (KV == kKvE4m3 ? 448.f : 127.f);
        if (sc == 0.f) sc = 1.f;  // a row of zeros (or whose scale underflows)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] / sc;
        if (r < rows) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + row * D + c * 8) = codes8<KV>(x);
          if (c == 0) (kind == 1 ? a.k_scale : a.v_scale)[(blk * Hkv + r) * a.block_size + off] = sc;
        }
      }
      if (kind == 1 && a.scores != nullptr && c == 0 && r < rows)
        a.scores[(blk * Hkv + r) * a.block_size + off] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NIT; ++i) raw[i] = nxt[i];
  }
}

template <int D, int KV, bool INTER, int NIT>
cudaError_t launch_inst(NormRopeArgs a, int batches, cudaStream_t stream) {
  a.rows_per_warp = NIT * (256 / D) * batches;
  const long long RPT = a.rows_per_warp;
  const long long wpt = (a.num_heads + RPT - 1) / RPT + 2 * ((a.num_kv_heads + RPT - 1) / RPT);
  const long long grid = (a.num_tokens * wpt + kNrWarps - 1) / kNrWarps;
  if (grid > 0x7fffffffLL / kNrWarps) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kNrWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<D, KV, INTER, NIT>, a);
}

// Rounds of a batch and batches of a warp. One round each keeps the smallest
// calls' latency down; with more rows than the machine holds warps for, two
// rounds and up to four batches spend the token's factors on more rows and keep
// reads under way. us per call, (rounds x batches) 1x1 / 2x1 / 2x2 / 2x4, from
// graph replays on one GB300, 48 rows of 128 a token (bf16): 64 tokens 2.6 / 2.9
// / 3.5 / 4.5, 256: 4.6 / 4.2 / 3.9 / 4.9, 512: 7.0 / 6.0 / 5.5 / 5.3, 1024:
// 13.9 / 10.3 / 8.8 / 7.7, 8192: 106 / 67 / 48 / 43; 80 rows of 128 (E4M3): 128:
// 5.0 / 4.9 / 5.3 / 5.2, 256: 7.4 / 6.3 / 7.1 / 5.6, 512: 13.0 / 9.4 / 9.2 / 8.5;
// 24 rows of 64: 256: 2.6 / 2.9, 1024: 4.6 / 4.0, 8192: 30 / 19.
template <int D, int KV, bool INTER>
cudaError_t launch_rounds(const NormRopeArgs& a, cudaStream_t stream) {
  constexpr int RPW = 256 / D;
  const long long rounds = static_cast<long long>(a.num_tokens) *
                           ((a.num_heads + 2LL * a.num_kv_heads + RPW - 1) / RPW);
  const long long slots = 32LL * a.num_sms;  // rounds in flight with half the warps of an SM
  if (rounds <= slots) return launch_inst<D, KV, INTER, 1>(a, 1, stream);
  if (rounds <= 2 * slots) return launch_inst<D, KV, INTER, 2>(a, 2, stream);
  return launch_inst<D, KV, INTER, 2>(a, 4, stream);
}

template <int D, int KV>
cudaError_t launch_kind(const NormRopeArgs& a, cudaStream_t stream) {
  return a.interleaved ? launch_rounds<D, KV, true>(a, stream)
                       : launch_rounds<D, KV, false>(a, stream);
}

}  // namespace

cudaError_t launch_norm_rope_store(const NormRopeArgs& a, cudaStream_t stream) {
  if (a.num_tokens <= 0) return cudaSuccess;
  if (a.kv == kKvE4m3) return launch_kind<128, kKvE4m3>(a, stream);
  if (a.kv == kKvInt8) return launch_kind<128, kKvInt8>(a, stream);
  return a.head_dim == 64 ? launch_kind<64, kKvBf16>(a, stream) : launch_kind<128, kKvBf16>(a, stream);
}

}  // namespace pa
