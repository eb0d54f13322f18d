// rope_append_paged: rotary positions of the new tokens' q and k rows, fused with the write of
// K and V into their page slots (sm_103a).
//
// With a_i = position * inv_freq_i, each pair (x1, x2) of the first rot dims of a head becomes
//     (x1 cos a_i - x2 sin a_i,  x2 cos a_i + x1 sin a_i) * attn_factor,
// the pair being dims (i, i + rot / 2) or, interleaved, (2i, 2i + 1); before it, q and k rows may
// be RMS-normalised per head: x / sqrt(mean x^2 + eps) * gamma. One pass in fp32, one rounding
// to bf16 at the end. The bound is memory: every q, k and v row is read once and written once
// (16 KB per token of the 16/8-head decoder). Measured inside a graph: 4,127 rows with norms 13.2 us
// (5.1 TB/s), 31 rows 2.6 us. At 8 dims of a row per lane instead of 4, loads in the same pass and a
// barrier per pass the first form took 21 us; now instruction issue (63 %) and memory are both near.
//
// The angle. At position 100,000 an fp32 product position * inv_freq is off by up to 0.004 rad,
// more than a bf16 rounding. Here a frequency is held in turns as a 64-bit binary fraction
// (inv_freq / 2 pi, its integer part dropped), so position * frequency mod 2^64 is the exact
// fraction of a turn of that frequency for every int32 position, one integer multiply; its upper
// half, as fp32, goes to sincospif.
//
// Layout. A unit is one token's KV head: its two q rows, its k row and its v row, 256 bytes each. A
// warp takes two units a pass (two heads of one token, unless the call has one KV head), 8 bytes
// (4 dims) of each row per lane, all eight loads in flight before anything else; 16 units per CTA
// pass. The cosines and sines of the pass's tokens are computed once by the CTA and shared through
// shared memory (with one sincospif per lane and pair the 8 heads of a token would compute them 8
// times), while the row loads are in flight; a lane multiplies them by gamma once for the rows that
// share both. The partner of a dim in the half layout is rot / 8 lanes away: the raw words are
// exchanged by two shuffles per row, before the norm, whose factor is common to the row.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "dependent_launch.cuh"
#include "pa_common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = kThreads / 16;       // units of a CTA pass: two a warp
constexpr int kMaxPairs = kHeadDim / 2;
constexpr int kTableTokens = 32;            // tokens whose cosines and sines are held at a time
// Two CTAs per SM: a pass in flight and one ahead of it for every warp, at 123 registers. Three or four
// CTAs of 80 or 64 registers spill and measured slower (16.8 and 24.1 against 13.2 us for 4,127 rows).
constexpr int kCtasPerSm = 2;

struct RopeParams {
  int32_t hkv_shift;  // log2 of the KV heads
  int32_t rot, interleaved;
  const double* inv_freq;
  float attn_factor;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;  // elements between consecutive tokens
  int64_t units;                         // rows << hkv_shift
  const int32_t* positions;
  const int64_t* slots;
  const float* q_gamma;
  const float* k_gamma;
  float eps;
  uint16_t* q_out;
  uint16_t* k_pool;
  uint16_t* v_pool;
  int64_t num_slots;
  int32_t* status;
};

__device__ __forceinline__ uint2 load_row8(const uint16_t* p) {
  return __ldcs(reinterpret_cast<const uint2*>(p));  // read once: do not keep it in L1
}

// The fraction of a turn in f radians, as a 64-bit binary fraction: f = m 2^e with an integer m, so
// frac(f / 2 pi) 2^64 is the low 64 bits of m C 2^e with C = 2^64 / (2 pi). Integer arithmetic: fp64
// instructions run at 1/64 of the fp32 rate here, and a CTA's 64 conversions in fp64 took longer
// than its rows (24 us for 4,127 rows).
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
  constexpr unsigned long long kTurns = 0x28be60db9391054aull;  // 2^64 / (2 pi)
  const long long bits = __double_as_longlong(f);
  const int field = static_cast<int>(bits >> 52) & 0x7ff;
  if (field == 0) return 0;  // zero (or subnormal: no turn at any int32 position)
  const unsigned long long m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
  const int e = field - 1075;
  const unsigned long long lo = m * kTurns, hi = __umul64hi(m, kTurns);
  unsigned long long r = 0;
  if (e >= 0) r = e < 64 ? lo << e : 0;
  else if (e > -64) r = (hi << (64 + e)) | (lo >> -e);
  else if (e > -128) r = hi >> (-e - 64);
  return bits < 0 ? 0 - r : r;
}

// The factors of a lane's 4 dims: a row x with partner values y turns into
//     inv * (x own + y other),   own = gamma cos, other = -+ gamma(partner) sin,
// inv being the row's norm (1 without one). Lanes past rot: own = gamma, other = 0.
struct Factors {
  float2 own[2], other[2];
};

template <bool kInterleaved>
__device__ __forceinline__ Factors factors(const float* gamma, int lane, int partner, float sign,
                                           const float2 (&cs)[2], const float2 (&sn)[2]) {
  Factors f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f.own[i] = cs[i];
    f.other[i] = kInterleaved ? make_float2(-sn[i].x, sn[i].y) : mul2(sn[i], make_float2(sign, sign));
  }
  if (gamma != nullptr) {
    const float4 g = *reinterpret_cast<const float4*>(gamma + 4 * lane);
    f.own[0] = mul2(f.own[0], make_float2(g.x, g.y));
    f.own[1] = mul2(f.own[1], make_float2(g.z, g.w));
    if (kInterleaved) {
      f.other[0] = mul2(f.other[0], make_float2(g.y, g.x));
      f.other[1] = mul2(f.other[1], make_float2(g.w, g.z));
    } else {
      const float4 h = *reinterpret_cast<const float4*>(gamma + 4 * partner);
      f.other[0] = mul2(f.other[0], make_float2(h.x, h.y));
      f.other[1] = mul2(f.other[1], make_float2(h.z, h.w));
    }
  }
  return f;
}

// Sum of a lane's 4 squares.
__device__ __forceinline__ float squares(uint2 raw) {
  const float2 x0 = make_float2(bf16lo(raw.x), bf16hi(raw.x)), x1 = make_float2(bf16lo(raw.y), bf16hi(raw.y));
  const float2 sq = fma2(x1, x1, mul2(x0, x0));
  return sq.x + sq.y;
}

// Rotation of one 128-dim row held 4 dims a lane by a warp; inv: its norm's factor.
template <bool kInterleaved>
__device__ __forceinline__ uint2 turn_row(uint2 raw, float inv, int partner, bool past, const Factors& f) {
  const float2 x0 = make_float2(bf16lo(raw.x), bf16hi(raw.x)), x1 = make_float2(bf16lo(raw.y), bf16hi(raw.y));
  float2 y0, y1;
  if (kInterleaved) {  // the partner is the pair's other dim
    y0 = make_float2(x0.y, x0.x);
    y1 = make_float2(x1.y, x1.x);
  } else {             // the partner is rot / 8 lanes away: exchange the raw words
    const uint32_t a = __shfl_sync(0xffffffffu, raw.x, partner), b = __shfl_sync(0xffffffffu, raw.y, partner);
    y0 = make_float2(bf16lo(a), bf16hi(a));
    y1 = make_float2(bf16lo(b), bf16hi(b));
  }
  if (past) y0 = y1 = make_float2(0.f, 0.f);  // past rot: not even 0 times an infinite partner
  const float2 inv2 = make_float2(inv, inv);
  const float2 r0 = mul2(fma2(y0, f.other[0], mul2(x0, f.own[0])), inv2);
  const float2 r1 = mul2(fma2(y1, f.other[1], mul2(x1, f.own[1])), inv2);
  return make_uint2(pack_bf16x2(r0.x, r0.y), pack_bf16x2(r1.x, r1.y));
}

// The rows of one warp's two units of a pass, as loaded.
struct UnitRows {
  uint2 q0[2], q1[2], k[2], v[2];
  int64_t slot[2];
};

// A lane's place in the rows of its warp's two units: unit i's rows start i * step further. Advanced by
// constants from pass to pass, so that a pass computes no address but the slots'.
struct UnitPlace {
  const uint16_t *q, *k, *v;
  const int64_t* slot;
  uint16_t* out;
  int64_t q_step, k_step, v_step, out_step;  // elements from unit 0's rows to unit 1's
  int slot_step;                             // tokens from unit 0 to unit 1
};

// left: tokens of the call from unit 0's on.
__device__ __forceinline__ void load_units(const UnitPlace& a, int64_t left, UnitRows& r) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r.q0[i] = r.q1[i] = r.k[i] = r.v[i] = make_uint2(0u, 0u);
    r.slot[i] = -1;
    if (i * a.slot_step < left) {
      const uint16_t* q = a.q + (i ? a.q_step : 0);
      r.q0[i] = load_row8(q);
      r.q1[i] = load_row8(q + kHeadDim);
      r.k[i] = load_row8(a.k + (i ? a.k_step : 0));
      r.v[i] = load_row8(a.v + (i ? a.v_step : 0));
      r.slot[i] = a.slot[i ? a.slot_step : 0];
    }
  }
}

// CTA b takes passes b * passes_per_cta .. of kUnits units each: consecutive tokens. Their cosines
// and sines are computed kTableTokens tokens at a time; between two such chunks no barrier holds a
// warp up, and each warp loads the rows of its next pass before it works on this one's.
template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) rope_append_kernel(const RopeParams p, int passes_per_cta) {
  __shared__ __align__(16) float cos_s[kTableTokens][kMaxPairs], sin_s[kTableTokens][kMaxPairs];
  const int tid = threadIdx.x, lane = tid & 31, u = (tid >> 5) * 2;
  const int pairs = p.rot >> 1;
  // half layout: lanes [0, rot / 8) hold the pairs' first dims, the next rot / 8 the second
  const int span = p.rot >> 3;
  float sign = 0.f;
  int partner = lane;
  if (kInterleaved) {
    sign = 4 * lane < p.rot ? 1.f : 0.f;
  } else if (lane < span) {
    sign = -1.f;
    partner = lane + span;
  } else if (lane < 2 * span) {
    sign = 1.f;
    partner = lane - span;
  }
  const int hkv = 1 << p.hkv_shift;
  const int tokens = kUnits >> p.hkv_shift;           // tokens of a pass: whole ones (hkv <= 8)
  const int chunk = kTableTokens / tokens;            // passes of a table
  const int64_t first = static_cast<int64_t>(blockIdx.x) * passes_per_cta * kUnits;
  const bool past = sign == 0.f;
  UnitPlace at;
  int64_t left;  // tokens from this warp's first one on
  const int g = u & (hkv - 1);  // (one KV head: the second unit is the next token's)
  {
    const int64_t t = (first + u) >> p.hkv_shift;
    left = (p.units >> p.hkv_shift) - t;
    at.q = p.q + t * p.q_stride + 2 * g * kHeadDim + 4 * lane;
    at.k = p.k + t * p.k_stride + g * kHeadDim + 4 * lane;
    at.v = p.v + t * p.v_stride + g * kHeadDim + 4 * lane;
    at.out = p.q_out + (t * (2 * hkv) + 2 * g) * kHeadDim + 4 * lane;
    at.slot = p.slots + t;
    at.q_step = hkv == 1 ? p.q_stride : 2 * kHeadDim;
    at.k_step = hkv == 1 ? p.k_stride : kHeadDim;
    at.v_step = hkv == 1 ? p.v_stride : kHeadDim;
    at.out_step = 2 * kHeadDim;
    at.slot_step = hkv == 1 ? 1 : 0;
  }
  const int64_t q_pass = tokens * p.q_stride, k_pass = tokens * p.k_stride, v_pass = tokens * p.v_stride;
  uint16_t* const k_out = p.k_pool + g * kHeadDim + 4 * lane;
  uint16_t* const v_out = p.v_pool + g * kHeadDim + 4 * lane;
  const int unit_head = hkv == 1 ? 0 : kHeadDim;  // from unit 0's head in a slot to unit 1's
  UnitRows rows;
  await_previous();
  load_units(at, left, rows);
  const int j = tid & (kMaxPairs - 1);  // this thread's frequency in the tables (kThreads is a multiple)
  const unsigned long long turn = j < pairs ? turn_fraction(p.inv_freq[j]) : 0;
  for (int pass = 0; pass < passes_per_cta; ++pass) {
    const int64_t unit0 = first + static_cast<int64_t>(pass) * kUnits;
    if (unit0 >= p.units) break;
    if (pass % chunk == 0) {
      if (pass > 0) __syncthreads();  // the table before has been read
      const int n = min(chunk, passes_per_cta - pass) * tokens;
      for (int i = tid; i < n * kMaxPairs; i += kThreads) {
        const int64_t t = (unit0 >> p.hkv_shift) + (i >> 6);
        if (j < pairs && (t << p.hkv_shift) < p.units) {
          const long long pos = p.positions[t];
          const unsigned long long phase = static_cast<unsigned long long>(pos) * turn;
          // the signed upper half: [-1/2, 1/2) turns, in half turns for sincospif
          const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * (1.0f / 2147483648.0f);
          float sn, cs;
          sincospif(half_turns, &sn, &cs);
          cos_s[i >> 6][j] = cs * p.attn_factor;
          sin_s[i >> 6][j] = sn * p.attn_factor;
        }
      }
      __syncthreads();
    }
    const UnitRows cur = rows;
    uint16_t* const out = at.out;
    if (pass + 1 < passes_per_cta) {
      at.q += q_pass;
      at.k += k_pass;
      at.v += v_pass;
      at.slot += tokens;
      at.out += tokens * (2 * hkv * kHeadDim);
      left -= tokens;
      load_units(at, left, rows);
    }
    // the norms of the warp's six rows together: six independent sums a reduction step
    float inv[6] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (p.q_gamma != nullptr || p.k_gamma != nullptr) {
      float sum[6] = {squares(cur.q0[0]), squares(cur.q1[0]), squares(cur.k[0]),
                      squares(cur.q0[1]), squares(cur.q1[1]), squares(cur.k[1])};
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
#pragma unroll
        for (int i = 0; i < 6; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
      }
#pragma unroll
      for (int i = 0; i < 6; ++i)
        if ((i % 3 < 2 ? p.q_gamma : p.k_gamma) != nullptr) inv[i] = rsqrtf(sum[i] * (1.0f / kHeadDim) + p.eps);
    }
    Factors fq, fk;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i == 0 || hkv == 1) {  // the second unit is another head of the same token
        float2 cs[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)};
        float2 sn[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const int row = (pass % chunk) * tokens + ((u + i) >> p.hkv_shift);
        if (sign != 0.f) {
          if (kInterleaved) {  // one angle a pair
            const float2 a = *reinterpret_cast<const float2*>(&cos_s[row][2 * lane]);
            const float2 b = *reinterpret_cast<const float2*>(&sin_s[row][2 * lane]);
            cs[0] = make_float2(a.x, a.x);
            cs[1] = make_float2(a.y, a.y);
            sn[0] = make_float2(b.x, b.x);
            sn[1] = make_float2(b.y, b.y);
          } else {
            const int at = 4 * (lane < span ? lane : lane - span);
            const float4 a = *reinterpret_cast<const float4*>(&cos_s[row][at]);
            const float4 b = *reinterpret_cast<const float4*>(&sin_s[row][at]);
            cs[0] = make_float2(a.x, a.y);
            cs[1] = make_float2(a.z, a.w);
            sn[0] = make_float2(b.x, b.y);
            sn[1] = make_float2(b.z, b.w);
          }
        }
        fq = factors<kInterleaved>(p.q_gamma, lane, partner, sign, cs, sn);
        fk = factors<kInterleaved>(p.k_gamma, lane, partner, sign, cs, sn);
      }
      const uint2 q0r = turn_row<kInterleaved>(cur.q0[i], inv[3 * i], partner, past, fq);
      const uint2 q1r = turn_row<kInterleaved>(cur.q1[i], inv[3 * i + 1], partner, past, fq);
      const uint2 k0r = turn_row<kInterleaved>(cur.k[i], inv[3 * i + 2], partner, past, fk);
      const int64_t slot = cur.slot[i];  // negative: a padding row, nothing is written
      if (slot >= p.num_slots && lane == 0) flag_error(p.status, PA_DEV_ERR_PAGE_OOB);
      if (slot >= 0 && slot < p.num_slots) {
        uint16_t* qo = out + i * at.out_step;
        *reinterpret_cast<uint2*>(qo) = q0r;
        *reinterpret_cast<uint2*>(qo + kHeadDim) = q1r;
        const int64_t to = slot * (hkv * kHeadDim) + i * unit_head;
        *reinterpret_cast<uint2*>(k_out + to) = k0r;
        *reinterpret_cast<uint2*>(v_out + to) = cur.v[i];
      }
    }
  }
}

}  // namespace
}  // namespace pa

extern "C" pa_status rope_append_paged(pa_dims dims, int32_t rot_dim, int32_t interleaved,
                                       const double* inv_freq, float attn_factor, const void* q,
                                       int64_t q_stride, const void* k_new, int64_t k_stride,
                                       const void* v_new, int64_t v_stride, int32_t rows,
                                       const int32_t* positions, const int64_t* slot_map,
                                       const float* q_gamma, const float* k_gamma, float eps,
                                       void* q_out, void* k_pool, void* v_pool, int64_t num_pages,
                                       int32_t* status, pa_stream_t stream) {
  using namespace pa;
  if (!gqa_dims_supported(dims)) return PA_ERR_UNSUPPORTED;
  if (rot_dim < 16 || rot_dim > kHeadDim || rot_dim % 16 != 0) {
    snprintf_error("rope_append_paged: rot_dim %d is not a multiple of 16 in [16, 128]", rot_dim);
    return PA_ERR_UNSUPPORTED;
  }
  const int64_t q_row = static_cast<int64_t>(dims.num_q_heads) * kHeadDim;
  const int64_t kv_row = static_cast<int64_t>(dims.num_kv_heads) * kHeadDim;
  if (rows < 0 || num_pages <= 0 || !(eps >= 0.f) || !(attn_factor == attn_factor)) return PA_ERR_INVALID_ARG;
  if (rows == 0) return PA_OK;
  if (!inv_freq || !q || !k_new || !v_new || !positions || !slot_map || !q_out || !k_pool || !v_pool)
    return PA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new) |
       reinterpret_cast<uintptr_t>(q_out) | reinterpret_cast<uintptr_t>(k_pool) |
       reinterpret_cast<uintptr_t>(v_pool) | reinterpret_cast<uintptr_t>(q_gamma) |
       reinterpret_cast<uintptr_t>(k_gamma)) & 15u)
    return PA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(inv_freq) | reinterpret_cast<uintptr_t>(slot_map)) & 7u) return PA_ERR_INVALID_ARG;
  // rows may lie apart (slices of one fused projection) but not over one another
  if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row || ((q_stride | k_stride | v_stride) & 7))
    return PA_ERR_INVALID_ARG;
  if (q_out == q && q_stride != q_row) return PA_ERR_INVALID_ARG;  // in place only where rows coincide
  const int sms = sm_count_current_device();
  if (sms <= 0) return PA_ERR_CUDA;
  RopeParams p;
  p.hkv_shift = dims.num_kv_heads == 8 ? 3 : dims.num_kv_heads == 4 ? 2 : dims.num_kv_heads == 2 ? 1 : 0;
  p.rot = rot_dim;
  p.interleaved = interleaved;
  p.inv_freq = inv_freq;
  p.attn_factor = attn_factor;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k_new);
  p.v = static_cast<const uint16_t*>(v_new);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.units = static_cast<int64_t>(rows) << p.hkv_shift;
  p.positions = positions;
  p.slots = slot_map;
  p.q_gamma = q_gamma;
  p.k_gamma = k_gamma;
  p.eps = eps;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_pool = static_cast<uint16_t*>(k_pool);
  p.v_pool = static_cast<uint16_t*>(v_pool);
  p.num_slots = num_pages * kPage;
  p.status = status;
  const int64_t passes = (p.units + kUnits - 1) / kUnits;
  // as many CTAs as are resident, each with the same number of passes
  const int64_t most = static_cast<int64_t>(sms) * kCtasPerSm;
  const int per_cta = static_cast<int>((passes + most - 1) / most);
  const unsigned grid = static_cast<unsigned>((passes + per_cta - 1) / per_cta);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_dependent(interleaved ? rope_append_kernel<true> : rope_append_kernel<false>,
                                         grid, kThreads, 0, st, 0, p, per_cta);
  return e == cudaSuccess ? PA_OK : record_cuda_error(e, "rope_append_kernel");
}

extern "C" pa_status pa_rope_inv_freq(int32_t rot_dim, double theta, const pa_rope_scaling* scaling,
                                      double* inv_freq, float* attn_factor) {
  using namespace pa;
  if (rot_dim < 2 || rot_dim % 2 != 0 || !(theta > 0.0) || !std::isfinite(theta) || !inv_freq || !attn_factor)
    return PA_ERR_INVALID_ARG;
  const int n = rot_dim / 2;
  const int32_t kind = scaling != nullptr ? scaling->kind : PA_ROPE_NONE;
  const double kTwoPi = 6.283185307179586477;
  if (kind != PA_ROPE_NONE && (!(scaling->factor > 0.0) || !std::isfinite(scaling->factor))) return PA_ERR_INVALID_ARG;
  *attn_factor = 1.0f;
  auto freq = [&](double base, int i) { return std::pow(base, -2.0 * i / rot_dim); };
  switch (kind) {
    case PA_ROPE_NONE:
      for (int i = 0; i < n; ++i) inv_freq[i] = freq(theta, i);
      return PA_OK;
    case PA_ROPE_LINEAR:
      for (int i = 0; i < n; ++i) inv_freq[i] = freq(theta, i) / scaling->factor;
      return PA_OK;
    case PA_ROPE_NTK: {
      if (rot_dim <= 2) return PA_ERR_INVALID_ARG;
      const double base = theta * std::pow(scaling->factor, rot_dim / (rot_dim - 2.0));
      for (int i = 0; i < n; ++i) inv_freq[i] = freq(base, i);
      return PA_OK;
    }
    case PA_ROPE_LLAMA3: {
      const double low = scaling->low_freq_factor, high = scaling->high_freq_factor;
      if (!(scaling->original_max_position > 0.0) || !(high > low)) return PA_ERR_INVALID_ARG;
      for (int i = 0; i < n; ++i) {
        const double f = freq(theta, i), turns = scaling->original_max_position * f / kTwoPi;
        const double keep = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
        inv_freq[i] = f / scaling->factor * (1.0 - keep) + f * keep;
      }
      return PA_OK;
    }
    case PA_ROPE_YARN: {
      if (!(scaling->original_max_position > 0.0) || !(scaling->beta_fast > scaling->beta_slow) ||
          !(scaling->beta_slow > 0.0) || theta == 1.0)
        return PA_ERR_INVALID_ARG;
      // the pair that makes `turns` turns over the original context
      auto pair_of = [&](double turns) {
        return rot_dim * std::log(scaling->original_max_position / (turns * kTwoPi)) / (2.0 * std::log(theta));
      };
      const double low = std::fmax(std::floor(pair_of(scaling->beta_fast)), 0.0);
      const double high = std::fmin(std::ceil(pair_of(scaling->beta_slow)), rot_dim - 1.0);
      for (int i = 0; i < n; ++i) {
        const double f = freq(theta, i);
        const double ramp = std::fmin(1.0, std::fmax(0.0, (i - low) / std::fmax(high - low, 1e-3)));
        inv_freq[i] = f / scaling->factor * ramp + f * (1.0 - ramp);
      }
      const double a = scaling->attn_factor > 0.0 ? scaling->attn_factor
                       : scaling->factor > 1.0    ? 0.1 * std::log(scaling->factor) + 1.0
                                                  : 1.0;
      *attn_factor = static_cast<float>(a);
      return PA_OK;
    }
    default: return PA_ERR_INVALID_ARG;
  }
}
