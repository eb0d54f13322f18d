// rope_append_paged: rotary positions of the new tokens' q and k rows, fused with the write of
// K and V into their page slots (sm_103a).
//
// With a_i = position * inv_freq_i, each pair (x1, x2) of the first rot dims of a head becomes
//     (x1 cos a_i - x2 sin a_i,  x2 cos a_i + x1 sin a_i) * attn_factor,
// the pair being dims (i, i + rot / 2) or, interleaved, (2i, 2i + 1); before it, q and k rows may
// be RMS-normalised per head: x / sqrt(mean x^2 + eps) * gamma. One pass in fp32, one rounding
// to bf16 at the end. The bound is memory: every q, k and v row is read once and written once
// (16 KB per token of the 16/8-head decoder), against ~70 operations per 16 bytes.
//
// The angle. At position 100,000 an fp32 product position * inv_freq is off by up to 0.004 rad,
// more than a bf16 rounding. Here a frequency is held in turns as a 64-bit binary fraction
// (inv_freq / 2 pi, its integer part dropped), so position * frequency mod 2^64 is the exact
// fraction of a turn of that frequency for every int32 position, one integer multiply; its upper
// half, as fp32, goes to sincospif.
//
// Layout. A unit is one token's KV head: its two q rows, its k row and its v row, 256 bytes each.
// Half a warp takes a unit, 16 bytes (8 dims) of each row per lane, all four loads in flight
// before anything else; 16 units per CTA pass. The cosines and sines of the pass's tokens are
// computed once by the CTA and shared through shared memory (with one sincospif per lane and pair
// the 8 heads of a token would compute them 8 times), while the row loads are in flight. The
// partner of a dim in the half layout is rot / 16 lanes away: the raw words are exchanged by four
// shuffles per row, before the norm, whose factor is common to the row.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "pa_common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = kThreads / 16;       // units of a CTA pass
constexpr int kMaxPairs = kHeadDim / 2;
// CTAs per SM of a long call: enough row loads in flight to cover the latency (8 x 16 KB per SM)
constexpr int kCtasPerSm = 8;

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

__device__ __forceinline__ uint4 load_row16(const uint16_t* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));  // read once: do not keep it in L1
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  x[0] = bf16lo(w.x); x[1] = bf16hi(w.x); x[2] = bf16lo(w.y); x[3] = bf16hi(w.y);
  x[4] = bf16lo(w.z); x[5] = bf16hi(w.z); x[6] = bf16lo(w.w); x[7] = bf16hi(w.w);
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// Norm (gamma != null) and rotation of one 128-dim row held 8 dims a lane by half a warp.
// kInterleaved: the pairs are inside a lane; else the partner dims are in lane `partner`, and
// sign is -1 for the first dims of the pairs, +1 for the second, 0 for lanes past rot.
template <bool kInterleaved>
__device__ __forceinline__ uint4 turn_row(uint4 raw, const float* gamma, float eps, int c, int partner,
                                          float sign, const float (&cs)[8], const float (&sn)[8]) {
  float x[8];
  unpack8(raw, x);
  float inv = 1.f;
  if (gamma != nullptr) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    inv = 1.0f / sqrtf(sum * (1.0f / kHeadDim) + eps);
    float g[8];
    load8(gamma + 8 * c, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= inv * g[i];
  }
  float r[8];
  if (kInterleaved) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {  // sign = 0: dims past rot keep their value
      r[i] = sign != 0.f ? x[i] * cs[i / 2] - x[i + 1] * sn[i / 2] : x[i];
      r[i + 1] = sign != 0.f ? x[i + 1] * cs[i / 2] + x[i] * sn[i / 2] : x[i + 1];
    }
  } else {
    uint4 other;
    other.x = __shfl_sync(0xffffffffu, raw.x, partner);
    other.y = __shfl_sync(0xffffffffu, raw.y, partner);
    other.z = __shfl_sync(0xffffffffu, raw.z, partner);
    other.w = __shfl_sync(0xffffffffu, raw.w, partner);
    float y[8];
    unpack8(other, y);
    if (gamma != nullptr) {
      float g[8];
      load8(gamma + 8 * (partner & 15), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= inv * g[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = sign != 0.f ? x[i] * cs[i] + sign * y[i] * sn[i] : x[i];
  }
  return make_uint4(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]), pack_bf16x2(r[4], r[5]),
                    pack_bf16x2(r[6], r[7]));
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeParams p) {
  __shared__ unsigned long long turn[kMaxPairs];
  // cosines and sines (times attn_factor) of a pass's tokens (at most one per unit), two buffers:
  // one barrier per pass
  __shared__ __align__(16) float cos_s[2][kUnits][kMaxPairs], sin_s[2][kUnits][kMaxPairs];
  const int tid = threadIdx.x, lane = tid & 31, c = lane & 15, u = tid >> 4;
  const int pairs = p.rot >> 1;
  if (tid < pairs) {
    double t = p.inv_freq[tid] * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    turn[tid] = static_cast<unsigned long long>(t * 18446744073709551616.0);  // 2^64
  }
  // half layout: lanes [0, rot/16) hold the pairs' first dims, the next rot/16 the second
  const int span = p.rot >> 4;
  float sign = 0.f;
  int partner = lane;
  if (kInterleaved) {
    sign = 8 * c < p.rot ? 1.f : 0.f;
  } else if (c < span) {
    sign = -1.f;
    partner = lane + span;
  } else if (c < 2 * span) {
    sign = 1.f;
    partner = lane - span;
  }
  const int hkv = 1 << p.hkv_shift;
  const int tokens = max(1, kUnits >> p.hkv_shift);  // tokens of a pass (16 / hkv: hkv <= 8)
  __syncthreads();
  int buf = 0;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kUnits; first < p.units;
       first += static_cast<int64_t>(gridDim.x) * kUnits, buf ^= 1) {
    const int64_t unit = first + u;
    const bool live = unit < p.units;
    const int64_t t = unit >> p.hkv_shift;
    const int g = static_cast<int>(unit) & (hkv - 1);
    uint4 q0 = {}, q1 = {}, k0 = {}, v0 = {};
    int64_t slot = -1;
    if (live) {
      const uint16_t* qr = p.q + t * p.q_stride + 2 * g * kHeadDim + 8 * c;
      q0 = load_row16(qr);
      q1 = load_row16(qr + kHeadDim);
      k0 = load_row16(p.k + t * p.k_stride + g * kHeadDim + 8 * c);
      v0 = load_row16(p.v + t * p.v_stride + g * kHeadDim + 8 * c);
      slot = p.slots[t];
    }
    // the pass's first token is a whole one: kUnits is a multiple of the KV heads
    for (int i = tid; i < tokens * kMaxPairs; i += kThreads) {
      const int64_t tt = (first >> p.hkv_shift) + (i >> 6);
      const int j = i & (kMaxPairs - 1);
      if (j < pairs && (tt << p.hkv_shift) < p.units) {
        const long long pos = p.positions[tt];
        const unsigned long long phase = static_cast<unsigned long long>(pos) * turn[j];
        // the signed upper half: [-1/2, 1/2) turns, in half turns for sincospif
        const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * (1.0f / 2147483648.0f);
        float sn, cs;
        sincospif(half_turns, &sn, &cs);
        cos_s[buf][i >> 6][j] = cs * p.attn_factor;
        sin_s[buf][i >> 6][j] = sn * p.attn_factor;
      }
    }
    __syncthreads();
    // (the other buffer is rewritten only after every thread has passed this barrier)
    float cs[8], sn[8];
    const int row = u >> p.hkv_shift;
    if (kInterleaved) {
      const int at = 8 * c < p.rot ? 4 * c : 0;
      const float4 a = *reinterpret_cast<const float4*>(&cos_s[buf][row][at]);
      const float4 b = *reinterpret_cast<const float4*>(&sin_s[buf][row][at]);
      cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w;
      sn[0] = b.x; sn[1] = b.y; sn[2] = b.z; sn[3] = b.w;
    } else {
      const int at = c < span ? 8 * c : (c < 2 * span ? 8 * (c - span) : 0);
      load8(&cos_s[buf][row][at], cs);
      load8(&sin_s[buf][row][at], sn);
    }
    const uint4 q0r = turn_row<kInterleaved>(q0, p.q_gamma, p.eps, c, partner, sign, cs, sn);
    const uint4 q1r = turn_row<kInterleaved>(q1, p.q_gamma, p.eps, c, partner, sign, cs, sn);
    const uint4 k0r = turn_row<kInterleaved>(k0, p.k_gamma, p.eps, c, partner, sign, cs, sn);
    if (slot >= p.num_slots) {
      if (c == 0) flag_error(p.status, PA_DEV_ERR_PAGE_OOB);
      slot = -1;
    }
    if (slot >= 0) {  // a negative slot: a padding row, nothing is written
      uint16_t* qo = p.q_out + (t * (2 * hkv) + 2 * g) * kHeadDim + 8 * c;
      *reinterpret_cast<uint4*>(qo) = q0r;
      *reinterpret_cast<uint4*>(qo + kHeadDim) = q1r;
      const int64_t at = (slot * hkv + g) * kHeadDim + 8 * c;
      *reinterpret_cast<uint4*>(p.k_pool + at) = k0r;
      *reinterpret_cast<uint4*>(p.v_pool + at) = v0;
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
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(passes, static_cast<int64_t>(sms) * kCtasPerSm));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (interleaved) rope_append_kernel<true><<<grid, kThreads, 0, st>>>(p);
  else rope_append_kernel<false><<<grid, kThreads, 0, st>>>(p);
  PA_CHECK_LAUNCH("rope_append_kernel");
  return PA_OK;
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
