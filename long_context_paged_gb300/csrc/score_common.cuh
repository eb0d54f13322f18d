// Score options of attn_decode_paged_score and attn_prefill_chunk_score: host checks and the
// arithmetic both attention kernels share.
//
// A row at position i sees key j when j < prefix, or first <= j <= i with
// first = max(row_start, i - window + 1). Its score is
//     s = softmax_scale <q, k>;  s <- cap tanh(s / cap);  s <- s - slope |i - j|.
// The kernels work in log2 units and count a bias's distances from the row's nearest visible key:
// the term they leave out, slope * nearest, is common to the row, so it only moves the log-sum-exp
// and is added there at the end. A row that sees nothing near (only a prefix far behind it) would
// otherwise have scores of -slope * 10^5, whose fp32 steps of 2^-8 are errors of the weights.
#pragma once

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "pa_common.cuh"

namespace pa {

struct ScoreParams {
  float cap_log2;         // softcap * log2 e; 0: no cap
  const float* slopes;    // [Hq] or null
  int32_t window;         // 0: no limit
  const int32_t* prefix;  // [batch] or null
  int32_t max_prefix;
  const int32_t* row_start;  // [rows] or null
  // softcap * log2 e * tanh(q_scale * s) of a raw product s as an odd polynomial s P(s^2), for
  // |s| <= poly_max (|q_scale s| <= 1; negative: not usable, not even for products of 0: scores are
  // then capped one by one)
  float poly[7], poly_max;
};

// Coefficients of x P(x^2) nearest to tanh x on |x| <= 1: least maximum error over a dense grid by
// iteratively reweighted least squares (Lawson), rounded to fp32. The error, 2.4e-8, times a cap of 50
// is 2^-19 of a score; the fp32 evaluation adds roundings of up to 2^-23, of either sign.
constexpr int kTanhTerms = 7;
__host__ __device__ constexpr double tanh_coefficient(int k) {
  constexpr double c[kTanhTerms] = {9.999997020e-01, -3.333213031e-01, 1.331958324e-01, -5.326583609e-02,
                                    1.997328550e-02, -5.951282568e-03, 9.637727635e-04};
  return c[k];
}

inline bool score_opts_valid(const pa_score_opts& o) {
  return (o.softcap == 0.f || (o.softcap >= 1e-6f && o.softcap < 1e30f)) && o.window >= 0 && o.max_prefix_len >= 0 &&
         o.max_prefix_len <= 131072;
}

// Keys a row can see at most, rounded up to whole pages: what the launch plans are sized by.
inline int score_max_visible(const pa_score_opts& o, int max_seq_len) {
  if (o.window <= 0) return max_seq_len;
  // the window may cut a page at each end, the prefix one
  const int64_t keys = static_cast<int64_t>(o.window) + 2 * kPage +
                       (o.prefix_lens != nullptr ? o.max_prefix_len + kPage : 0);
  return static_cast<int>(std::min<int64_t>(max_seq_len, keys));
}

// q's factor (*q_scale): the softmax scale in log2 units or, with a cap, over the cap.
inline ScoreParams score_params(const pa_score_opts& o, float softmax_scale, float* q_scale) {
  ScoreParams s{};
  s.cap_log2 = o.softcap * kLog2e;
  s.slopes = o.alibi_slopes;
  s.window = o.window;
  s.prefix = o.max_prefix_len > 0 ? o.prefix_lens : nullptr;
  s.max_prefix = o.max_prefix_len;
  s.row_start = o.row_start;
  *q_scale = o.softcap > 0.f ? softmax_scale / o.softcap : softmax_scale * kLog2e;
  s.poly_max = -1.f;
  const double x = *q_scale;
  // the folded coefficients, down to softcap x^13 and up to softcap x, stay in fp32's range
  if (o.softcap > 0.f && o.softcap <= 1e6f && x >= 0x1p-10 && x <= 0x1p4) {
    double a = static_cast<double>(s.cap_log2) * x;
    for (int k = 0; k < kTanhTerms; ++k, a *= x * x) s.poly[k] = static_cast<float>(tanh_coefficient(k) * a);
    s.poly_max = static_cast<float>(1.0 / x);
  }
  return s;
}

// Prefix of sequence b: negative or past the host's bound is cut and flagged.
__device__ __forceinline__ int score_prefix(const ScoreParams& s, int b, int32_t* status, bool report) {
  if (s.prefix == nullptr) return 0;
  const int n = s.prefix[b];
  if (n >= 0 && n <= s.max_prefix) return n;
  if (report) flag_error(status, PA_DEV_ERR_LENGTH);
  return n < 0 ? 0 : s.max_prefix;
}

// First key of a row's own range: 0 <= first; first > i when the row sees no key of its own.
__device__ __forceinline__ int score_first_key(const ScoreParams& s, int row, int i) {
  int lo = s.row_start != nullptr ? max(s.row_start[row], 0) : 0;
  if (s.window > 0) lo = max(lo, i - s.window + 1);
  return lo;
}

// A head's slope in log2 units, over `scale`. A finite slope stays finite: at distance 0 its bias
// is 0.
__device__ __forceinline__ float slope_over(const ScoreParams& s, int head, float scale) {
  const float a = s.slopes[head], r = a * kLog2e / scale;
  return isinf(r) && !isinf(a) ? copysignf(3.402823466e38f, a) : r;
}

// tanh by one exponential: 1 - 2 / (e^{2x} + 1), within 2^-22 absolutely (near 0 the exponential's
// error of 2^-22 counts half and the quotient is near 1); exact at the ends (e^{2x} = inf gives 1, 0
// gives -1), NaN stays NaN.
__device__ __forceinline__ float tanh_exp(float x) {
  return 1.0f - __fdividef(2.0f, fast_exp2(x * (2.0f * kLog2e)) + 1.0f);
}

// tanh of a score: the polynomial up to |x| = 1; beyond it the exponential form, whose errors shrink
// there with 1 - tanh^2 and the quotient. A cap of 50 makes an absolute error of 2^-22 one of 10^-5 in
// the log-sum-exp of a row with few keys, 2^-24 one that fp32 has anyway.
__device__ __forceinline__ float tanh_score(float x) {
  const float t = x * x;
  float y = static_cast<float>(tanh_coefficient(kTanhTerms - 1));
#pragma unroll
  for (int k = kTanhTerms - 2; k >= 0; --k) y = fmaf(y, t, static_cast<float>(tanh_coefficient(k)));
  return t <= 1.0f ? y * x : tanh_exp(x);
}

// The score in log2 units of q's scaled product x: capped, then the bias at `distance` (from the
// nearest visible key) of a head of slope slope2 / log2 e.
__device__ __forceinline__ float score_of(const ScoreParams& s, float x, float slope2, int distance) {
  if (s.cap_log2 != 0.f) x = s.cap_log2 * tanh_score(x);
  if (s.slopes != nullptr) x = fmaf(-slope2, static_cast<float>(distance), x);
  return x;
}

}  // namespace pa
