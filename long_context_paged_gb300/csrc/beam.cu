// beam_select: the best k continuations of each request's beams, over beams and vocabulary (sm_103a).
//
// Candidate (b, v) of a request has the score
//     scores[b] + logits[b][v] - ln sum_u exp(logits[b][u])
// and the k best are kept, equal scores in the order of (b, v). Within a beam the order is that of the
// logits themselves, whatever the beam's score and normaliser: so one pass over a beam's logits finds
// both its normaliser (running maximum and sum) and its k largest logits, and only those few meet the
// other beams' in a second launch. Scores are formed as pairs of floats there (48 bits): what decides
// between beams is the normalisers' precision (fp32 sums of exponentials), not the rounding of a sum
// of large parts.
//
// The logits are read once from memory. A row is cut into pieces so that a few rows still fill the GPU; a CTA
// takes a piece, a thread 16-byte vectors kThreads apart. Measured on a GB300 (calls of a graph): 64 x 8 rows
// of 151,936 in bf16 42 us (147 MB: 21.6 us at a copy's rate), the first launch 34 of them, bound by
// instruction issue (64 % of the busy SMs' slots; 3.5 TB/s): 5 an element to unpack, exponentiate and add,
// as many again per piece for the selection; 16 x 5 rows of 51,865 in fp32 14.8 us; one request 8.5 us, two
// launches of dependent loads. Candidate selection by k rounds of a block-wide maximum took 477 us for the
// first of these; scores in fp64 in the second launch cost it 4 us of 14 (this GPU's fp64 rate is 1/60 of fp32's).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dependent_launch.cuh"
#include "pa_common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBeams = 64;
constexpr int kMaxK = 64;
constexpr int kMaxRows = 65535;
constexpr int kList = 1024;  // candidates of a piece that the quick selection holds
constexpr int kFound = 512;  // candidates of a request that the quick ranking holds
// Pieces of a row: as many as give kTargetCtas CTAs in all (three rounds of what the GPU holds, so that one
// CTA's selection runs beside another's loads), none of them below four vectors a thread.
constexpr int kTargetCtas = 2736;
constexpr int kMinVectors = 4 * kThreads;

struct BeamParams {
  const void* logits;
  int64_t row_stride;
  int32_t requests, beams, vocab, k, eos, pieces;
  const float* scores;
  const int32_t* live;
  float* out_scores;
  int32_t* parents;
  int32_t* tokens;
  int32_t* live_out;
  // workspace: of each row and piece, the k largest logits in order, and (maximum, sum of exp)
  float2* best;   // [rows][pieces][k]: value, token as bits (-1: none)
  float2* stats;  // [rows][pieces]
};

// fp32 as an unsigned integer of the same order; -inf and NaN are 0, below everything else.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (!(x > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);  // (-0 and 0 are equal)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

__device__ __forceinline__ uint64_t warp_max64(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u;
  return static_cast<uint64_t>(hi) << 32 | __reduce_max_sync(0xffffffffu, lo);
}

// A row's beam takes part with its tokens: it is live and has a score. (-inf: not in use.)
__device__ __forceinline__ bool expands(const BeamParams& p, int row) {
  const float s = p.scores[row];
  return (p.live == nullptr || p.live[row] != 0) && s > -INFINITY && s < INFINITY;
}

// The row's logits as 16-byte vectors of kVec, after `head` and before `tail` single ones.
template <class T>
struct Row {
  static constexpr int kVec = 16 / sizeof(T);
  const T* base;
  int head, vectors, tail;
  __device__ Row(const T* b, int n) : base(b) {
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(b) & 15u) / sizeof(T));
    head = min(n, off == 0 ? 0 : kVec - off);
    vectors = (n - head) / kVec;
    tail = n - head - vectors * kVec;
  }
};

__device__ __forceinline__ void unpack(uint4 w, float (&x)[8]) {
  x[0] = bf16lo(w.x); x[1] = bf16hi(w.x); x[2] = bf16lo(w.y); x[3] = bf16hi(w.y);
  x[4] = bf16lo(w.z); x[5] = bf16hi(w.z); x[6] = bf16lo(w.w); x[7] = bf16hi(w.w);
}
__device__ __forceinline__ void unpack(uint4 w, float (&x)[4]) {
  x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
  x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ float single(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ float single(float v) { return v; }

// A logit's rank among a row's: by value, then the lower token.
__device__ __forceinline__ uint64_t rank_of(float x, int token) {
  const uint32_t o = order_of(x);
  return o == 0 ? 0ull : static_cast<uint64_t>(o) << 32 | ~static_cast<uint32_t>(token);
}

// A thread's state over its logits: the largest, and the sum of exponentials against a reference that
// follows the largest at a distance (40 at most: sums stay below 2^77), so that nothing is rescaled at
// every new maximum.
struct Seen {
  float top = -INFINITY, ref = -INFINITY, sum = 0.f;

  // The largest of the next logits.
  __device__ __forceinline__ void reach(float most) {
    if (most > ref + 40.f) {
      sum = ref == -INFINITY ? 0.f : sum * fast_exp2((ref - most) * kLog2e);
      ref = most;
    }
    top = fmaxf(top, most);
  }
  // Those logits. (x - ref, then the factor: one rounding each, so no error that all terms share.)
  __device__ __forceinline__ void take(float x) { sum += fast_exp2((x - (ref == -INFINITY ? 0.f : ref)) * kLog2e); }
  template <int n>
  __device__ __forceinline__ void take(const float (&x)[n]) {
    const float base = ref == -INFINITY ? 0.f : -ref;
    const float2 minus = make_float2(base, base), log2e = make_float2(kLog2e, kLog2e);
    float2 part = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < n; i += 2) {
      const float2 e = mul2(add2(make_float2(x[i], x[i + 1]), minus), log2e);
      part = add2(part, make_float2(fast_exp2(e.x), fast_exp2(e.y)));
    }
    sum += part.x + part.y;
  }
};

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The largest logit of a vector, and of four.
__device__ __forceinline__ float most_of(uint4 w, uint16_t) {
  const uint32_t m = max_bf16x2(max_bf16x2(w.x, w.y), max_bf16x2(w.z, w.w));
  return fmaxf(bf16lo(m), bf16hi(m));
}
__device__ __forceinline__ float most_of(uint4 w, float) {
  return fmax3(__uint_as_float(w.x), __uint_as_float(w.y), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
}
__device__ __forceinline__ float most_of(const uint4 (&w)[4], uint16_t) {
  uint32_t m[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) m[j] = max_bf16x2(max_bf16x2(w[j].x, w[j].y), max_bf16x2(w[j].z, w[j].w));
  const uint32_t all = max_bf16x2(max_bf16x2(m[0], m[1]), max_bf16x2(m[2], m[3]));
  return fmaxf(bf16lo(all), bf16hi(all));
}
__device__ __forceinline__ float most_of(const uint4 (&w)[4], float) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m = fmax3(m, __uint_as_float(w[j].x), __uint_as_float(w[j].y));
    m = fmax3(m, __uint_as_float(w[j].z), __uint_as_float(w[j].w));
  }
  return m;
}

template <class T>
__global__ void __launch_bounds__(kThreads) beam_rows_kernel(const BeamParams p) {
  constexpr int kVec = Row<T>::kVec;
  __shared__ uint64_t warp_best[kWarps], list[kList];
  __shared__ uint32_t warp_bound[kWarps];
  __shared__ float2 warp_stats[kWarps];
  __shared__ int found, holding;
  __shared__ uint8_t holders[kThreads];
  const int row = static_cast<int>(blockIdx.y), piece = static_cast<int>(blockIdx.x);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) found = holding = 0;
  launch_next();
  await_previous();
  if (!expands(p, row)) return;
  const Row<T> r(static_cast<const T*>(p.logits) + row * p.row_stride, p.vocab);
  const uint4* body = reinterpret_cast<const uint4*>(r.base + r.head);
  int per = (r.vectors + p.pieces - 1) / p.pieces;
  // long pieces in whole rounds of four vectors a thread (the last one is shorter)
  if (per > 3 * kMinVectors) per = (per + kMinVectors - 1) / kMinVectors * kMinVectors;
  const int v0 = min(r.vectors, piece * per), v1 = min(r.vectors, v0 + per);
  // the first piece has the single logits before the vectors, the last those after
  const int lead = piece == 0 ? r.head : 0, trail = piece == p.pieces - 1 ? r.tail : 0;
  const int trail_at = r.head + r.vectors * kVec;
  Seen seen;
  if (tid < lead) {
    const float x = single(r.base[tid]);
    seen.reach(x);
    seen.take(x);
  }
  int v = v0 + tid;
  for (; v + 3 * kThreads < v1; v += 4 * kThreads) {
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = body[v + j * kThreads];
    seen.reach(most_of(w, T()));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[kVec];
      unpack(w[j], x);
      seen.take(x);
    }
  }
  for (; v < v1; v += kThreads) {
    const uint4 w = body[v];
    float x[kVec];
    unpack(w, x);
    seen.reach(most_of(w, T()));
    seen.take(x);
  }
  if (tid < trail) {
    const float x = single(r.base[trail_at + tid]);
    seen.reach(x);
    seen.take(x);
  }
  // A bound that k logits at least reach: the q-th best thread of each warp that has vectors (q of them
  // make k; a thread counts by its largest logit), and of those the least.
  const uint32_t mine = order_of(seen.top);
  const int warps = min(kWarps, max(1, (v1 - v0 + 31) / 32));
  uint32_t bound = 0;
  if (warp < warps) {
    uint32_t left = mine;
    for (int q = (p.k + warps - 1) / warps; q > 0; --q) {
      bound = __reduce_max_sync(0xffffffffu, left);
      if (lane == __ffs(__ballot_sync(0xffffffffu, left == bound)) - 1) left = 0;
    }
  }
  // maximum and sum of the CTA
  float wm = seen.top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
  float ws = seen.ref == wm ? seen.sum : seen.sum * fast_exp2((seen.ref - wm) * kLog2e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
  if (lane == 0) {
    warp_stats[warp] = make_float2(wm, ws);
    warp_bound[warp] = bound;
  }
  __syncthreads();
  const int64_t out = static_cast<int64_t>(row) * p.pieces + piece;
  if (tid == 0) {
    float cm = -INFINITY, cs = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) cm = fmaxf(cm, warp_stats[w].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      cs += warp_stats[w].x == cm ? warp_stats[w].y : warp_stats[w].y * fast_exp2((warp_stats[w].x - cm) * kLog2e);
    p.stats[out] = make_float2(cm, cs);
  }
  bound = warp_bound[0];
  for (int w = 1; w < warps; ++w) bound = min(bound, warp_bound[w]);
  // Logits that reach the bound go to a list. Only threads whose own largest reaches it have one: they are
  // listed, and all threads look through those threads' vectors (a second read of a small part of the
  // piece, from L2 mostly).
  const float least = bound > 0 ? value_of(bound) : -INFINITY;
  const bool holds = mine > 0 && mine >= bound;
  auto keep = [&](float x, int token) {
    if (!(x >= least) || x == -INFINITY) return;
    const int i = atomicAdd(&found, 1);
    if (i < kList) list[i] = rank_of(x, token);
  };
  if (tid < lead) keep(single(r.base[tid]), tid);
  if (tid < trail) keep(single(r.base[trail_at + tid]), trail_at + tid);
  if (holds) holders[atomicAdd(&holding, 1)] = static_cast<uint8_t>(tid);
  __syncthreads();
  const int each = (v1 - v0 + kThreads - 1) / kThreads, looks = holding * each;
  for (int i = tid; i < looks; i += kThreads) {
    const int of = i / each, v = v0 + holders[of] + (i - of * each) * kThreads;
    if (v >= v1) continue;
    const uint4 w = body[v];
    if (!(most_of(w, T()) >= least)) continue;  // most vectors
    float x[kVec];
    unpack(w, x);
#pragma unroll
    for (int j = 0; j < kVec; ++j) keep(x[j], r.head + v * kVec + j);
  }
  __syncthreads();
  const int n = found;
  if (n <= kList) {
    // an entry's place is the number of those above it
    for (int i = tid; i < max(n, p.k); i += kThreads) {
      if (i >= n) {
        p.best[out * p.k + i] = make_float2(-INFINITY, __int_as_float(-1));
        continue;
      }
      const uint64_t c = list[i];
      int place = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) place += list[j] > c ? 1 : 0;
      if (place < p.k)
        p.best[out * p.k + place] = make_float2(value_of(static_cast<uint32_t>(c >> 32)),
                                                __int_as_float(static_cast<int>(~static_cast<uint32_t>(c))));
    }
    return;
  }
  // More than the list holds (most of a row's logits alike or banned, in a pattern that leaves a warp
  // without a high one): the k largest one after the other, each found below the last.
  uint64_t top = ~0ull;
  for (int k = 0; k < p.k; ++k) {
    uint64_t best = 0;
    auto look = [&](float x, int token) {
      const uint64_t c = rank_of(x, token);
      if (c < top) best = max(best, c);
    };
    if (holds || lead > 0 || trail > 0) {
      if (tid < lead) look(single(r.base[tid]), tid);
      if (tid < trail) look(single(r.base[trail_at + tid]), trail_at + tid);
      for (int v = v0 + tid; v < v1; v += kThreads) {
        float x[kVec];
        unpack(body[v], x);
#pragma unroll
        for (int i = 0; i < kVec; ++i) look(x[i], r.head + v * kVec + i);
      }
    }
    best = warp_max64(best);
    if (lane == 0) warp_best[warp] = best;
    __syncthreads();
    top = warp_best[0];
    for (int w = 1; w < kWarps; ++w) top = max(top, warp_best[w]);
    __syncthreads();
    if (tid == 0)
      p.best[out * p.k + k] = make_float2(value_of(static_cast<uint32_t>(top >> 32)),
                                          __int_as_float(top == 0 ? -1 : static_cast<int>(~static_cast<uint32_t>(top))));
  }
}

// Scores as a pair of floats whose sum they are, lo at most half a step of hi (48 bits: fp64 is 50 times
// slower here, and took most of this launch).
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair exact_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return Pair{s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Pair add(Pair a, float b) {
  const Pair s = exact_sum(a.hi, b);
  return exact_sum(s.hi, s.lo + a.lo);
}
// ln x, of a normal x >= 2^-1 below 2^31: x = 2^e f with f in [3/4, 3/2), so that logf is off by half a step
// of at most 0.41 (3e-8) and the rest is nearly exact; e times the high part of ln 2 (14 bits) is exact.
__device__ __forceinline__ Pair natural_log(float x) {
  const int e = (__float_as_int(x) - 0x3f400000) >> 23;
  const float f = __int_as_float(__float_as_int(x) - (e << 23));
  constexpr float kHigh = 11357.f / 16384.f, kLow = -2.9088971304691e-5f;  // ln 2
  return exact_sum(e * kHigh, logf(f) + e * kLow);
}
// A pair as an integer of the same order; 0, below all, if it is -inf or NaN.
__device__ __forceinline__ uint64_t order_of(Pair x) {
  const uint32_t hi = order_of(x.hi);
  return hi == 0 ? 0ull : static_cast<uint64_t>(hi) << 32 | order_of(x.lo);
}

// A candidate of a request: its score's order, and its place.
struct Candidate {
  uint64_t score;
  uint32_t place;  // ~(beam * vocab + token): a lower place is a larger number
};
__device__ __forceinline__ bool better(const Candidate& a, const Candidate& b) {
  return (a.score > b.score) | ((a.score == b.score) & (a.place > b.place));  // (no branches)
}

__global__ void __launch_bounds__(kThreads) beam_merge_kernel(const BeamParams p) {
  __shared__ Pair shift[kMaxBeams];    // score minus normaliser of a beam
  __shared__ uint8_t kind[kMaxBeams];  // 0: no candidates, 1: its tokens, 2: itself (finished)
  __shared__ Candidate warp_best[kWarps];
  __shared__ Candidate list[kFound];
  __shared__ int found;
  extern __shared__ uint8_t used[];    // [beams][pieces] candidates taken
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = static_cast<int>(blockIdx.x), lists = p.beams * p.pieces;
  await_previous();
  if (tid == 0) found = 0;
  for (int i = tid; i < lists; i += kThreads) used[i] = 0;
  for (int b = warp; b < p.beams; b += kWarps) {
    const int row = n * p.beams + b;
    const float2* stats = p.stats + static_cast<int64_t>(row) * p.pieces;
    // (read beside the score and the flag; of a row that is not expanded it is whatever was there)
    const float2 mine = lane < p.pieces ? stats[lane] : make_float2(-INFINITY, 0.f);
    if (!expands(p, row)) {
      if (lane == 0) {
        const float s = p.scores[row];
        kind[b] = p.live != nullptr && p.live[row] == 0 && s > -INFINITY && s < INFINITY ? 2 : 0;
        shift[b] = Pair{s, 0.f};
      }
      continue;
    }
    float m = mine.x;
    for (int i = 32 + lane; i < p.pieces; i += 32) m = fmaxf(m, stats[i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    Pair sum{mine.x == m ? mine.y : mine.y * fast_exp2((mine.x - m) * kLog2e), 0.f};
    for (int i = 32 + lane; i < p.pieces; i += 32) {
      const float2 v = stats[i];
      sum = add(sum, v.x == m ? v.y : v.y * fast_exp2((v.x - m) * kLog2e));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float hi = __shfl_xor_sync(0xffffffffu, sum.hi, o), lo = __shfl_xor_sync(0xffffffffu, sum.lo, o);
      // (lanes add the same two pairs in the same order)
      sum = lane & o ? add(Pair{hi, lo + sum.lo}, sum.hi) : add(Pair{sum.hi, sum.lo + lo}, hi);
    }
    if (lane == 0) {
      // (a NaN or +inf among the logits, or nothing but -inf: no candidates)
      const bool good = m > -INFINITY && m < INFINITY && sum.hi >= 0.5f && sum.hi < 2147483648.f;
      kind[b] = good ? 1 : 0;
      if (good) {
        const Pair norm = natural_log(sum.hi);  // (sum.lo is below 2^-24 of it: ln moves by as much)
        Pair s = exact_sum(p.scores[row], -m);
        s = add(s, -norm.hi);
        shift[b] = add(s, -(norm.lo + sum.lo / sum.hi));
      }
    }
  }
  __syncthreads();
  const float2* entries = p.best + static_cast<int64_t>(n) * lists * p.k;
  auto candidate = [&](int b, float2 e) {
    Candidate c{0, 0};
    const int token = __float_as_int(e.y);
    if (token >= 0) {
      c.score = order_of(add(shift[b], e.x));
      c.place = ~static_cast<uint32_t>(b * p.vocab + token);
    }
    return c;
  };
  auto entry = [&](int list, int at) {
    const int b = list / p.pieces;
    Candidate c{0, 0};
    if (kind[b] == 1 && at < p.k) {
      c = candidate(b, entries[static_cast<int64_t>(list) * p.k + at]);
    } else if (kind[b] == 2 && at == 0 && list == b * p.pieces) {
      c.score = order_of(shift[b]);
      c.place = ~static_cast<uint32_t>(b * p.vocab + max(p.eos, 0));
    }
    return c;
  };
  auto write = [&](int place, const Candidate& c) {
    const int at = n * p.k + place;
    if (c.score == 0) {
      p.out_scores[at] = -INFINITY;
      p.parents[at] = p.tokens[at] = -1;
      p.live_out[at] = 0;
      return;
    }
    const uint32_t index = ~c.place;
    const int b = static_cast<int>(index / static_cast<uint32_t>(p.vocab));
    const int token = kind[b] == 2 ? p.eos : static_cast<int>(index - static_cast<uint32_t>(b) * p.vocab);
    p.out_scores[at] = value_of(static_cast<uint32_t>(c.score >> 32));
    p.parents[at] = b;
    p.tokens[at] = token;
    p.live_out[at] = kind[b] == 1 && token != p.eos ? 1 : 0;
  };
  // A bound that k candidates at least reach, as in the first launch: from the best heads of each warp's
  // lists (by score alone: equal ones all count). Candidates that reach it, in their lists' order, are ranked.
  {
    // (the lists go round the warps, so that every warp has some of each beam)
    const int first = lane * kWarps + warp;
    uint64_t best = 0;
    for (int i = first; i < lists; i += kThreads) best = max(best, entry(i, 0).score);
    const int warps = min(kWarps, lists);
    uint64_t bound = 0;
    if (warp < warps) {
      uint64_t left = best;
      for (int q = (p.k + warps - 1) / warps; q > 0; --q) {
        bound = warp_max64(left);
        // one thread of those that have it
        const uint32_t same = __ballot_sync(0xffffffffu, left == bound);
        if (lane == __ffs(same) - 1) left = 0;
      }
    }
    if (lane == 0) warp_best[warp] = Candidate{bound, 0};
    __syncthreads();
    bound = warp_best[0].score;
    for (int w = 1; w < warps; ++w) bound = min(bound, warp_best[w].score);
    bound = max(bound, static_cast<uint64_t>(1));
    if (best >= bound) {
      for (int i = first; i < lists; i += kThreads) {
        const int b = i / p.pieces;
        auto keep = [&](const Candidate& c) {
          if (c.score < bound) return false;
          const int to = atomicAdd(&found, 1);
          if (to < kFound) list[to] = c;
          return true;
        };
        if (kind[b] != 1) {
          keep(entry(i, 0));
          continue;
        }
        // four entries' loads at a time
        const float2* e = entries + static_cast<int64_t>(i) * p.k;
        bool more = true;
        for (int at = 0; at < p.k && more; at += 4) {
          float2 v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = at + j < p.k ? e[at + j] : make_float2(0.f, __int_as_float(-1));
#pragma unroll
          for (int j = 0; j < 4; ++j) more = more && keep(candidate(b, v[j]));
        }
      }
    }
    __syncthreads();
    const int m = found;
    if (m <= kFound) {
      for (int i = tid; i < max(m, p.k); i += kThreads) {
        if (i >= m) {
          write(i, Candidate{0, 0});
          continue;
        }
        const Candidate c = list[i];
        int place = 0;
#pragma unroll 8
        for (int j = 0; j < m; ++j) place += better(list[j], c) ? 1 : 0;
        if (place < p.k) write(place, c);
      }
      return;
    }
  }
  // More than the list holds: one after the other, each thread with the heads of its lists.
  auto mine = [&](int& from) {
    Candidate c{0, 0};
    for (int i = tid; i < lists; i += kThreads) {
      const Candidate h = entry(i, used[i]);
      if (better(h, c)) {
        c = h;
        from = i;
      }
    }
    return c;
  };
  int from = -1;
  Candidate best = mine(from);
  for (int k = 0; k < p.k; ++k) {
    Candidate c = best;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Candidate other;
      other.score = __shfl_xor_sync(0xffffffffu, c.score, o);
      other.place = __shfl_xor_sync(0xffffffffu, c.place, o);
      if (better(other, c)) c = other;
    }
    if (lane == 0) warp_best[warp] = c;
    __syncthreads();
    Candidate top = warp_best[0];
    for (int w = 1; w < kWarps; ++w)
      if (better(warp_best[w], top)) top = warp_best[w];
    __syncthreads();
    if (top.score == 0) {
      if (tid == 0) write(k, top);
    } else if (best.score == top.score && best.place == top.place) {
      write(k, top);
      ++used[from];
      best = mine(from);
    }
  }
}

int pieces_of(int32_t requests, int32_t beams, int32_t vocab, int32_t logits_type) {
  const int64_t rows = std::max<int64_t>(1, static_cast<int64_t>(requests) * beams);
  const int64_t most = std::max<int64_t>(1, vocab / (kMinVectors * (logits_type == PA_BF16 ? 8 : 4)));
  return static_cast<int>(std::min(most, std::max<int64_t>(1, kTargetCtas / rows)));
}

bool beam_sizes_valid(int32_t requests, int32_t beams, int32_t vocab, int32_t k) {
  return requests >= 0 && beams > 0 && vocab > 0 && k > 0;
}

bool beam_sizes_supported(int32_t requests, int32_t beams, int32_t vocab, int32_t k) {
  return beams <= kMaxBeams && k <= kMaxK && static_cast<int64_t>(beams) * vocab < (1ll << 31) &&
         static_cast<int64_t>(requests) * beams <= kMaxRows;
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_beam_workspace_size(int32_t requests, int32_t beams, int32_t vocab, int32_t k) {
  using namespace pa;
  if (!beam_sizes_valid(requests, beams, vocab, k) || !beam_sizes_supported(requests, beams, vocab, k)) return 0;
  const size_t lists = static_cast<size_t>(requests) * beams * pieces_of(requests, beams, vocab, PA_FP32);  // (the most)
  return (lists * (k + 1) * sizeof(float2) + 255) / 256 * 256;
}

extern "C" pa_status beam_select(const void* logits, int32_t logits_type, int64_t row_stride, int32_t requests,
                                 int32_t beams, int32_t vocab, const float* scores, const int32_t* live, int32_t k,
                                 int32_t eos_token, float* out_scores, int32_t* parents, int32_t* tokens,
                                 int32_t* live_out, void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  using namespace pa;
  if (!beam_sizes_valid(requests, beams, vocab, k) || row_stride < vocab || eos_token < -1 || eos_token >= vocab ||
      (logits_type != PA_BF16 && logits_type != PA_FP32))
    return PA_ERR_INVALID_ARG;
  if (!beam_sizes_supported(requests, beams, vocab, k)) {
    snprintf_error("beam_select: at most %d beams of a request, %d candidates, 2^31 tokens of all its beams and %d rows",
                   kMaxBeams, kMaxK, kMaxRows);
    return PA_ERR_UNSUPPORTED;
  }
  // in place: a request's results replace its own inputs only if there are as many
  if (k != beams && ((out_scores && out_scores == scores) || (live && live_out == live))) return PA_ERR_INVALID_ARG;
  if (requests == 0) return PA_OK;
  if (!logits || !scores || !out_scores || !parents || !tokens || !live_out) return PA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) & (logits_type == PA_BF16 ? 1u : 3u)) return PA_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < pa_beam_workspace_size(requests, beams, vocab, k))
    return PA_ERR_WORKSPACE_TOO_SMALL;
  if (reinterpret_cast<uintptr_t>(workspace) & 7u) return PA_ERR_INVALID_ARG;
  const int pieces = pieces_of(requests, beams, vocab, logits_type);
  const size_t lists = static_cast<size_t>(requests) * beams * pieces;
  float2* best = static_cast<float2*>(workspace);
  const BeamParams p{logits, row_stride, requests, beams, vocab, k, eos_token, pieces, scores, live, out_scores,
                     parents, tokens, live_out, best, best + lists * k};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(pieces), static_cast<unsigned>(requests * beams));
  cudaError_t e = logits_type == PA_BF16 ? launch_dependent(beam_rows_kernel<uint16_t>, grid, kThreads, 0, st, 0, p)
                                         : launch_dependent(beam_rows_kernel<float>, grid, kThreads, 0, st, 0, p);
  if (e == cudaSuccess)
    e = launch_dependent(beam_merge_kernel, static_cast<unsigned>(requests), kThreads,
                         static_cast<size_t>(beams) * pieces, st, 0, p);
  return e == cudaSuccess ? PA_OK : record_cuda_error(e, "beam_select");
}
