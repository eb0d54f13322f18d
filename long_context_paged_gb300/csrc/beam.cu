// beam_select: the best k continuations of each request's beams, over beams and vocabulary (sm_103a).
//
// Candidate (b, v) of a request has the score
//     scores[b] + logits[b][v] - ln sum_u exp(logits[b][u])
// and the k best are kept, equal scores in the order of (b, v). Within a beam that is the order of the logits
// themselves, whatever the beam's score and normaliser. So one pass over a beam's logits finds its
// normaliser (a sum against a running reference) and the largest logit of every unit, 2 KB of the row. With all beams'
// normalisers known the units are ordered by the scores of those (equal ones as they lie): the k best
// candidates are all in the k best units, since each of these has one candidate at least that comes before
// all of any other unit. The second launch looks through those k units alone. Scores are formed as pairs of
// floats there (48 bits; logits of a beam that differ by less than 2^-45 of its score may count as equal, or
// change places): what decides between beams is the normalisers' precision (below: Seen), not the rounding of a sum of
// large parts.
//
// The logits are read once from memory. A row is cut into pieces so that a few rows still fill the GPU; a CTA
// takes a piece, a warp a unit, a lane four 16-byte vectors of it. Measured on a GB300 (calls of a graph): 64 x 8 rows
// of 151,936 in bf16 36.5 us (147 MB: 21.6 us at a copy's rate), the first launch 25 of them, its instructions (5 an
// element to unpack, exponentiate and add) 0.6 of what the SMs can issue; 16 x 5 rows of 51,865 in fp32 12.4 us; one
// request 7.5 us. The second launch is a chain of some 1,000 instructions of each warp: normalisers 2 us, units 3,
// candidates 2.5. Choosing each piece's k largest in the first launch, for the second to join, took 41.4, 14.6 and
// 8.5 us (all of a piece's warps wait for its selection, three times); rounds of a block-wide maximum there 477 us
// for the first of these; scores in fp64 in the second launch cost it 4 us (this GPU's fp64 rate is 1/60 of fp32's).
#include <cuda_runtime.h>
#include <math_constants.h>
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
constexpr int kUnit = 128;   // 16-byte vectors of a unit: four a lane, 2 KB
constexpr int kUnits = 512;  // units that the quick choice of them holds
// Threads of the second launch: one for every vector of the k units that are looked through, at most 1,024. With 512
// and 1,024: 10 kept of 16 x 5 rows 13.0 and 11.6 us (both launches), 8 of 64 x 8 37.3 and 35.6, 4 of one request 7.1
// and 8.0; with 256 the last one 7.5.
constexpr int kPickFew = 512, kPickMany = 1024;
constexpr int kFound = 512;  // candidates that the quick ranking holds
constexpr int kFewFound = 128;  // so few are ranked sooner than a closer bound is found
// Pieces of a row: as many as give kTargetCtas CTAs in all (three rounds of the six that an SM holds), and at most
// one for every kWarps units or part of that many (9 units: pieces of 5 and 4, some warps without one). 64 x 8 rows with 912, 1,824, 2,736 and 5,472: 41.5, 39.4, 38.5 and 39.5 us at one stage of
// this kernel; registers for seven or eight CTAs an SM: 36 -> 38.
constexpr int kTargetCtas = 2736;

struct BeamParams {
  const void* logits;
  int64_t row_stride;
  int32_t requests, beams, vocab, k, eos;
  int32_t units, pieces;  // of a row
  uint32_t over_units;    // (2^32 - 1) / units
  const float* scores;
  const int32_t* live;
  float* out_scores;
  int32_t* parents;
  int32_t* tokens;
  int32_t* live_out;
  // workspace
  float2* stats;  // [rows][pieces] reference and sum of exponentials
  float* tops;    // [rows][units] largest logit
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

__device__ __forceinline__ uint64_t warp_min64(uint64_t v) {
  const uint32_t hi = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : ~0u;
  return static_cast<uint64_t>(hi) << 32 | __reduce_min_sync(0xffffffffu, lo);
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
  __device__ int last_unit() const { return max(0, (vectors + kUnit - 1) / kUnit - 1); }
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

// e to the difference of two references: expf is off by 2^-23 at most, and the difference is exact.
__device__ __forceinline__ float factor(float d) { return expf(d); }

// A thread's sum of exponentials over its logits, against a reference that follows the largest of them at a distance
// (kLag at most, so that little is rescaled). The distance is short because terms are formed from it: x - ref and
// its product with log2 e are rounded by 2^-24 |x - ref| each, an error that terms alike have alike. (A lag of 40, by
// which nothing is ever rescaled, left normalisers off by 5e-6, by what a thread happened to read first.) References are
// whole numbers, so that differences between them are exact. The sum is a pair of floats: its error is that of one
// vector's however many there are. In all a normaliser is off by at most 1.4e-7 y (y: distance below ref of the terms
// that matter, at most the logarithm of their number) + 2.4e-7 (ex2) + 24 * 2^-24 (sums of vectors, lanes, warps and
// pieces): 2^-18.
constexpr float kLag = 4.f;

struct Seen {
  float top = -INFINITY, ref = -INFINITY, sum = 0.f, low = 0.f;

  // The largest of the next logits.
  __device__ __forceinline__ void reach(float most) {
    if (most > ref + kLag) {
      const float to = rintf(most), f = factor(ref - to);  // (0 at first, which leaves a NaN)
      sum *= f;
      low *= f;
      ref = to;
    }
    top = fmaxf(top, most);
  }
  // The sum of those logits' terms. (x - ref, then the factor: one rounding each; a product folded into the difference
  // would overflow at the type's lowest value.)
  __device__ __forceinline__ float term(float x) const { return fast_exp2((x - (ref == -INFINITY ? 0.f : ref)) * kLog2e); }
  template <int n>
  __device__ __forceinline__ float terms(const float (&x)[n]) const {
    const float base = ref == -INFINITY ? 0.f : -ref;
    const float2 minus = make_float2(base, base), log2e = make_float2(kLog2e, kLog2e);
    float2 part = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < n; i += 2) {
      const float2 e = mul2(add2(make_float2(x[i], x[i + 1]), minus), log2e);
      part = add2(part, make_float2(fast_exp2(e.x), fast_exp2(e.y)));
    }
    return part.x + part.y;
  }
  __device__ __forceinline__ void add(float part) {
    const float s = sum + part, t = s - sum;
    low += (sum - (s - t)) + (part - t);
    sum = s;
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
  __shared__ float2 warp_stats[kWarps];
  const int row = static_cast<int>(blockIdx.y), piece = static_cast<int>(blockIdx.x);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  launch_next();
  await_previous();
  if (!expands(p, row)) return;
  const Row<T> r(static_cast<const T*>(p.logits) + row * p.row_stride, p.vocab);
  const uint4* body = reinterpret_cast<const uint4*>(r.base + r.head);
  const int per = (p.units + p.pieces - 1) / p.pieces, u1 = min(p.units, (piece + 1) * per);
  float* tops = p.tops + static_cast<int64_t>(row) * p.units;
  Seen seen;
  for (int u = piece * per + warp; u < u1; u += kWarps) {
    const int v = u * kUnit + lane;
    float most;
    if ((u + 1) * kUnit <= r.vectors) {
      uint4 w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = body[v + j * 32];
      most = most_of(w, T());
      seen.reach(most);
      float part[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x[kVec];
        unpack(w[j], x);
        part[j] = seen.terms(x);
      }
      seen.add((part[0] + part[1]) + (part[2] + part[3]));
    } else {  // the row's last unit
      most = -INFINITY;
      for (int i = v; i < min(r.vectors, (u + 1) * kUnit); i += 32) {
        const uint4 w = body[i];
        float x[kVec];
        unpack(w, x);
        const float m = most_of(w, T());
        seen.reach(m);
        seen.add(seen.terms(x));
        most = fmaxf(most, m);
      }
    }
    // the single logits before the vectors are the first unit's, those after them the last one's
    const int first = u == 0 && lane < r.head ? lane : -1;
    const int last = u == r.last_unit() && lane < r.tail ? r.head + r.vectors * kVec + lane : -1;
    if (first >= 0 || last >= 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = i == 0 ? first : last;
        if (at < 0) continue;
        const float x = single(r.base[at]);
        seen.reach(x);
        seen.add(seen.term(x));
        most = fmaxf(most, x);
      }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, order_of(most));
    if (lane == 0) tops[u] = top > 0 ? value_of(top) : -INFINITY;
  }
  // sum of the CTA, against its largest logit as a whole number (no thread's reference is above it): one that does not
  // depend on which thread read what (rows alike that start elsewhere in 16 bytes then differ by roundings at most, and
  // mostly not at all)
  const uint32_t top = __reduce_max_sync(0xffffffffu, order_of(seen.top));
  const float wr = top > 0 ? rintf(value_of(top)) : -INFINITY;
  float ws = seen.sum + seen.low;
  if (seen.ref != wr) ws *= factor(seen.ref - wr);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
  if (lane == 0) warp_stats[warp] = make_float2(wr, ws);
  __syncthreads();
  if (warp != 0) return;
  const float2 mine = lane < kWarps ? warp_stats[lane] : make_float2(-INFINITY, 0.f);
  float cr = mine.x;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) cr = fmaxf(cr, __shfl_xor_sync(0xffffffffu, cr, o));
  float cs = mine.x == cr ? mine.y : mine.y * factor(mine.x - cr);
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) cs += __shfl_xor_sync(0xffffffffu, cs, o);
  if (lane == 0) p.stats[static_cast<int64_t>(row) * p.pieces + piece] = make_float2(cr, cs);
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
// ln x, of a normal x >= 2^-1 below 2^33: x = 2^e f with f in [3/4, 3/2), so that logf is off by half a step
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

// The largest of the threads' candidates, to every thread. `scratch` may be used again after the next barrier.
template <int kPickWarps>
__device__ __forceinline__ Candidate best_of_all(Candidate c, Candidate* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Candidate other;
    other.score = __shfl_xor_sync(0xffffffffu, c.score, o);
    other.place = __shfl_xor_sync(0xffffffffu, c.place, o);
    if (better(other, c)) c = other;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = c;
  __syncthreads();
  c = scratch[0];
  for (int w = 1; w < kPickWarps; ++w)
    if (better(scratch[w], c)) c = scratch[w];
  return c;
}

// A score's order that at least k of the threads' `best` reach (0: fewer than k have one): the q-th best thread of
// each of the first `warps` warps (q of them make k), and of those the least. (Threads of equal ones all count.)
__device__ __forceinline__ uint64_t bound_of(uint64_t best, int k, int warps, uint64_t* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t bound = 0;
  if (warp < warps) {
    uint64_t left = best;
    for (int q = (k + warps - 1) / warps; q > 0; --q) {
      bound = warp_max64(left);
      // one thread of those that have it
      const uint32_t same = __ballot_sync(0xffffffffu, left == bound);
      if (lane == __ffs(same) - 1) left = 0;
    }
  }
  __syncthreads();
  if (lane == 0) scratch[warp] = bound;
  __syncthreads();
  return warp_min64(lane < warps ? scratch[lane] : ~0ull);
}

// f(entry, its place among all by `better`) for the entries that are this thread's to write: kRankLanes threads
// count for one.
constexpr int kRankLanes = 8;
template <int kPickThreads, class F>
__device__ __forceinline__ void rank_all(const Candidate* list, int n, F f) {
  const int part = threadIdx.x % kRankLanes;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kPickThreads / kRankLanes) {
    const int i = i0 + threadIdx.x / kRankLanes;
    const Candidate c = list[min(i, n - 1)];
    int place = 0;
#pragma unroll 4
    for (int j = part; j < n; j += kRankLanes) place += better(list[j], c) ? 1 : 0;
#pragma unroll
    for (int o = 1; o < kRankLanes; o <<= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
    if (i < n && part == 0) f(c, place);
  }
}

// A chosen unit.
struct Chosen {
  const void* row;  // its row's logits
  Pair shift;
  int32_t beam, unit;  // unit: -1 for a beam that has ended
  int32_t head, vectors, tail;
};

template <class T, int kPickThreads>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const BeamParams p) {
  constexpr int kVec = Row<T>::kVec, kPickWarps = kPickThreads / 32;
  constexpr int kHeld = 2048 / kPickThreads;
  __shared__ Pair shift[kMaxBeams];    // score minus normaliser of a beam
  __shared__ uint8_t kind[kMaxBeams];  // 0: no candidates, 1: its tokens, 2: itself (finished)
  __shared__ Candidate warp_best[kPickWarps];
  __shared__ uint64_t warp_bound[kPickWarps], cut;
  __shared__ Candidate list[kUnits > kFound ? kUnits : kFound];
  __shared__ Chosen of[kMaxK];
  __shared__ int units_found, found, longest;  // longest: most vectors of a chosen unit
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = static_cast<int>(blockIdx.x), units = p.beams * p.units;
  await_previous();
  if (tid == 0) {
    units_found = found = longest = 0;
    cut = 1;
  }
  // units go round the warps, so that every warp has some of each beam; a thread's first ones are asked for now
  const float* tops = p.tops + static_cast<int64_t>(n) * units;
  const int mine0 = lane * kPickWarps + warp;
  float held[kHeld];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) held[j] = mine0 + j * kPickThreads < units ? tops[mine0 + j * kPickThreads] : 0.f;
  for (int b = warp; b < p.beams; b += kPickWarps) {
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
    Pair sum{mine.x == m ? mine.y : mine.y * factor(mine.x - m), 0.f};
    for (int i = 32 + lane; i < p.pieces; i += 32) {
      const float2 v = stats[i];
      sum = add(sum, v.x == m ? v.y : v.y * factor(v.x - m));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float hi = __shfl_xor_sync(0xffffffffu, sum.hi, o), lo = __shfl_xor_sync(0xffffffffu, sum.lo, o);
      // (lanes add the same two pairs in the same order)
      sum = lane & o ? add(Pair{hi, lo + sum.lo}, sum.hi) : add(Pair{sum.hi, sum.lo + lo}, hi);
    }
    if (lane == 0) {
      // (a NaN or +inf among the logits, or nothing but -inf: no candidates)
      // (m is within 0.5 of the largest logit: its term is e^-0.5 at least, and none is above e^0.5)
      const bool good = m > -INFINITY && m < INFINITY && sum.hi >= 0.5f && sum.hi < 0x1p33f;
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
  // a unit's best score, by its largest logit
  auto beam_of = [&](int i) {
    const int q = static_cast<int>(__umulhi(static_cast<uint32_t>(i), p.over_units));  // off by one at most
    return i - q * p.units >= p.units ? q + 1 : q;
  };
  auto unit_score = [&](int i, float top) {
    const int b = beam_of(i), what = kind[b];
    const bool own = what == 2 && i == b * p.units;
    const uint64_t score = order_of(own ? shift[b] : add(shift[b], top));
    return what == 1 || own ? score : uint64_t(0);
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
  // The k best units, by their largest logit's score, equal ones in their order: the k best candidates are all in
  // them, since each of them has one at least that is better than any of the other units, equal ones being earlier.
  uint64_t key[kHeld], best = 0;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    key[j] = mine0 + j * kPickThreads < units ? unit_score(mine0 + j * kPickThreads, held[j]) : uint64_t(0);
    best = max(best, key[j]);
  }
#pragma unroll 1
  for (int i = mine0 + kHeld * kPickThreads; i < units; i += kPickThreads) best = max(best, unit_score(i, tops[i]));
  const uint64_t bound = max(bound_of(best, p.k, min(kPickWarps, units), warp_bound), static_cast<uint64_t>(1));
  if (best >= bound) {
    auto keep = [&](int i, uint64_t score) {
      if (score < bound) return;
      const int to = atomicAdd(&units_found, 1);
      if (to < kUnits) list[to] = Candidate{score, ~static_cast<uint32_t>(i)};
    };
#pragma unroll
    for (int j = 0; j < kHeld; ++j) keep(mine0 + j * kPickThreads, key[j]);
#pragma unroll 1
    for (int i = mine0 + kHeld * kPickThreads; i < units; i += kPickThreads) keep(i, unit_score(i, tops[i]));
  }
  __syncthreads();
  const int m = units_found, chosen = min(m, p.k);
  auto choose = [&](const Candidate& c, int place) {
    if (place >= p.k) return;
    const int i = static_cast<int>(~c.place), b = beam_of(i);
    const T* row = static_cast<const T*>(p.logits) + (static_cast<int64_t>(n) * p.beams + b) * p.row_stride;
    const Row<T> r(row, p.vocab);
    const int u = i - b * p.units;
    of[place] = Chosen{row, shift[b], b, kind[b] == 2 ? -1 : u, r.head, r.vectors, r.tail};
    if (place == p.k - 1) cut = c.score;
    atomicMax(&longest, max(1, min(kUnit, r.vectors - u * kUnit)));
  };
  if (m <= kUnits) {
    rank_all<kPickThreads>(list, m, choose);
  } else {  // most units alike: one after the other
    Candidate last{~0ull, ~0u};
#pragma unroll 1
    for (int k = 0; k < p.k; ++k) {
      Candidate c{0, 0};
#pragma unroll 1
      for (int i = mine0; i < units; i += kPickThreads) {
        const Candidate x{unit_score(i, tops[i]), ~static_cast<uint32_t>(i)};
        if (better(last, x) && better(x, c)) c = x;
      }
      last = best_of_all<kPickWarps>(c, warp_best);
      if (tid == 0) choose(last, k);
    }
  }
  __syncthreads();
  // This thread's vectors of the chosen units: the units take turns, so that every warp has some of each, however
  // short they are and however far apart the beams' scores. (The first 8 places have the single logits too.)
  const int places = chosen * max(longest, 8);
  const uint32_t over_chosen = 0xffffffffu / static_cast<uint32_t>(max(chosen, 1));
  auto unit_of = [&](int i, int& at) -> const Chosen& {
    at = static_cast<int>(__umulhi(static_cast<uint32_t>(i), over_chosen));  // off by one at most
    int which = i - at * chosen;
    if (which >= chosen) {
      ++at;
      which -= chosen;
    }
    return of[which];
  };
  auto vector_of = [&](const Chosen& c, int v) {
    return reinterpret_cast<const uint4*>(static_cast<const T*>(c.row) + c.head)[v];
  };
  // f(a candidate) for those that reach `least`
  auto each_candidate = [&](uint64_t least, auto f) {
    // x + shift >= least: no x below the difference less its rounding
    const float reach = value_of(static_cast<uint32_t>(least >> 32));
#pragma unroll 1
    for (int i = tid; i < places; i += kPickThreads) {
      int at;
      const Chosen& c = unit_of(i, at);
      const int u = c.unit, v = u * kUnit + at;
      const uint32_t place = static_cast<uint32_t>(c.beam) * p.vocab;
      const Pair base = c.shift;
      if (u < 0) {
        if (at == 0) f(Candidate{order_of(base), ~(place + static_cast<uint32_t>(max(p.eos, 0)))});
        continue;
      }
      const T* row = static_cast<const T*>(c.row);
      float floor = (reach - base.hi) - (fabsf(reach) + fabsf(base.hi)) * 0x1p-21f;
      if (!(floor < CUDART_INF_F)) floor = -CUDART_INF_F;
      auto one = [&](float x, int token) {
        if (x < floor) return;
        const uint64_t score = order_of(add(base, x));
        if (score >= least) f(Candidate{score, ~(place + token)});
      };
      if (v < c.vectors) {
        const uint4 w = vector_of(c, v);
        if (!(most_of(w, T()) < floor)) {
          float x[kVec];
          unpack(w, x);
#pragma unroll
          for (int j = 0; j < kVec; ++j) one(x[j], c.head + v * kVec + j);
        }
      }
      if (u == 0 && at < c.head) one(single(row[at]), at);
      if (at < c.tail && u == max(0, (c.vectors - 1) / kUnit)) {
        const int token = c.head + c.vectors * kVec + at;
        one(single(row[token]), token);
      }
    }
  };
  // Candidates that reach the worst of k units' best are ranked. If there are fewer units, or many such candidates (a
  // beam far ahead of the others that has fewer than k units, last units of a few logits), only those that reach what
  // k threads' best vectors do. (That bound at once, always: 1.0 to 1.8 us more.)
  uint64_t least = cut;
#pragma unroll 1
  for (int pass = chosen < p.k ? 1 : 0; pass < 2; ++pass) {
    if (pass == 1) {
      best = 0;
#pragma unroll 1
      for (int i = tid; i < places; i += kPickThreads) {
        int at;
        const Chosen& c = unit_of(i, at);
        const int v = c.unit * kUnit + at;
        if (c.unit < 0 ? at == 0 : v < c.vectors)
          best = max(best, order_of(c.unit < 0 ? c.shift : add(c.shift, most_of(vector_of(c, v), T()))));
      }
      least = max(least, bound_of(best, p.k, max(1, min(kPickWarps, chosen * longest / 32)), warp_bound));
      if (tid == 0) found = 0;
      __syncthreads();
    }
    each_candidate(least, [&](const Candidate& c) {
      const int to = atomicAdd(&found, 1);
      if (to < kFound) list[to] = c;
    });
    __syncthreads();
    const int all = found;
    if (all > (pass == 0 ? kFewFound : kFound)) continue;
    rank_all<kPickThreads>(list, all, [&](const Candidate& c, int place) {
      if (place < p.k) write(place, c);
    });
    if (tid >= all && tid < p.k) write(tid, Candidate{0, 0});
    return;
  }
  // More than the list holds (most of the units' logits alike, or all high): one after the other.
  Candidate last{~0ull, ~0u};
#pragma unroll 1
  for (int k = 0; k < p.k; ++k) {
    Candidate c{0, 0};
    each_candidate(least, [&](const Candidate& x) {
      if (better(last, x) && better(x, c)) c = x;
    });
    last = best_of_all<kPickWarps>(c, warp_best);
    if (tid == 0) write(k, last);
  }
}

int units_of(int32_t vocab, int32_t logits_type) {
  const int vectors = vocab / (logits_type == PA_BF16 ? 8 : 4);  // of an aligned row: others have as many, or one less
  return std::max(1, (vectors + kUnit - 1) / kUnit);
}

int pieces_of(int32_t requests, int32_t beams, int units) {
  const int64_t rows = std::max<int64_t>(1, static_cast<int64_t>(requests) * beams);
  return static_cast<int>(std::min<int64_t>((units + kWarps - 1) / kWarps, std::max<int64_t>(1, kTargetCtas / rows)));
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
  const size_t rows = static_cast<size_t>(requests) * beams;
  const int units = units_of(vocab, PA_FP32);  // (the more)
  return (rows * (pieces_of(requests, beams, units) * sizeof(float2) + units * sizeof(float)) + 255) / 256 * 256;
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
  const int units = units_of(vocab, logits_type), pieces = pieces_of(requests, beams, units);
  float2* stats = static_cast<float2*>(workspace);
  const BeamParams p{logits, row_stride, requests, beams, vocab, k, eos_token, units, pieces,
                     0xffffffffu / static_cast<uint32_t>(units), scores, live, out_scores,
                     parents, tokens, live_out, stats,
                     reinterpret_cast<float*>(stats + static_cast<size_t>(requests) * beams * pieces)};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(pieces), static_cast<unsigned>(requests * beams));
  const bool few = k * kUnit <= kPickFew;
  auto launch = [&](auto* rows_kernel, auto* pick_kernel) {
    const cudaError_t e = launch_dependent(rows_kernel, grid, kThreads, 0, st, 0, p);
    return e == cudaSuccess ? launch_dependent(pick_kernel, static_cast<unsigned>(requests), few ? kPickFew : kPickMany, 0, st, 0, p) : e;
  };
  const cudaError_t e =
      logits_type == PA_BF16
          ? launch(beam_rows_kernel<uint16_t>, few ? beam_pick_kernel<uint16_t, kPickFew> : beam_pick_kernel<uint16_t, kPickMany>)
          : launch(beam_rows_kernel<float>, few ? beam_pick_kernel<float, kPickFew> : beam_pick_kernel<float, kPickMany>);
  return e == cudaSuccess ? PA_OK : record_cuda_error(e, "beam_select");
}
