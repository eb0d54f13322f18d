// attn_prefill_chunk_score on the tensor cores (tcgen05 + TMEM + TMA), sm_103a: causal chunks over the
// paged cache with capped scores, a distance bias, and window, prefix and document masks.
//
// Definition: score_common.cuh. Work as in the plain prefill: a job is 128 queries of one chunk x both
// query heads of one KV head, two 128-row M tiles that share every K/V tile of 128 keys; S = Q K^T and
// O += P V are tcgen05.mma with accumulators in TMEM (S_0, S_1, O_0, O_1 of 128 columns each), P is
// written over S as bf16. What differs:
//
//  * Key tiles. A job's rows see the prefix and a span that ends at their positions; a plan kernel
//    reduces the rows' masks to a list of key tiles per query tile (tiles of the prefix, then of the
//    span; what lies between is never touched) and splits the listed work over the CTAs. A tile that a
//    row sees whole takes no masking; on the others a row's visible keys are two 32-bit mask words.
//  * Scores. 8 softmax warps, one thread per row, as there: a row's 128 raw products come from TMEM with
//    their maximum, and the weights go back as bf16 in one pass. The cap's tanh and the bias are taken in
//    that same pass wherever a bound of the scores' maximum follows from the products' maximum (see
//    score_bound), as a polynomial and a stepped distance on the FMA pipe, whose work then hides behind
//    the MUFU unit's exponentials. Measured (4,096 queries at 61,440): masks alone 1,270-1,330 us (1,600-
//    1,680 TFLOP/s), as the plain kernel; cap 1,920 us (an exponential and a quotient per score took 3,146,
//    a pass of its own for the polynomial 2,309, two polynomials by range 2,480: the code of the pass then
//    no longer stays in the instruction cache); bias 1,740 us; both 2,560 us. What bounds it is a row's
//    chain S -> weights -> P V: each paired FMA more per two scores costs 85 us. 16 softmax warps, two
//    threads per row meeting at a barrier per tile, were slower (1,611 us with masks alone, 2,540 with a
//    cap): at 96 to 104 registers a thread the pass spills.
//  * Rounding. The weights are rounded to bf16 for P V: the tensor cores take P and V in one type, and V
//    is bf16. Each is off by at most 2^-8 of itself, with either sign; their sum l takes them unrounded.
//    Outputs are off by 0.0023 of their norm against 64 bits where the last rounding alone is off by
//    0.0017. P in two bf16 parts would take P V, half of the tensor work, twice. The plain kernel does the
//    same; the decode keeps its weights in fp32.
//  * Non-finite K and V rows are kept from the rows that do not see them: the slots behind a sequence's
//    end are cleared by the producers, and rows that a non-finite value reached are repaired (repair_rows).
#include <algorithm>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "dependent_launch.cuh"
#include "pa_common.cuh"
#include "score_common.cuh"
#include "tc_common.cuh"

namespace pa {

bool make_map_3d(CUtensorMap* map, const void* base, uint64_t outer, uint64_t heads,
                 uint32_t box_rows);

namespace {

constexpr int kTileM = 128;   // queries per job (per head)
constexpr int kTileN = 128;   // keys per K/V tile
constexpr int kThreads = 384;  // 8 softmax warps (M tile w / 4, rows 32 * (w % 4)) and four of control
constexpr int kVWarp = 8;      // V tiles
constexpr int kMmaWarp = 9;
constexpr int kKWarp = 10;     // Q and K tiles
constexpr int kSchedWarp = 11;  // walks the work split and publishes the pieces
constexpr int kPieceRing = 4;
constexpr int kPieceReaders = 11;  // every warp but the publisher
// Register split: the two softmax warpgroups grow to 208 registers a thread, the control warpgroup
// shrinks to 88: 256 * 208 + 128 * 88 = 64,512 = 384 * 168, the budget the CTA is launched with
// (checked on the host before every launch).
constexpr int kSoftmaxRegs = 208;
constexpr int kControlRegs = 88;
constexpr int kLaunchRegs = (256 * kSoftmaxRegs + 128 * kControlRegs) / kThreads;
constexpr int kMaxGrid = 512;
constexpr uint32_t kBlockBytes = 128 * 128;  // 128 rows x 64 bf16 (one swizzled 64-dim block)
constexpr uint32_t kTileBytes = 2 * kBlockBytes;
constexpr float kRescaleThreshold = 8.0f;
constexpr float kMaxSlack = 80.0f;  // log2 units: how far a bound taken for the max may be above it
constexpr int kMaxBatch = 128;
constexpr int kVStages = 3;   // V is needed a whole P*V later than K: one more stage in flight
// Fixed cost of a job beyond its key tiles, in tiles (its epilogue and the restart of its chain)
constexpr int kJobCost = 3;
// Up to this many keys a call whose jobs fit one to a CTA is not split. One CTA a job, without plan
// and merge, is faster while a job has few tiles (300 queries at 700: 22.2 us, split 28.0; 375 at 0:
// 14.3, split 25.2) and no longer at 2,000 keys (300 at 1,700: 34.0, split 32.2; 100 at 1,948: 32.7,
// split 39.3). The host's bound of the lengths decides, since the grid does not wait for the lengths.
constexpr int kWholeKeys = 1024;
// A partial result: o [2 heads][32 float4 columns][128 rows], then lse [2][128] fp32.
constexpr size_t kRecordO = 2 * 128 * 128 * sizeof(float);
constexpr size_t kRecordBytes = kRecordO + 2 * 128 * sizeof(float);
constexpr int kMergeRows = 128;

// One piece of the walk: key tiles [jb, je) of the list of job (b, g, qt), with the chunk's first
// packed row q0, its length n, the sequence's keys L and the chunk's offset off; J = the list's
// length. List entry i is tile i for i < n1 (the prefix's), else tile i + shift; [lo, hi) is what
// the job's rows see besides the prefix. valid = 0 ends the walk.
struct PieceDesc {
  int32_t b, g, qt, q0, n, L, off, J, jb, je, valid;
  int32_t prefix, n1, shift, lo, hi;
};

// ---------------------------------------------------------------------------------------------
// The plan: one TileDesc per query tile (all KV heads share it), the running count of units (key
// tiles plus kJobCost a job) before each, and the CTAs' shares. Jobs are ordered KV head, then query
// tile over all chunks; job g * tiles + i starts at unit g * units + ws_units[i].
// ---------------------------------------------------------------------------------------------
struct TileDesc {
  int32_t b, qt, q0, n, L, off;
  int32_t J;                 // key tiles of the job (at least 1: rows that see nothing are written too)
  int32_t prefix, n1, shift, lo, hi;
  uint32_t repair;           // bit h: query head h has rows for repair_rows
};
struct PlanHeader {
  int32_t tiles, rounds, grid;
  int32_t repair;        // a tile has rows for repair_rows
  long long units;       // units of one KV head's jobs
  long long whole_jobs;  // jobs below this one were done whole, in the round-robin phase
};

// kCapT: tanh cap, kBiasT: distance bias (the masks are there in any case). scale_log2 is the
// factor of the raw products: softmax_scale * log2 e, or softmax_scale / cap with a cap.
template <bool kCapT, bool kBiasT>
struct PrefillScoreParams {
  static constexpr bool kCap = kCapT, kBias = kBiasT;
  int32_t hkv, hq;           // KV heads and query heads of the call (hq = 2 hkv)
  const int32_t* cu_q_lens;
  const int32_t* seq_lens;
  const int32_t* block_table;
  int32_t bt_stride;
  int32_t batch;
  int64_t num_pages;
  float scale_log2;
  uint16_t* out;
  float* lse;
  int32_t* status;
  ScoreParams score;
  int32_t total_q, max_tiles, max_q_len;
  const uint16_t* q_rows;    // the operands, for repair_rows
  const uint16_t* k_rows;
  const uint16_t* v_rows;
  PlanHeader* ws_plan;
  TileDesc* ws_tiles;        // [max_tiles]
  long long* ws_units;       // [max_tiles + 1] units of the tiles before, in one head
  int32_t* ws_first_tile;    // [batch + 1]
  long long* ws_tail;        // [grid + 1] first unit of each CTA's range after the whole jobs
  uint8_t* ws_records;       // [2 * grid][kRecordBytes]
};

constexpr int kPlanThreads = 1024;
constexpr int kPlanTiles = 4096;  // tiles whose key-tile counts the plan keeps in shared memory

__device__ __forceinline__ long long block_scan_incl(long long v, long long* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  __syncthreads();  // (the sums of an earlier scan have been read)
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  long long before = 0;
  for (int w = 0; w < warp; ++w) before += warp_sums[w];
  return v + before;
}

// A chunk's first packed row, rows, keys and prefix, and its query tiles: none for an empty chunk, and
// none (flagged) for one that does not fit its sequence, its table row, the packing or the host's bound
// (which the merge's grid is sized by).
struct Chunk {
  int32_t q0, n, L, prefix, tiles;
};
template <class P>
__device__ __forceinline__ Chunk chunk_of(const P& p, int b, bool report) {
  Chunk c;
  c.q0 = p.cu_q_lens[b];
  c.n = p.cu_q_lens[b + 1] - c.q0;
  c.L = p.seq_lens[b];
  c.tiles = c.prefix = 0;
  if (c.n <= 0) return c;
  if (c.n > c.L || c.n > p.max_q_len || c.L > p.bt_stride * kPage || c.q0 < 0 || c.n > p.total_q - c.q0) {
    if (report) flag_error(p.status, PA_DEV_ERR_LENGTH);
    return c;
  }
  c.tiles = (c.n + kTileM - 1) / kTileM;
  c.prefix = min(score_prefix(p.score, b, p.status, report), c.L);
  return c;
}

// The key tiles of query tile qt of chunk c (sequence b), by a whole warp: the lanes reduce the masks
// of its 128 rows.
template <class P>
__device__ __forceinline__ TileDesc tile_desc(const P& p, const Chunk& c, int b, int qt, int lane) {
  TileDesc d;
  d.b = b;
  d.qt = qt;
  d.q0 = c.q0;
  d.n = c.n;
  d.L = c.L;
  d.off = c.L - c.n;
  d.prefix = c.prefix;
  int lo = 0x7fffffff, hi = 0;
  if (p.score.row_start == nullptr) {  // a row sees at least itself: the ends decide
    lo = score_first_key(p.score, 0, d.off + qt * kTileM);
    hi = d.off + min(d.n, (qt + 1) * kTileM);
  } else {
#pragma unroll
    for (int k = 0; k < kTileM / 32; ++k) {
      const int row = qt * kTileM + 32 * k + lane;
      if (row < d.n) {
        const int first = score_first_key(p.score, d.q0 + row, d.off + row);
        if (first <= d.off + row) {
          lo = min(lo, first);
          hi = max(hi, d.off + row + 1);
        }
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
  }
  d.lo = lo;
  d.hi = hi;
  d.n1 = (d.prefix + kTileN - 1) / kTileN;
  const int end = (hi + kTileN - 1) / kTileN;
  const int t0 = max(min(lo, hi) / kTileN, d.n1);
  d.shift = t0 - d.n1;
  d.J = max(1, d.n1 + max(0, end - t0));
  d.repair = 0;
  return d;
}

// Key tiles [jb, je) of job (g, d) as a piece.
__device__ __forceinline__ PieceDesc piece_of(const TileDesc& d, int g, int jb, int je) {
  PieceDesc c;
  c.b = d.b;
  c.g = g;
  c.qt = d.qt;
  c.q0 = d.q0;
  c.n = d.n;
  c.L = d.L;
  c.off = d.off;
  c.J = d.J;
  c.prefix = d.prefix;
  c.n1 = d.n1;
  c.shift = d.shift;
  c.lo = d.lo;
  c.hi = d.hi;
  c.jb = jb;
  c.je = je;
  c.valid = jb < je;
  return c;
}

// The job of CTA blockIdx.x when a call is not split (kWhole: at most as many jobs as CTAs), by a
// whole warp, without a plan: four chunks a lane (kMaxBatch = 128), their tiles scanned.
template <class P>
__device__ PieceDesc whole_job(const P& p, int lane) {
  const bool report = blockIdx.x == 0;
  int tiles[4], mine = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int b = 4 * lane + k;
    tiles[k] = b < p.batch ? chunk_of(p, b, report).tiles : 0;
    mine += tiles[k];
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  const int total = __shfl_sync(0xffffffffu, incl, 31);
  if (report && lane == 0 && total > p.max_tiles) flag_error(p.status, PA_DEV_ERR_LENGTH);
  PieceDesc none;
  none.valid = 0;
  if (total == 0) return none;
  const int g = static_cast<int>(blockIdx.x) / total, i = static_cast<int>(blockIdx.x) - g * total;
  if (g >= p.hkv) return none;
  // the lane whose chunks hold tile i names the chunk and the tile in it
  int left = i - (incl - mine), b = -1, qt = 0;
  const bool here = left >= 0 && left < mine;
  if (here) {
    b = 4 * lane;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (b == 4 * lane + k && left >= tiles[k]) {
        left -= tiles[k];
        ++b;
      }
    }
    qt = left;
  }
  const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  b = __shfl_sync(0xffffffffu, b, from);
  qt = __shfl_sync(0xffffffffu, qt, from);
  const TileDesc d = tile_desc(p, chunk_of(p, b, false), b, qt, lane);
  return piece_of(d, g, 0, d.J);
}

// One CTA: the chunks' query tiles, each tile's key tiles (a warp per tile; its 128 rows' masks
// reduced by the lanes), a scan of their units, and the balanced split of the work.
template <class P>
__global__ void __launch_bounds__(kPlanThreads, 1) prefill_plan_kernel(const P p, int G) {
  await_previous();
  asm volatile("griddepcontrol.launch_dependents;");  // its CTAs wait for this grid's completion
  __shared__ long long warp_sums[kPlanThreads / 32];
  __shared__ int32_t first_tile[kMaxBatch + 1];
  __shared__ Chunk chunks[kMaxBatch];
  __shared__ long long carry;
  __shared__ int32_t rounds;
  __shared__ int32_t count[kPlanTiles];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- chunks
  int nqt = 0;
  if (tid < p.batch) {
    chunks[tid] = chunk_of(p, tid, true);
    nqt = chunks[tid].tiles;
  }
  const long long tiles_incl = block_scan_incl(nqt, warp_sums);
  if (tid < p.batch) first_tile[tid] = static_cast<int32_t>(min(tiles_incl - nqt, static_cast<long long>(p.max_tiles)));
  if (tid == p.batch - 1) {
    // (chunks that overlap in the packing could need more tiles than it has rows for: the rest is
    // dropped and flagged)
    if (tiles_incl > p.max_tiles) flag_error(p.status, PA_DEV_ERR_LENGTH);
    first_tile[p.batch] = static_cast<int32_t>(min(tiles_incl, static_cast<long long>(p.max_tiles)));
  }
  __syncthreads();
  const int tiles = first_tile[p.batch];

  // ---- tiles
  for (int i = warp; i < tiles; i += kPlanThreads / 32) {
    int b = 0, hi_b = p.batch;  // the last b with first_tile[b] <= i has tiles
    while (hi_b - b > 1) {
      const int mid = (b + hi_b) >> 1;
      if (first_tile[mid] <= i) b = mid; else hi_b = mid;
    }
    const TileDesc d = tile_desc(p, chunks[b], b, i - first_tile[b], lane);
    if (lane == 0) {
      p.ws_tiles[i] = d;
      if (i < kPlanTiles) count[i] = d.J;
    }
  }
  auto key_tiles = [&](int i) { return i < kPlanTiles ? count[i] : p.ws_tiles[i].J; };
  for (int b = tid; b <= p.batch; b += kPlanThreads) p.ws_first_tile[b] = first_tile[b];
  if (tid == 0) carry = 0;
  __syncthreads();

  // ---- units before each tile
  for (int i0 = 0; i0 < tiles; i0 += kPlanThreads) {
    const int i = i0 + tid;
    const long long u = i < tiles ? key_tiles(i) + kJobCost : 0;
    const long long incl = block_scan_incl(u, warp_sums) + carry;
    if (i < tiles) p.ws_units[i] = incl - u;
    __syncthreads();
    if (tid == kPlanThreads - 1) carry = incl;
    __syncthreads();
  }
  const long long T = carry;
  if (tid == 0) {
    p.ws_units[tiles] = T;
    rounds = 0;
  }
  __syncthreads();

  // ---- the split: whole jobs round-robin while they stay within the equal share,
  //      then the remaining units in consecutive ranges that level the CTAs
  const long long total = T * p.hkv, target = (total + G - 1) / G;
  const int jobs = tiles * p.hkv;
  auto job_cost = [&](int jo) { return static_cast<long long>(key_tiles(jo % tiles) + kJobCost); };
  const int rmax = jobs / G;
  if (tid == 0) rounds = rmax;
  __syncthreads();
  if (tid < G) {
    long long acc = 0;
    int r = 0;
    for (; r < rmax; ++r) {
      acc += job_cost(tid + r * G);
      if (acc > target) break;
    }
    if (r < rmax) atomicMin(&rounds, r);
  }
  __syncthreads();
  const int n_rounds = rounds;
  long long tail = 0;
  if (tid < G) {
    long long whole = 0;
    for (int r = 0; r < n_rounds; ++r) whole += job_cost(tid + r * G);
    tail = target - whole;
  }
  const long long excl = block_scan_incl(tail, warp_sums) - tail;
  const int n_dp = n_rounds * G;
  const long long T0 = n_dp < jobs ? (n_dp / tiles) * T + p.ws_units[n_dp % tiles] : total;
  if (tid < G) p.ws_tail[tid] = min(total, T0 + excl);
  if (tid == 0) {
    p.ws_tail[G] = total;
    *p.ws_plan = PlanHeader{tiles, n_rounds, G, 0, T, n_dp};
  }
}

// The pieces one CTA owns, in order: whole jobs c, c + G, ..., then its range of units.
template <class P>
struct ScoreWalker {
  const P* p;
  long long U0, U1, T, u0;  // u0: first unit of the current job
  int tiles, rounds, round, G, job;
  PieceDesc cur;

  __device__ void set(int jo, bool whole) {
    job = jo;
    cur.valid = 0;
    if (jo >= tiles * p->hkv) return;
    const int g = jo / tiles, i = jo - g * tiles;
    const TileDesc d = p->ws_tiles[i];
    u0 = g * T + p->ws_units[i];
    cur = whole ? piece_of(d, g, 0, d.J)
                : piece_of(d, g, static_cast<int>(max(U0, u0) - u0), static_cast<int>(min(U1, u0 + d.J) - u0));
    if (!whole && u0 >= U1) cur.valid = 0;
  }

  __device__ void start_tail() {
    cur.valid = 0;
    if (U0 >= U1) return;
    const int g = static_cast<int>(U0 / T);
    const long long rem = U0 - g * T;
    int lo = 0, hi = tiles;  // last tile with units before it <= rem
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p->ws_units[mid] <= rem) lo = mid; else hi = mid;
    }
    set(g * tiles + lo, false);
    // a range that starts in the cost units after a job's last key tile holds none of its tiles
    if (!cur.valid && u0 + cur.J + kJobCost < U1) set(job + 1, false);
  }

  __device__ void start(const P& pp) {
    p = &pp;
    const PlanHeader h = *pp.ws_plan;
    tiles = h.tiles;
    rounds = h.rounds;
    G = h.grid;
    T = h.units;
    U0 = pp.ws_tail[blockIdx.x];
    U1 = pp.ws_tail[blockIdx.x + 1];
    round = 0;
    if (rounds > 0) set(static_cast<int>(blockIdx.x), true);
    else start_tail();
  }

  __device__ void next() {
    if (round < rounds) {
      if (++round < rounds) set(static_cast<int>(blockIdx.x) + round * G, true);
      else start_tail();
      return;
    }
    set(job + 1, false);
  }
};

// ---------------------------------------------------------------------------------------------
// The attention kernel.
// ---------------------------------------------------------------------------------------------
struct ScoreSmem {  // placed at a 1024-byte aligned address (swizzle atoms)
  uint8_t q[2][2][kBlockBytes];   // [M tile][64-dim block]
  uint8_t k[2][2][kBlockBytes];   // [stage][64-dim block]
  uint8_t v[kVStages][2][kBlockBytes];
  PieceDesc piece[kPieceRing];
  uint64_t q_full, q_empty;
  uint64_t k_full[2], k_empty[2];
  // pv_full[st]: P_0 of the tile in V stage st is in TMEM and that V tile has landed (four
  // softmax-0 warps arrive, the V producer arrives and its copies complete bytes on it); p1_full: P_1
  uint64_t pv_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2], p1_full, o_ready[2], o_free[2];
  uint64_t mma_done;
  uint64_t piece_full[kPieceRing], piece_empty[kPieceRing];
  uint64_t tail_full[2];          // copies of a tile that its producer clears the tail of: K, V
  uint32_t tmem_base;
};
static_assert(sizeof(ScoreSmem) <= 232448, "prefill shared memory over the 227 KB limit");

__device__ __forceinline__ bool wait_or_flag(uint64_t* bar, uint32_t parity, int32_t* status) {
  if (mbar_wait_bounded(bar, parity)) return true;
  flag_error(status, PA_DEV_ERR_TIMEOUT);
  return false;
}

// What the softmax needs of a row: the keys it sees (prefix, or [lo, qpos]) and the nearest one's
// distance (0 when it sees its own position).
struct RowMask {
  int prefix, lo, qpos, nearest;
};

// Visible keys among the 32 from `base` on, bit c = key base + c.
__device__ __forceinline__ uint32_t row_mask_word(const RowMask& m, int base) {
  auto below = [](int n) { return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u); };
  return below(m.prefix - base) | (below(m.qpos + 1 - base) & ~below(m.lo - base));
}

// Whether one of a word's two bf16 is not finite (its exponent is all ones).
__device__ __forceinline__ bool word_not_finite(uint32_t w) {
  return (((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0;
}

// x, or fp32's smallest normal number where it is below (NaN stays NaN).
__device__ __forceinline__ float above_zero(float x) { return x < 1.17549435e-38f ? 1.17549435e-38f : x; }
__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }

// Two pages' first slots: the 32 keys from `base` on. Entries of keys outside `used` are not looked up.
template <class P>
__device__ __forceinline__ void word_slots(const P& p, const int32_t* bt_row, int base, uint32_t used, int64_t (&slot)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = (used >> (16 * h) & 0xffffu) != 0 ? bt_row[base / kPage + h] : 0;
    slot[h] = static_cast<int64_t>(e < 0 || e >= p.num_pages ? 0 : e) * kPage;  // (flagged by the producers)
  }
}

// The non-finite values of V that rows of a warp see: bit r of word k, row r of the warp in dim 4 lane + k.
struct NonFinite {
  uint32_t nan[4], up[4], down[4];
  // Whether x is known to be row r's weighted mean in dim 4 lane + k, or is so now: a finite value was not
  // reached by another key's; NaN or infinities of both signs make it NaN, whatever their weights; an
  // infinity makes it that infinity, unless its own weight is 0 (a score of -inf) and it is NaN.
  __device__ __forceinline__ bool settled(int r, int k, float& x) const {
    if (!not_finite(x)) return true;
    const bool u = up[k] >> r & 1u, d = down[k] >> r & 1u;
    if ((nan[k] >> r & 1u) || (u && d)) {
      x = CUDART_NAN_F;
      return true;
    }
    return (u && x == CUDART_INF_F) || (d && x == -CUDART_INF_F);
  }
};

// A masked key's P is 0, and 0 times a non-finite V is NaN: a V row that one row of a tile sees and
// another does not (a later token, another document, the rest of a prompt's page) reaches both through
// the MMA. A job's rows that came out non-finite are put right here, 32 rows of one head by a warp:
//   1. One walk over the V rows that any of them sees notes who sees which non-finite values; where that
//      settles what a row is (NonFinite::settled), nothing more is done.
//   2. The others are computed again from their visible keys, kRows at a time: a key per lane for the
//      scores, four dims per lane for the sum. Weights and rescalings stay above 0 (fp32's smallest normal
//      number) where the score is a number, that 0 times an infinity is not taken for NaN.
// Only inputs that hold non-finite values come here, and once their job's rows are stored: no wait of
// another warp runs meanwhile. Measured with all rows of a job non-finite, per key of the job: 0.06 us for
// the walk, 1.5 us where every row is computed again (4,093 keys: 0.24 and 5.9 ms beside 58 us).
template <class P>
__device__ __forceinline__ void repair_rows(const P& p, const TileDesc& d, int g, int t, int quarter) {
  constexpr int kRows = 8;
  const int lane = threadIdx.x & 31, head = 2 * g + t;
  const int row0 = d.qt * kTileM + quarter * 32;  // the warp's first row, in the chunk
  const int32_t* bt_row = p.block_table + static_cast<int64_t>(d.b) * p.bt_stride;
  const int64_t slot_row = static_cast<int64_t>(p.hkv) * kHeadDim;
  const uint16_t* const v_lane = p.v_rows + g * kHeadDim + 4 * lane;

  // this lane's 4 dims of a row, as stored
  auto out_at = [&](int r) {
    return reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(d.q0 + row0 + r) * p.hq + head) * kHeadDim) + lane;
  };
  auto load = [&](int r, float (&x)[4]) {
    const uint2 w = *out_at(r);
    x[0] = bf16lo(w.x);
    x[1] = bf16hi(w.x);
    x[2] = bf16lo(w.y);
    x[3] = bf16hi(w.y);
  };
  auto store = [&](int r, const float (&x)[4]) {
    *out_at(r) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  };
  auto mask_of = [&](int r) {
    RowMask m;
    m.prefix = d.prefix;
    m.qpos = d.off + row0 + r;
    m.lo = score_first_key(p.score, d.q0 + row0 + r, m.qpos);
    m.nearest = m.lo <= m.qpos ? 0 : max(0, m.qpos + 1 - m.prefix);
    return m;
  };

  // the rows to look at: not finite, and not for a score that is NaN (then all of the row is)
  uint32_t bad = 0;
  for (int r = 0; r < min(32, d.n - row0); ++r) {
    float x[4];
    load(r, x);
    const bool odd = not_finite(x[0]) || not_finite(x[1]) || not_finite(x[2]) || not_finite(x[3]);
    if (!__any_sync(0xffffffffu, odd)) continue;
    if (p.lse != nullptr && isnan(p.lse[static_cast<int64_t>(d.q0 + row0 + r) * p.hq + head])) continue;
    bad |= 1u << r;
  }
  if (bad == 0) return;

  const bool mine = bad >> lane & 1u;
  RowMask rm{};
  if (mine) rm = mask_of(lane);
  NonFinite nf;
#pragma unroll
  for (int k = 0; k < 4; ++k) nf.nan[k] = nf.up[k] = nf.down[k] = 0;
  for (int w = 0; w < 4 * d.J; ++w) {
    const int base = ((w >> 2) < d.n1 ? w >> 2 : (w >> 2) + d.shift) * kTileN + 32 * (w & 3);
    const uint32_t seen = mine ? row_mask_word(rm, base) : 0u;
    const uint32_t any = __reduce_or_sync(0xffffffffu, seen);
    if (any == 0) continue;
    int64_t slot[2];
    word_slots(p, bt_row, base, any, slot);
#pragma unroll 1
    for (int c0 = 0; c0 < 32; c0 += 16) {
      uint2 vw[16];
      const int64_t first = c0 == 0 ? slot[0] : slot[1];
      bool found = false;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        vw[c] = make_uint2(0u, 0u);
        if (any >> (c0 + c) & 1u) vw[c] = *reinterpret_cast<const uint2*>(v_lane + (first + c) * slot_row);
        found = found || word_not_finite(vw[c].x) || word_not_finite(vw[c].y);
      }
      if (!__any_sync(0xffffffffu, found)) continue;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const uint32_t rows = __ballot_sync(0xffffffffu, seen >> (c0 + c) & 1u);
        const float v[4] = {bf16lo(vw[c].x), bf16hi(vw[c].x), bf16lo(vw[c].y), bf16hi(vw[c].y)};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (isnan(v[k])) nf.nan[k] |= rows;
          else if (not_finite(v[k])) (v[k] > 0.f ? nf.up[k] : nf.down[k]) |= rows;
        }
      }
    }
  }

  uint32_t again = 0;
  for (uint32_t left = bad; left != 0; left &= left - 1) {
    const int r = __ffs(left) - 1;
    float x[4];
    load(r, x);
    bool wrong = false;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (!nf.settled(r, k, x[k])) wrong = true;
    if (__any_sync(0xffffffffu, wrong)) again |= 1u << r;
    else store(r, x);
  }

  float slope2 = 0.f;
  if constexpr (P::kBias) slope2 = slope_over(p.score, head, 1.0f);
#pragma unroll 1
  while (again != 0) {
    int row[kRows];
    RowMask m[kRows];
    float top[kRows], sum[kRows], acc[kRows][4];  // running maximum, the lane's share of the sum, the lane's dims
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      row[i] = again != 0 ? __ffs(again) - 1 : row[0];  // (fewer left: the first one again)
      again &= again - 1;
      m[i] = mask_of(row[i]);
      top[i] = -CUDART_INF_F;
      sum[i] = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][k] = 0.f;
    }
    for (int w = 0; w < 4 * d.J; ++w) {
      const int base = ((w >> 2) < d.n1 ? w >> 2 : (w >> 2) + d.shift) * kTileN + 32 * (w & 3);
      uint32_t seen[kRows], any = 0;
#pragma unroll
      for (int i = 0; i < kRows; ++i) any |= seen[i] = row_mask_word(m[i], base);
      if (any == 0) continue;
      int64_t slot[2];
      word_slots(p, bt_row, base, any, slot);
      float s[kRows] = {};
      if (any >> lane & 1u) {  // scores: key base + lane
        const uint4* k_row = reinterpret_cast<const uint4*>(
            p.k_rows + ((lane < 16 ? slot[0] : slot[1]) + (lane & 15)) * slot_row + g * kHeadDim);
#pragma unroll 4
        for (int c = 0; c < kHeadDim / 8; ++c) {
          const uint4 kw = k_row[c];
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const uint4 qw = reinterpret_cast<const uint4*>(
                p.q_rows + (static_cast<int64_t>(d.q0 + row0 + row[i]) * p.hq + head) * kHeadDim)[c];
            s[i] += bf16lo(qw.x) * bf16lo(kw.x) + bf16hi(qw.x) * bf16hi(kw.x) + bf16lo(qw.y) * bf16lo(kw.y) +
                    bf16hi(qw.y) * bf16hi(kw.y) + bf16lo(qw.z) * bf16lo(kw.z) + bf16hi(qw.z) * bf16hi(kw.z) +
                    bf16lo(qw.w) * bf16lo(kw.w) + bf16hi(qw.w) * bf16hi(kw.w);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const bool sees = seen[i] >> lane & 1u;
        const float x = score_of(p.score, s[i] * p.scale_log2, slope2, abs(m[i].qpos - base - lane) - m[i].nearest);
        float mx = sees ? x : -CUDART_INF_F;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (mx > top[i]) {
          const float alpha = top[i] == -CUDART_INF_F ? 0.f : above_zero(fast_exp2(top[i] - mx));
          top[i] = mx;
          sum[i] *= alpha;
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][k] *= alpha;
        }
        s[i] = sees && !(x == -CUDART_INF_F) ? above_zero(fast_exp2(x - top[i])) : 0.f;
        sum[i] += s[i];
      }
#pragma unroll 1
      for (int c0 = 0; c0 < 32; c0 += 8) {
        uint2 vw[8];
        const int64_t first = c0 < 16 ? slot[0] : slot[1];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          vw[c] = make_uint2(0u, 0u);
          if (any >> (c0 + c) & 1u)
            vw[c] = *reinterpret_cast<const uint2*>(v_lane + (first + (c0 & 15) + c) * slot_row);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float v[4] = {bf16lo(vw[c].x), bf16hi(vw[c].x), bf16lo(vw[c].y), bf16hi(vw[c].y)};
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const float pr = __shfl_sync(0xffffffffu, s[i], c0 + c);
            if (!(seen[i] >> (c0 + c) & 1u)) continue;
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][k] = fmaf(pr, v[k], acc[i][k]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][k] = sum[i] == 0.f ? 0.f : acc[i][k] / sum[i];
      store(row[i], acc[i]);
    }
  }
}

// tc::tmem_ld32_max with the maximum of the magnitudes.
__device__ __forceinline__ void tmem_ld32_absmax(uint32_t taddr, uint32_t (&r)[32], float& mx) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.abs.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,"
      "%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(mx)
      : "r"(taddr));
}

// softcap * tanh of a pair of raw products as s P(s^2), plus `add` (log2 units).
struct CapPoly {
  float2 k2[kTanhTerms];
  __device__ __forceinline__ explicit CapPoly(const float (&a)[kTanhTerms]) {
    // Read where they are used: an index that the compiler does not know to be 0 keeps the loads from being
    // moved out of the tile loop, whose registers they would take (cap and bias 2,830 us against 2,560).
    int z;
    asm volatile("mov.u32 %0, 0;" : "=r"(z));
#pragma unroll
    for (int k = 0; k < kTanhTerms; ++k) k2[k] = make_float2(a[k + z], a[k + z]);
  }
  __device__ __forceinline__ float2 operator()(float2 s, float2 add) const {
    const float2 t = mul2(s, s);
    float2 y = k2[kTanhTerms - 1];
#pragma unroll
    for (int k = kTanhTerms - 2; k >= 0; --k) y = fma2(y, t, k2[k]);
    return fma2(y, s, add);
  }
};

// -inf for the keys that the row does not see.
__device__ __forceinline__ void mask_tile(uint32_t (&sb)[kTileN], const RowMask& rm, int k0) {
#pragma unroll
  for (int w = 0; w < kTileN / 32; ++w) {
    const uint32_t seen = row_mask_word(rm, k0 + 32 * w);
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (!(seen >> c & 1u)) sb[32 * w + c] = 0xff800000u;
  }
}

// The maximum of each 32-column piece (four independent partial maxima of two elements a step).
__device__ __forceinline__ void piece_max(const uint32_t (&sb)[kTileN], float (&cm)[4]) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t* v = sb + 32 * w;
    float pm[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) pm[k] = fmax3(__uint_as_float(v[k]), __uint_as_float(v[k + 4]), __uint_as_float(v[k + 8]));
#pragma unroll
    for (int c = 12; c < 28; c += 8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) pm[k] = fmax3(pm[k], __uint_as_float(v[c + k]), __uint_as_float(v[c + 4 + k]));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) pm[k] = fmaxf(pm[k], __uint_as_float(v[28 + k]));
    cm[w] = fmax3(pm[0], pm[1], fmaxf(pm[2], pm[3]));
  }
}

// Whether a warp's tile can be scored in the weights' own pass: the products within the tanh
// polynomial's range and no key masked (with a cap), the bias linear over the tile's visible keys,
// and a bound `top` of each row's largest score near enough to it. cm: the largest visible product of
// each 32-column piece (magnitude with a cap). cap tanh(max |s|) bounds capped scores, and their max
// is at least its negative; the distance of a piece's nearest column bounds its bias, which falls by
// 31 slopes over the piece. The exponents' reference may be above the max by up to kMaxSlack: the
// weights that matter then stay 2^46 above fp32's smallest normal number. d0: bias distance of
// column 0.
template <class P>
__device__ __forceinline__ bool score_bound(const P& p, const RowMask& rm, int k0, float slope2, const float (&cm)[4],
                                            bool hidden, bool partial, float& top, float& d0) {
  bool good = true;
  float slack = 0.f;
  if constexpr (P::kCap) {
    const float hi = fmax3(cm[0], cm[1], fmaxf(cm[2], cm[3]));
    good = !partial && hi <= p.score.poly_max;
    top = p.score.cap_log2 * tanh_exp(hi * p.scale_log2);
    slack = 2.f * top;
  }
  if constexpr (P::kBias) {
    d0 = static_cast<float>(rm.qpos - k0 - rm.nearest);
    top = -CUDART_INF_F;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float d = fmaxf(d0 - (slope2 >= 0.f ? 32.f * c + 31.f : 32.f * c), 0.f);
      const float hi = P::kCap ? p.score.cap_log2 * tanh_exp(cm[c] * p.scale_log2) : cm[c] * p.scale_log2;
      top = fmaxf(top, fmaf(-slope2, d, hi));
    }
    slack += fabsf(slope2) * 31.f;
    good = good && (k0 + kTileN - 1 <= rm.qpos || k0 >= rm.prefix);  // keys after the row: in the prefix
  }
  return __all_sync(0xffffffffu, hidden || (good && slack <= kMaxSlack));
}

// Any other tile: scores in log2 units, in place.
template <class P>
__device__ __forceinline__ void score_tile(const P& p, uint32_t (&sb)[kTileN], const RowMask& rm, int k0,
                                           float slope2, float mx) {
  const float at = static_cast<float>(rm.qpos - k0);  // the column of the row's own position
  const float near = static_cast<float>(rm.nearest);
  if constexpr (P::kCap) {
    if (__all_sync(0xffffffffu, mx <= p.score.poly_max)) {
      const CapPoly poly(p.score.poly);
#pragma unroll
      for (int c = 0; c < kTileN; c += 2) {
        const float2 y = poly(make_float2(__uint_as_float(sb[c]), __uint_as_float(sb[c + 1])), make_float2(0.f, 0.f));
        sb[c] = __float_as_uint(y.x);
        sb[c + 1] = __float_as_uint(y.y);
      }
    } else {
#pragma unroll
      for (int c = 0; c < kTileN; ++c)
        sb[c] = __float_as_uint(p.score.cap_log2 * tanh_score(__uint_as_float(sb[c]) * p.scale_log2));
    }
  }
  if constexpr (P::kBias) {
    const float scale = P::kCap ? 1.0f : p.scale_log2;
#pragma unroll
    for (int c = 0; c < kTileN; ++c)
      sb[c] = __float_as_uint(fmaf(near - fabsf(at - static_cast<float>(c)), slope2, __uint_as_float(sb[c]) * scale));
  }
}

// repair_rows of a CTA's one job. (Not inlined: kept out of the tile loop's registers.)
template <class P>
__device__ __noinline__ void repair_job(const P& p, const PieceDesc& c, int t, int quarter) {
  TileDesc d;
  d.b = c.b;
  d.qt = c.qt;
  d.q0 = c.q0;
  d.n = c.n;
  d.off = c.off;
  d.J = c.J;
  d.prefix = c.prefix;
  d.n1 = c.n1;
  d.shift = c.shift;
  __syncwarp();
  repair_rows(p, d, c.g, t, quarter);
}

// kWhole: a CTA per job; nothing is split, and neither plan nor merge is needed.
template <class P, bool kWhole>
__global__ void __launch_bounds__(kThreads, 1)
prefill_score_kernel(const __grid_constant__ CUtensorMap q_map,
                     const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const P p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((smem_addr(smem_raw) & 1023u) != 0) {
    // not the layout this kernel was built for: do nothing (the merge then has nothing to read but
    // what an earlier call left; the error flag says that the call failed)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(p.status, PA_DEV_ERR_INTERNAL);
    return;
  }
  ScoreSmem& s = *reinterpret_cast<ScoreSmem*>(smem_raw);
  if (threadIdx.x == 0) {
    mbar_init(&s.q_full, 1);
    mbar_init(&s.q_empty, 2);       // released by each M tile's softmax
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.k_full[i], 1);
      mbar_init(&s.k_empty[i], 2);
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.o_ready[i], 1);
      mbar_init(&s.o_free[i], 4);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&s.pv_full[i], 5);   // 4 softmax-0 warps + the V producer (+ its bytes)
      mbar_init(&s.v_empty[i], 2);
    }
    mbar_init(&s.p1_full, 4);
    mbar_init(&s.mma_done, 1);
    mbar_init(&s.tail_full[0], 1);
    mbar_init(&s.tail_full[1], 1);
    for (int i = 0; i < kPieceRing; ++i) {
      mbar_init(&s.piece_full[i], 1);
      mbar_init(&s.piece_empty[i], kPieceReaders);
    }
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tc::tmem_alloc<512>(&s.tmem_base);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s.tmem_base;
  // a programmatic dependent of its plan kernel, set up so far while that ran; its merge kernel
  // waits for its completion
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const bool work = kWhole || p.ws_plan->rounds > 0 || p.ws_tail[blockIdx.x] < p.ws_tail[blockIdx.x + 1];

  if (!work) {
    // nothing to do but to give the tensor memory back
  } else if (warp >= kVWarp) {
    tc::regs_decrease<kControlRegs>();
  if (warp == kSchedWarp) {
    // ------------------------------------------------------------------ scheduler
    if constexpr (kWhole) {  // this CTA's one job, then the end (the ring has room for both)
      const PieceDesc d = whole_job(p, lane);
      if (lane == 0) {
        s.piece[0] = d;
        mbar_arrive(&s.piece_full[0]);
        s.piece[1].valid = 0;
        mbar_arrive(&s.piece_full[1]);
      }
    } else if (lane == 0) {
      ScoreWalker<P> sw;
      sw.start(p);
      for (uint32_t k = 0;; ++k) {
        const uint32_t slot = k % kPieceRing, ph = (k / kPieceRing) & 1;
        if (!wait_or_flag(&s.piece_empty[slot], ph ^ 1u, p.status)) break;
        s.piece[slot] = sw.cur;
        mbar_arrive(&s.piece_full[slot]);  // release: the readers' waits make it visible
        if (!sw.cur.valid) break;
        sw.next();
      }
    }
    __syncwarp();
  } else if (warp == kVWarp || warp == kKWarp) {
    // ------------------------------------------------------------------ TMA producers
    const bool is_k = warp == kKWarp;
    const CUtensorMap* map = is_k ? &k_map : &v_map;
    uint8_t(*ring)[2][kBlockBytes] = is_k ? s.k : s.v;
    const uint32_t nst = is_k ? 2u : static_cast<uint32_t>(kVStages);
    uint64_t* full = is_k ? s.k_full : s.pv_full;
    uint64_t* empty = is_k ? s.k_empty : s.v_empty;
    const int oob_token = static_cast<int>(p.num_pages * kPage);  // zero-filled coordinate
    uint64_t* tail_full = &s.tail_full[is_k ? 0 : 1];
    bool ok = true;
    uint32_t it = 0, tails = 0;
    for (uint32_t jc = 0;; ++jc) {
      const uint32_t slot = jc % kPieceRing, ph = (jc / kPieceRing) & 1;
      ok = __all_sync(0xffffffffu, wait_or_flag(&s.piece_full[slot], ph, p.status));
      if (!ok) break;
      const PieceDesc pc = s.piece[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.piece_empty[slot]);
      if (!pc.valid) break;
      const int32_t* bt_row = p.block_table + static_cast<int64_t>(pc.b) * p.bt_stride;
      // lane l < 8: first token of the tile's l-th page; a page no row of the job sees is not looked
      // up and arrives as zeros
      auto page_token = [&](int j) {
        int tok = oob_token;
        const int key0 = (j < pc.n1 ? j : j + pc.shift) * kTileN + kPage * lane;
        const bool used = key0 < pc.prefix || (key0 + kPage > pc.lo && key0 < pc.hi);
        if (lane < kTileN / kPage && used) {
          const int e = bt_row[key0 / kPage];
          if (e < 0 || e >= p.num_pages) {
            flag_error(p.status, PA_DEV_ERR_PAGE_OOB);
            tok = 0;
          } else {
            tok = e * kPage;
          }
        }
        return tok;
      };
      if (is_k) {
        if (lane == 0) {
          ok = wait_or_flag(&s.q_empty, (jc & 1) ^ 1u, p.status);
          if (ok) {
            mbar_arrive_expect_tx(&s.q_full, 4 * kBlockBytes);
            for (int t = 0; t < 2; ++t)
              for (int kb = 0; kb < 2; ++kb)
                tc::tma_load_3d(s.q[t][kb], &q_map, kb * 64, 2 * pc.g + t, pc.q0 + pc.qt * kTileM, &s.q_full);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      int tok = page_token(pc.jb);
      int tok_next = (pc.jb + 1 < pc.je) ? page_token(pc.jb + 1) : oob_token;
      for (int j = pc.jb; j < pc.je && ok; ++j, ++it) {
        const int st = it % nst;
        const uint32_t eph = (it / nst) & 1;
        const int tok_ahead = (j + 2 < pc.je) ? page_token(j + 2) : oob_token;
        if (lane == 0) ok = wait_or_flag(&empty[st], eph ^ 1u, p.status);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        // The page that holds the sequence's last key L - 1 is loaded whole. The pool slots after it may
        // hold anything (unwritten ones a NaN): their rows are cleared before the tile is handed on, that
        // neither a product, not even of a row that sees nothing of the tile, nor P = 0 meets them. (The
        // pages after it are never loaded: zeros.) Only a piece's last tile can run past the end.
        const int zl = pc.L - (j < pc.n1 ? j : j + pc.shift) * kTileN;
        const bool tail = zl > 0 && zl < kTileN && (zl & (kPage - 1)) != 0;
        uint64_t* landed = tail ? tail_full : &full[st];
        if (lane == 0) mbar_arrive_expect_tx(landed, kTileBytes);
        __syncwarp();
        // 16 lanes issue the tile's 16 copies at once (page lane / 2, 64-dim block lane % 2)
        const int pg = (lane >> 1) & 7, kb = lane & 1;
        const int tk = __shfl_sync(0xffffffffu, tok, pg);
        if (lane < 2 * (kTileN / kPage))
          tc::tma_load_3d(ring[st][kb] + pg * 2048, map, kb * 64, pc.g, tk, landed);
        if (tail) {
          ok = __all_sync(0xffffffffu, wait_or_flag(tail_full, tails & 1, p.status));
          ++tails;
          if (!ok) break;
          for (int e = zl * 16 + lane; e < ((zl + 15) & ~15) * 16; e += 32) {
            const int r = e >> 4, c = e & 15;   // row, 16-byte chunk (8 per 64-dim block)
            *reinterpret_cast<uint4*>(ring[st][c >> 3] + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[st]);
        }
        tok = tok_next;
        tok_next = tok_ahead;
      }
      if (!ok) break;
    }
    // do not leave while copies into this CTA's shared memory may still be landing
    if (lane == 0 && it > 0) {
      for (uint32_t k = (it >= nst ? it - nst : 0); k < it; ++k)
        wait_or_flag(&full[k % nst], (k / nst) & 1, p.status);
    }
    if (lane == 0 && tails > 0) wait_or_flag(tail_full, (tails - 1) & 1, p.status);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMA issuer (lane 0)
    // The tensor pipe queues only about one instruction ahead of the issuing thread: descriptors
    // are built once and selected, a K step is a constant added to the start field, and the only
    // waits are for P of each M tile (P_0's barrier also takes the V copies' bytes) and the next K.
    constexpr uint32_t id_s = tc::idesc_bf16(128, kTileN, 0, 0);    // S = Q K^T
    constexpr uint32_t id_o = tc::idesc_bf16(128, 128, 0, 1);       // O = P V, V MN-major
    static_assert(kVStages == 3, "the V descriptor selection below assumes three stages");
    if (lane == 0) {
      const uint64_t dq0 = tc::smem_desc_sw128(smem_addr(s.q[0][0]), 16, 1024);
      const uint64_t dq1 = tc::smem_desc_sw128(smem_addr(s.q[1][0]), 16, 1024);
      const uint64_t dk0 = tc::smem_desc_sw128(smem_addr(s.k[0][0]), 16, 1024);
      const uint64_t dk1 = tc::smem_desc_sw128(smem_addr(s.k[1][0]), 16, 1024);
      const uint64_t dv0 = tc::smem_desc_sw128(smem_addr(s.v[0][0]), kBlockBytes, 1024);
      const uint64_t dv1 = tc::smem_desc_sw128(smem_addr(s.v[1][0]), kBlockBytes, 1024);
      const uint64_t dv2 = tc::smem_desc_sw128(smem_addr(s.v[2][0]), kBlockBytes, 1024);
      auto issue_s = [&](uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = ((kk >> 2) * kBlockBytes + (kk & 3) * 32) >> 4;
          if (kk == 0) tc::mma_ss_c<false>(d, a + off, b + off, id_s);
          else tc::mma_ss_c<true>(d, a + off, b + off, id_s);
        }
      };
      auto issue_pv = [&](uint32_t d, uint32_t a, uint64_t b, uint32_t acc) {
        tc::mma_ts(d, a, b, id_o, acc);
#pragma unroll
        for (int kk = 1; kk < 8; ++kk) tc::mma_ts_c<true>(d, a + kk * 8, b + kk * (2048 >> 4), id_o);
      };
      uint32_t kst = 0, kph = 0;     // K ring: stage and parity of the next tile to consume
      uint32_t vst = 0, vph = 0;     // V ring: stage and parity of the current tile
      uint32_t tph = 0;              // parity of the current tile's S / P phases
      bool ok = true;
      for (uint32_t jc = 0; ok; ++jc) {
        const uint32_t pslot = jc % kPieceRing;
        if (!wait_or_flag(&s.piece_full[pslot], (jc / kPieceRing) & 1, p.status)) break;
        const volatile PieceDesc& pv = s.piece[pslot];
        const int pvalid = pv.valid, pjb = pv.jb, pje = pv.je;
        mbar_arrive(&s.piece_empty[pslot]);
        if (!pvalid) break;
        const int nt = pje - pjb;
        const uint32_t qph = jc & 1, oph = (jc - 1) & 1;
        ok = wait_or_flag(&s.q_full, qph, p.status) && wait_or_flag(&s.k_full[kst], kph, p.status);
        if (!ok) break;
        tc::fence_after_sync();
        uint64_t dk = kst ? dk1 : dk0;
        issue_s(tmem, dq0, dk);
        tc::mma_commit(&s.s_full[0]);
        issue_s(tmem + 128, dq1, dk);
        tc::mma_commit(&s.s_full[1]);
        kph ^= kst;
        kst ^= 1u;
        for (int i = 0; i < nt; ++i) {
          const bool more = i + 1 < nt;
          const uint64_t dv = vst == 0 ? dv0 : (vst == 1 ? dv1 : dv2);
          const uint32_t acc = i > 0 ? 1u : 0u;
          if (!wait_or_flag(&s.pv_full[vst], vph, p.status) ||
              (i == 0 && jc > 0 && !wait_or_flag(&s.o_free[0], oph, p.status))) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          issue_pv(tmem + 256, tmem, dv, acc);
          if (more) {
            if (!wait_or_flag(&s.k_full[kst], kph, p.status)) { ok = false; break; }
            tc::fence_after_sync();
            dk = kst ? dk1 : dk0;
            issue_s(tmem, dq0, dk);
            tc::mma_commit(&s.s_full[0]);
          } else {
            tc::mma_commit(&s.o_ready[0]);
          }
          if (!wait_or_flag(&s.p1_full, tph, p.status) ||
              (i == 0 && jc > 0 && !wait_or_flag(&s.o_free[1], oph, p.status))) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          issue_pv(tmem + 384, tmem + 128, dv, acc);
          if (more) {
            issue_s(tmem + 128, dq1, dk);
            tc::mma_commit(&s.s_full[1]);
            kph ^= kst;
            kst ^= 1u;
          } else {
            tc::mma_commit(&s.o_ready[1]);
          }
          vst = vst == 2 ? 0u : vst + 1;
          vph ^= vst == 0 ? 1u : 0u;
          tph ^= 1u;
        }
      }
    }
    __syncwarp();
    // every MMA lane 0 issued must have finished before TMEM is released
    if (lane == 0) {
      tc::mma_commit(&s.mma_done);
      wait_or_flag(&s.mma_done, 0, p.status);
    }
    __syncwarp();
  }
  } else {
    tc::regs_increase<kSoftmaxRegs>();
    // ------------------------------------------------------------------ softmax warps
    const int t = warp >> 2;                       // M tile = query head 2g + t
    const int quarter = warp & 3;                  // TMEM lanes 32*quarter .. +31
    const int r = quarter * 32 + lane;             // row of the tile
    const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_bits + t * 128;
    const uint32_t t_o = tmem + lane_bits + 256 + t * 128;
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    const bool leader = quarter == 0 && lane == 0;  // releases stages for this M tile
    constexpr bool kLog2Units = P::kCap || P::kBias;  // scores scored ahead of the weights' pass
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t jc = 0;; ++jc) {
      // the next piece; its slot is held until the epilogue, which reads the rest of it
      const uint32_t pslot = jc % kPieceRing;
      if (!__all_sync(0xffffffffu, wait_or_flag(&s.piece_full[pslot], (jc / kPieceRing) & 1, p.status))) break;
      const volatile PieceDesc& pv = s.piece[pslot];
      if (!pv.valid) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.piece_empty[pslot]);
        break;
      }
      const int pjb = pv.jb, nt = pv.je - pjb;
      const int n1 = pv.n1, shift = pv.shift;
      const int qrow = pv.qt * kTileM + r;
      RowMask rm;
      rm.prefix = pv.prefix;
      rm.qpos = pv.off + qrow;                     // absolute position of this query
      rm.lo = qrow < pv.n ? score_first_key(p.score, pv.q0 + qrow, rm.qpos) : 0;
      rm.nearest = rm.lo <= rm.qpos ? 0 : max(0, rm.qpos + 1 - rm.prefix);
      [[maybe_unused]] float slope2 = 0.f;         // the head's slope in log2 units
      if constexpr (P::kBias) slope2 = slope_over(p.score, 2 * pv.g + t, 1.0f);
      float m_used = -CUDART_INF_F, l = 0.f;
      for (int i = 0; i < nt; ++i) {
        const uint32_t cur = it + i;
        ok = __all_sync(0xffffffffu, wait_or_flag(&s.s_full[t], cur & 1, p.status));
        if (!ok) break;
        // S_t(cur) is done, and its commit also covers P_t V(cur - 1): this M tile is finished
        // with K stage cur and V stage cur - 1 (the last V stage of a piece is released after
        // the epilogue's wait), and with Q after the piece's last tile
        if (leader) {
          mbar_arrive(&s.k_empty[cur & 1]);
          if (i > 0) mbar_arrive(&s.v_empty[(cur - 1) % kVStages]);
          if (i + 1 == nt) mbar_arrive(&s.q_empty);
        }
        tc::fence_after_sync();
        uint32_t sb[kTileN];  // raw products (fp32 bits) of this row
        float cm[4];          // the maximum of each 32-column piece (of magnitudes with a cap)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if constexpr (P::kCap) tmem_ld32_absmax(t_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(sb + c * 32), cm[c]);
          else tc::tmem_ld32_max(t_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(sb + c * 32), cm[c]);
        }
        tc::tmem_wait_ld();
        const int j = pjb + i;
        const int k0 = (j < n1 ? j : j + shift) * kTileN;
        // A row that sees no key of the tile (one that sees nothing at all makes every tile such a
        // one for its warp) is not masked key by key: its exponents' offset is -inf.
        const bool hidden = k0 >= rm.prefix && (k0 + kTileN <= rm.lo || k0 > rm.qpos || rm.lo > rm.qpos);
        const bool partial = !hidden && k0 + kTileN > rm.prefix && (k0 < rm.lo || k0 + kTileN - 1 > rm.qpos);
        bool one_pass = true;             // (scores without options always are)
        [[maybe_unused]] float d0 = 0.f;  // bias distance of column 0, from the nearest visible key
        float top = 0.f;                  // the scores' maximum, or a bound of it (log2 units)
        // without a cap the raw products are masked: a bias leaves -inf what it is
        if (!P::kCap && partial) {
          mask_tile(sb, rm, k0);
          piece_max(sb, cm);
        }
        if constexpr (kLog2Units) {
          one_pass = score_bound<P>(p, rm, k0, slope2, cm, hidden, partial, top, d0);
          if (!one_pass) {
            score_tile<P>(p, sb, rm, k0, slope2, fmax3(cm[0], cm[1], fmaxf(cm[2], cm[3])));
            if (P::kCap && partial) mask_tile(sb, rm, k0);
            piece_max(sb, cm);
            top = fmax3(cm[0], cm[1], fmaxf(cm[2], cm[3]));
          }
        } else {
          top = fmax3(cm[0], cm[1], fmaxf(cm[2], cm[3])) * p.scale_log2;
        }
        if (hidden) top = -CUDART_INF_F;
        const bool grow = top > m_used + kRescaleThreshold;
        if (__any_sync(0xffffffffu, grow)) {
          const float m_new = grow ? top : m_used;
          const float alpha = (m_used == -CUDART_INF_F) ? 0.f : fast_exp2(m_used - m_new);
          if (i > 0) {
            // O_t holds the sum through the previous tile: P_t V(cur - 1) completed before
            // S_t(cur), whose completion this thread has already observed
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t o32[32];
              tc::tmem_ld32(t_o + c * 32, o32);
              tc::tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o32[k] = __float_as_uint(__uint_as_float(o32[k]) * alpha);
              tc::tmem_st32(t_o + c * 32, o32);
            }
            tc::tmem_wait_st();
          }
          l *= alpha;
          m_used = m_new;
        }
        // weights (bf16) over S's first 64 columns. A row that has not met a visible key yet keeps
        // m_used = -inf; a finite offset then gives exp2(-inf) = 0 for its masked scores, not NaN.
        const float m_eff = hidden ? CUDART_INF_F : (m_used == -CUDART_INF_F) ? 0.f : m_used;
        const float2 nm2 = make_float2(-m_eff, -m_eff);
        float2 ls[4];  // 4 independent paired partial sums
#pragma unroll
        for (int k = 0; k < 4; ++k) ls[k] = make_float2(0.f, 0.f);
        auto weights = [&](auto exponent) {  // exponent(pair of sb, index of the pair)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float2 x = exponent(make_float2(__uint_as_float(sb[c * 64 + 2 * k]),
                                                    __uint_as_float(sb[c * 64 + 2 * k + 1])), c * 32 + k);
              const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
              ls[k & 3] = add2(ls[k & 3], e);
              pk[k] = pack_bf16x2(e.x, e.y);
            }
            tc::tmem_st32(t_s + c * 32, pk);
          }
        };
        if constexpr (kLog2Units) {
          if (one_pass) {
            // the bias of pairs k, k + 4, ...: distances are small integers, stepped exactly
            [[maybe_unused]] float2 dist[4];
            const float2 ns2 = make_float2(-slope2, -slope2), step = make_float2(-8.f, -8.f);
#pragma unroll
            for (int k = 0; k < 4; ++k) dist[k] = make_float2(d0 - 2.f * k, d0 - 2.f * k - 1.f);
            auto offset = [&](int n) {  // - (slope distance) - m
              if constexpr (!P::kBias) return nm2;
              const float2 b = fma2(dist[n & 3], ns2, nm2);
              dist[n & 3] = add2(dist[n & 3], step);
              return b;
            };
            if constexpr (P::kCap) {
              const CapPoly poly(p.score.poly);
              weights([&](float2 x, int n) { return poly(x, offset(n)); });
            } else {
              weights([&](float2 x, int n) { return fma2(x, sc2, offset(n)); });
            }
          } else {
            weights([&](float2 x, int) { return add2(x, nm2); });
          }
        } else {
          weights([&](float2 x, int) { return fma2(x, sc2, nm2); });
        }
        const float2 lsum = add2(add2(ls[0], ls[1]), add2(ls[2], ls[3]));
        if (!hidden) l += lsum.x + lsum.y;  // (not even 0: a key the row does not see may be NaN)
        tc::tmem_wait_st();
        tc::fence_before_sync();
        // one elected arrive per warp: 128 arrivals on one barrier word serialise for hundreds
        // of cycles on the path to the next P*V
        __syncwarp();
        if (lane == 0) mbar_arrive(t == 0 ? &s.pv_full[cur % kVStages] : &s.p1_full);
      }
      if (!ok) break;
      // epilogue of the piece: O / l
      ok = __all_sync(0xffffffffu, wait_or_flag(&s.o_ready[t], jc & 1, p.status));
      if (!ok) break;
      tc::fence_after_sync();
      if (leader) mbar_arrive(&s.v_empty[(it + nt - 1) % kVStages]);
      const PieceDesc desc = s.piece[pslot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.piece_empty[pslot]);
      const bool live = qrow < desc.n;
      // a row may see nothing, or nothing that carries weight: l = 0, o = 0, lse = -inf
      const bool none = l == 0.f;
      const float inv = none ? 0.f : 1.0f / l;
      const bool whole = pjb == 0 && pjb + nt == desc.J;
      const int head = 2 * desc.g + t;
      // all of O's 128 columns at once; they are then released to the next piece's first P*V
      uint32_t o[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_ld32(t_o + c * 32, o[c]);
      tc::tmem_wait_ld();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.o_free[t]);
      float z = 0.f;  // NaN if any of the row's values is not finite
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int k = 0; k < 32; ++k) z = fmaf(__uint_as_float(o[c][k]), 0.f, z);
      }
      uint8_t* rec = p.ws_records + (2 * static_cast<size_t>(blockIdx.x) + (pjb == 0 ? 1 : 0)) * kRecordBytes;
      if (whole) {
        uint16_t* out_row = p.out + (static_cast<int64_t>(desc.q0 + qrow) * p.hq + head) * kHeadDim;
        if (live) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint32_t* v = &o[k >> 2][8 * (k & 3)];
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(v[0]) * inv, __uint_as_float(v[1]) * inv);
            w.y = pack_bf16x2(__uint_as_float(v[2]) * inv, __uint_as_float(v[3]) * inv);
            w.z = pack_bf16x2(__uint_as_float(v[4]) * inv, __uint_as_float(v[5]) * inv);
            w.w = pack_bf16x2(__uint_as_float(v[6]) * inv, __uint_as_float(v[7]) * inv);
            *reinterpret_cast<uint4*>(out_row + 8 * k) = w;
          }
          if (none && z != 0.f) {  // (0 times what no weight was on)
#pragma unroll 1
            for (int k = 0; k < 16; ++k) *reinterpret_cast<uint4*>(out_row + 8 * k) = make_uint4(0u, 0u, 0u, 0u);
          }
          if (p.lse != nullptr) {
            float v = none ? -CUDART_INF_F : (m_used + log2f(l)) * kLn2;
            if constexpr (P::kBias) {
              if (!none && rm.nearest > 0) v -= p.score.slopes[head] * static_cast<float>(rm.nearest);
            }
            p.lse[static_cast<int64_t>(desc.q0 + qrow) * p.hq + head] = v;
          }
        }
      } else {
        // a piece of a job shared with neighbouring CTAs: slot 1 if it starts the job, else 0
        float4* dst = reinterpret_cast<float4*>(rec) + t * 32 * 128 + r;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const uint32_t* v = &o[k >> 3][4 * (k & 7)];
          dst[k * 128] = make_float4(__uint_as_float(v[0]) * inv, __uint_as_float(v[1]) * inv,
                                     __uint_as_float(v[2]) * inv, __uint_as_float(v[3]) * inv);
        }
        reinterpret_cast<float*>(rec + kRecordO)[t * 128 + r] = none ? -CUDART_INF_F : (m_used + log2f(l)) * kLn2;
      }
      // (a sum that is NaN: the row sees a score that is, and all of it is NaN)
      if (__any_sync(0xffffffffu, live && z != 0.f && l > 0.f)) {
        if constexpr (kWhole) {
          repair_job(p, desc, t, quarter);
        } else if (lane == 0) {  // for prefill_repair_kernel
          atomicOr(&p.ws_tiles[p.ws_first_tile[desc.b] + desc.qt].repair, 1u << head);
          p.ws_plan->repair = 1;
        }
      }
      it += nt;
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc<512>(tmem);
  }
}

// Combine the pieces of jobs that were cut by CTA range boundaries. Eight CTAs per job (two
// heads x four 32-dim quarters), one thread per row. The pieces are slot 1 of the first CTA and
// slot 0 of each later CTA.
template <class P>
__global__ void __launch_bounds__(kMergeRows) prefill_score_merge_kernel(const P p) {
  // A programmatic dependent of prefill_score_kernel, whose CTAs let it launch once they have seen
  // the plan: the plan is read before the wait for that grid's results, further down.
  // CTA (qt, g * 8 + t * 4 + quarter, b), counted from the end of the grid: rows of query tile
  // qt, head 2g + t, dims 32 * quarter .. +31; one thread per row. A job cut into pieces is
  // merged by 8 CTAs, so the few split jobs of a call are spread over many SMs instead of one CTA
  // each. The split jobs are the last ones (the whole-job rounds take the first), so the grid is
  // walked backwards: their CTAs start first and the rest only check and exit.
  const int b = gridDim.z - 1 - blockIdx.z;
  const int y = gridDim.y - 1 - blockIdx.y;
  const int g = y >> 3, t = (y >> 2) & 1, quarter = y & 3;
  const int qt = gridDim.x - 1 - blockIdx.x;
  const PlanHeader h = *p.ws_plan;
  const int tile = p.ws_first_tile[b] + qt;
  if (tile >= p.ws_first_tile[b + 1] || g * h.tiles + tile < h.whole_jobs) {
    // no such tile, or a job done whole. (Every CTA waits, that this grid does not end before the
    // one whose results the stream's next work may read.)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const TileDesc d = p.ws_tiles[tile];
  const int G = min(h.grid, kMaxGrid);
  const long long u0 = g * h.units + p.ws_units[tile], J = d.J;
  const int q0 = d.q0, n = d.n;
  // the split's range starts, staged in shared memory: one round of loads instead of a chain of
  // dependent ones per binary search
  __shared__ long long tail[kMaxGrid + 1];
  for (int i = threadIdx.x; i <= G; i += kMergeRows) tail[i] = p.ws_tail[i];
  __syncthreads();
  // the CTA whose range [tail[c], tail[c + 1]) holds unit u (the last c with a start <= u: a CTA
  // with an empty range shares its start with the next one)
  auto cta_of = [&](long long u) {
    int lo = 0, hi = G;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tail[mid] <= u) lo = mid; else hi = mid;
    }
    return lo;
  };
  const int c0 = cta_of(u0), c1 = cta_of(u0 + J - 1);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c0 == c1) return;
  const int r = threadIdx.x;
  const int qrow = qt * kTileM + r;
  if (qrow >= n) return;
  // the piece in CTA c0 starts the job (slot 1); later CTAs hold continuations (slot 0); CTAs with
  // an empty range in between hold nothing
  auto rec_of = [&](int c) {
    return p.ws_records + (2 * static_cast<size_t>(c) + (c == c0 ? 1 : 0)) * kRecordBytes;
  };
  auto empty_range = [&](int c) { return tail[c] == tail[c + 1]; };
  float m = -CUDART_INF_F;
  for (int c = c0; c <= c1; ++c)
    if (!empty_range(c)) m = fmaxf(m, reinterpret_cast<const float*>(rec_of(c) + kRecordO)[t * 128 + r]);
  float acc[32];
#pragma unroll
  for (int d = 0; d < 32; ++d) acc[d] = 0.f;
  float sum = 0.f;
#pragma unroll 2
  for (int c = c0; c <= c1; ++c) {
    if (empty_range(c)) continue;
    const uint8_t* rec = rec_of(c);
    const float lp = reinterpret_cast<const float*>(rec + kRecordO)[t * 128 + r];
    if (lp == -CUDART_INF_F) continue;  // the piece held no key visible to this row
    const float w = fast_exp2((lp - m) * kLog2e);
    sum += w;
    const float4* o = reinterpret_cast<const float4*>(rec) + (t * 32 + quarter * 8) * 128 + r;
    float4 v[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) v[d] = o[d * 128];
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      acc[4 * d] += w * v[d].x;
      acc[4 * d + 1] += w * v[d].y;
      acc[4 * d + 2] += w * v[d].z;
      acc[4 * d + 3] += w * v[d].w;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  const int head = 2 * g + t;
  uint4* dst = reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(q0 + qrow) * p.hq + head) * kHeadDim +
                                        32 * quarter);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint4 w;
    w.x = pack_bf16x2(acc[8 * k + 0] * inv, acc[8 * k + 1] * inv);
    w.y = pack_bf16x2(acc[8 * k + 2] * inv, acc[8 * k + 3] * inv);
    w.z = pack_bf16x2(acc[8 * k + 4] * inv, acc[8 * k + 5] * inv);
    w.w = pack_bf16x2(acc[8 * k + 6] * inv, acc[8 * k + 7] * inv);
    dst[k] = w;
  }
  if (quarter == 0 && p.lse != nullptr) {
    float v = m + logf(sum);
    if constexpr (P::kBias) {  // distances were counted from the nearest visible key
      const int pos = d.off + qrow;
      if (sum != 0.f && score_first_key(p.score, q0 + qrow, pos) > pos)
        v -= p.score.slopes[head] * static_cast<float>(max(0, pos + 1 - d.prefix));
    }
    p.lse[static_cast<int64_t>(q0 + qrow) * p.hq + head] = v;
  }
}

// The jobs of a split call with rows for repair_rows, a warp per head and 32 rows; most calls have none.
template <class P>
__global__ void __launch_bounds__(256, 1) prefill_repair_kernel(const P p) {
  await_previous();
  const PlanHeader& h = *p.ws_plan;
  if (h.repair == 0) return;
  const int warp = threadIdx.x >> 5, t = warp >> 2;
  for (int job = blockIdx.x; job < h.tiles * p.hkv; job += gridDim.x) {
    const int g = job / h.tiles;
    const TileDesc d = p.ws_tiles[job - g * h.tiles];
    if (d.repair >> (2 * g + t) & 1u) repair_rows(p, d, g, t, warp & 3);
  }
}

// ---------------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------------
size_t align256(size_t x) { return (x + 255) / 256 * 256; }

struct ScoreWs {
  size_t plan, tiles, units, first_tile, tail, records, total;
};

ScoreWs score_ws(int batch, int grid, int max_tiles) {
  ScoreWs w;
  w.plan = 0;
  w.tiles = 256;
  w.units = align256(w.tiles + sizeof(TileDesc) * max_tiles);
  w.first_tile = align256(w.units + sizeof(long long) * (max_tiles + 1));
  w.tail = align256(w.first_tile + sizeof(int32_t) * (batch + 1));
  w.records = align256(w.tail + sizeof(long long) * (grid + 1));
  w.total = align256(w.records + 2 * static_cast<size_t>(grid) * kRecordBytes);
  return w;
}

// Query tiles of a call: each chunk may end in one that is not full.
int score_tiles(int64_t total_q, int batch) { return static_cast<int>(total_q / kTileM + batch); }

// One persistent CTA per SM.
int score_grid() { return std::min(sm_count_current_device(), kMaxGrid); }

// Allows an instance its shared memory and reads its registers.
template <class P, bool kWhole>
cudaError_t configure_score(int smem, int* regs) {
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncSetAttribute(prefill_score_kernel<P, kWhole>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, prefill_score_kernel<P, kWhole>);
  if (e == cudaSuccess) *regs = fa.numRegs;
  return e;
}

// Plan, attention, merge and repair of one call, or its attention alone (whole: a CTA per job); each
// is a programmatic dependent of the one before.
template <class P>
pa_status launch_score(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const P& p,
                       int grid, bool whole, cudaStream_t stream) {
  const int smem = static_cast<int>(sizeof(ScoreSmem));
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    int regs = 0, regs_whole = 0;
    cudaError_t e = configure_score<P, false>(smem, &regs);
    if (e == cudaSuccess) e = configure_score<P, true>(smem, &regs_whole);
    if (e != cudaSuccess) return record_cuda_error(e, "cudaFuncSetAttribute(prefill_score)");
    // The in-kernel register split needs the full launch budget; a build that launched with
    // fewer registers per thread would make setmaxnreg.inc wait forever, so refuse to launch.
    if (std::min(regs, regs_whole) < kLaunchRegs) {
      snprintf_error("prefill_score_kernel built with %d registers/thread, needs %d for its split",
                     std::min(regs, regs_whole), kLaunchRegs);
      return PA_ERR_UNSUPPORTED;
    }
    // same carveout for the kernels after it: no reconfiguration between them
    e = cudaFuncSetAttribute(prefill_score_merge_kernel<P>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(prefill_repair_kernel<P>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return record_cuda_error(e, "cudaFuncSetAttribute(prefill score merge)");
    configured_device = dev;
  }
  if (whole) {
    const cudaError_t e = launch_dependent(prefill_score_kernel<P, true>, static_cast<unsigned>(p.max_tiles * p.hkv),
                                           kThreads, smem, stream, 0, qm, km, vm, p);
    return e == cudaSuccess ? PA_OK : record_cuda_error(e, "prefill_score_kernel");
  }
  cudaError_t e = launch_dependent(prefill_plan_kernel<P>, 1, kPlanThreads, 0, stream, 0, p, grid);
  if (e != cudaSuccess) return record_cuda_error(e, "prefill_plan_kernel");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefill_score_kernel<P, false>, qm, km, vm, p);
  if (e != cudaSuccess) return record_cuda_error(e, "prefill_score_kernel");
  cfg.gridDim = dim3((p.max_q_len + kTileM - 1) / kTileM, p.hkv * 8, p.batch);
  cfg.blockDim = dim3(kMergeRows);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, prefill_score_merge_kernel<P>, p);
  if (e != cudaSuccess) return record_cuda_error(e, "prefill_score_merge_kernel");
  e = launch_dependent(prefill_repair_kernel<P>, static_cast<unsigned>(grid), 256, 0, stream, 0, p);
  return e == cudaSuccess ? PA_OK : record_cuda_error(e, "prefill_repair_kernel");
}

}  // namespace

size_t prefill_score_workspace_bytes(int batch, int total_q) {
  const int grid = score_grid();
  if (grid <= 0 || batch <= 0 || total_q < 0) return 0;
  return score_ws(batch, grid, score_tiles(total_q, batch)).total;
}

pa_status launch_prefill_score(int32_t hkv, const void* q, int32_t total_q, const int32_t* cu_q_lens,
                               const void* k_pool, const void* v_pool, int64_t num_pages,
                               const int32_t* block_table, int32_t bt_stride,
                               const int32_t* seq_lens, int32_t batch, int32_t max_q_len,
                               int32_t max_seq_len, float softmax_scale, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, int32_t* status, cudaStream_t stream,
                               int32_t max_ctas, const pa_score_opts& score) {
  if (batch > kMaxBatch) {
    snprintf_error("attn_prefill_chunk_score: at most %d chunks per call", kMaxBatch);
    return PA_ERR_UNSUPPORTED;
  }
  if (num_pages * kPage >= (int64_t(1) << 31) || total_q >= (1 << 24)) return PA_ERR_UNSUPPORTED;
  const int full_grid = score_grid();
  if (full_grid <= 0) return PA_ERR_CUDA;
  const int grid = max_ctas > 0 ? std::min(full_grid, static_cast<int>(max_ctas)) : full_grid;
  const int max_tiles = score_tiles(total_q, batch);
  const ScoreWs w = score_ws(batch, grid, max_tiles);
  if (workspace == nullptr || workspace_bytes < w.total) return PA_ERR_WORKSPACE_TOO_SMALL;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PA_ERR_INVALID_ARG;
  CUtensorMap qm, km, vm;
  const int hq = kGroup * hkv;
  if (!make_map_3d(&qm, q, static_cast<uint64_t>(total_q), hq, kTileM) ||
      !make_map_3d(&km, k_pool, static_cast<uint64_t>(num_pages) * kPage, hkv, kPage) ||
      !make_map_3d(&vm, v_pool, static_cast<uint64_t>(num_pages) * kPage, hkv, kPage)) {
    snprintf_error("cuTensorMapEncodeTiled failed for the prefill operands");
    return PA_ERR_CUDA;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto run = [&](auto p) {
    p.hkv = hkv;
    p.hq = hq;
    p.cu_q_lens = cu_q_lens;
    p.seq_lens = seq_lens;
    p.block_table = block_table;
    p.bt_stride = bt_stride;
    p.batch = batch;
    p.num_pages = num_pages;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.status = status;
    p.score = score_params(score, softmax_scale, &p.scale_log2);
    p.total_q = total_q;
    p.max_tiles = max_tiles;
    p.max_q_len = max_q_len;
    p.q_rows = static_cast<const uint16_t*>(q);
    p.k_rows = static_cast<const uint16_t*>(k_pool);
    p.v_rows = static_cast<const uint16_t*>(v_pool);
    p.ws_plan = reinterpret_cast<PlanHeader*>(ws + w.plan);
    p.ws_tiles = reinterpret_cast<TileDesc*>(ws + w.tiles);
    p.ws_units = reinterpret_cast<long long*>(ws + w.units);
    p.ws_first_tile = reinterpret_cast<int32_t*>(ws + w.first_tile);
    p.ws_tail = reinterpret_cast<long long*>(ws + w.tail);
    p.ws_records = ws + w.records;
    return launch_score(qm, km, vm, p, grid, max_tiles * hkv <= grid && max_seq_len <= kWholeKeys, stream);
  };
  const bool cap = score.softcap > 0.f, bias = score.alibi_slopes != nullptr;
  return cap ? (bias ? run(PrefillScoreParams<true, true>()) : run(PrefillScoreParams<true, false>()))
             : (bias ? run(PrefillScoreParams<false, true>()) : run(PrefillScoreParams<false, false>()));
}

}  // namespace pa
