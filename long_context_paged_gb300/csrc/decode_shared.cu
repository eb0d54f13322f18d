// attn_decode_paged_shared: decode attention of rows that share leading pages (sm_103a).
//
// Row r's softmax over its L_r keys is a sum over two disjoint sets, the keys of the pages that its
// group shares and the keys of its own pages after them:
//     o_r = (e^{m1} O1_r + e^{m2} O2_r) / (e^{m1} l1_r + e^{m2} l2_r),
// with running maximum m, sum l and unnormalised O of each set. The first set is the same for the whole
// group, so its K and V are read once and meet all the group's query rows in one matrix product:
// 64 rows x the 2 query heads of a KV head are the 128 rows of a tcgen05 tile. With R rows a shared key
// costs 512 bytes of a KV head's cache and 4 * 128 * 2 R operations, so up to about 64 rows the call is
// bound by HBM and reads the shared keys at its rate, R times fewer bytes than the plain decode.
//
// Measured on a GB300 (calls of a graph, 152 CTAs): 16 groups of 4 rows over 5,000 to 30,000 keys 155 us,
// 6.3 TB/s of the bytes that have to be read (0.93 of a copy's rate; 64 rows read alone would be 3.7 GB);
// 8 rows over 67,500 keys 59 us, of which the units take 41 (6.7 TB/s), the plan 3.5, the first copies 3.7,
// the merge and its start 5 and the slowest CTA 4; 4 rows over 1,000 keys 13.4 us, a chain of latencies;
// 307 rows in 4 groups 85 us, of which the units take 62 (64 rows a pass: three passes over the keys of 131
// rows; about 290 of the 955 units a head are of such tiles, the others of few or single rows), the plan 4, the
// slowest CTA 6, the merge 6. Short calls of few rows are quicker as attn_decode_paged, which reads a shared key
// once a row, in one launch: for one group of R rows over n keys up to about (R - 1) n = 27,000 (4 rows over 1,000
// keys 6.5 us, 2 over 16,000 22 and 24, 8 over 3,000 17 and 18).
//
// Work split. A segment is a run of keys with the rows that see all of it: (64 rows of a group, its
// shared pages) or (one row, its own pages). Segments are cut into units of 128 keys, laid end to end
// and divided into equal slices, one per CTA of a KV head; the Hkv CTAs of a slice read the heads of
// the same pages at about the same time. A slice's part of a segment (a piece) leaves (m, l, O) in the
// workspace; the merge joins a row's pieces of both sets. The segments are laid out from lengths that only the
// GPU knows: by every CTA for itself, or, where there are many, by a plan kernel of one CTA.
//
// Per unit, in a CTA: S = Q K^T (A = Q, B = K in shared memory, fp32 in TMEM), P = 2^(scale S - m) by a
// thread per row, written over S as bf16, O += P V (A = P in TMEM, B = V in shared memory). With 8 rows or
// fewer most of those 128 matrix rows would be padding and one warp would do all exponentials, so the
// products are turned round: S^T = K Q^T (A = K, 16 columns), a thread per key, O^T += V^T P^T (A = V, B = P
// in shared memory; 16 x 4 rows: 190 us with a thread per row, 169 with a thread per key). There the weights are
// two bf16s each, 16 more columns that cost nothing measurable, so that beams' and single rows' results are
// the plain decode's. Units go to two softmax warpgroups in turn, each with an S and an O of its own, so that one's
// exponentials run beside
// the other's products. K and V come by tiled TMA, a page per copy.
//
// Tried and left out: 64-key units (16 x 4 rows 216 -> 270 us: an issuing thread's waits and commits cost
// more than its products); two row tiles on one K/V tile, a stream each, for 65 to 128 rows (4 groups of up to
// 131 rows 112 -> 148 us: a stream's scores wait for its own weights and products, which two streams on
// alternate units hide).
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>

#include "dependent_launch.cuh"
#include "pa_common.cuh"
#include "tc_common.cuh"

namespace pa {

bool make_map_pages(CUtensorMap* map, const void* base, uint64_t num_pages, uint64_t heads);
bool make_map_heads(CUtensorMap* map, const void* base, uint64_t outer, uint64_t heads, uint32_t box_heads,
                    uint32_t box_rows);

namespace {

constexpr int kTileRows = 64;     // rows of a group per segment (x 2 query heads = 128)
constexpr int kFewRows = 8;       // a segment of so many rows is computed with its keys as the matrix's rows
constexpr int kFew = 2 * kFewRows;
constexpr int kTileKeys = 128;    // keys of a unit
constexpr int kTilePages = kTileKeys / kPage;
constexpr int kStages = 3;        // K and V tiles in flight, of each
constexpr int kThreads = 384;     // 8 softmax warps, two producers, two MMA issuers
constexpr int kKProducerWarp = 8;  // units, Q and K
constexpr int kVProducerWarp = 11;
constexpr int kPvWarp = 9;        // issues O += P V
constexpr int kScoreWarp = 10;    // issues S = Q K^T
constexpr int kInfos = 8;         // published units in flight: more than the stages can hold
constexpr int kQBoxRows = 8;      // query rows of a copy
constexpr uint32_t kTileBytes = kTileKeys * 256;   // a unit's keys
constexpr uint32_t kQBlockBytes = 128 * 128;
constexpr uint32_t kPageBytes = kPage * 256;       // a page's 16 keys of one head: two groups of 8 keys, each
constexpr uint32_t kGroupBytes = 8 * 256;          // of them 1 KB of the first 64 dims and 1 KB of the others
constexpr uint32_t kHalfBytes = 8 * 128;
// The Q buffer: a segment of many rows has all of it. Those of few rows, which come after all of those,
// have two small Q buffers in turn and, for each stream, their weights in it (bf16 [2 halves of the keys]
// [kFew rows' high parts, then their low ones][64 keys]).
constexpr uint32_t kFewHalfBytes = kFew * 128;
constexpr uint32_t kFewQBytes = 2 * kFewHalfBytes;
constexpr uint32_t kWeightsAt = 2 * kFewQBytes;
constexpr uint32_t kWeightHalfBytes = 2 * kFewHalfBytes;
constexpr uint32_t kWeightBytes = 2 * kWeightHalfBytes;
static_assert(kWeightsAt + 2 * kWeightBytes <= 2 * kQBlockBytes, "the small buffers fit in the large one");
constexpr float kRescaleThreshold = 8.0f;     // log2 units a row's maximum may lag behind
constexpr int kMaxBatch = 4096;
constexpr int kMaxGroups = 4096;
constexpr int kMaxKeys = 131072;  // of a sequence: units are counted in 32 bits
constexpr int kMaxSlices = 256;   // CTAs per KV head
// Registers of a softmax thread and of the others; 256 x 208 + 128 x 88 = 384 x 168, what the CTA is
// launched with (checked on the host).
constexpr int kSoftmaxRegs = 208;
constexpr int kControlRegs = 88;
constexpr int kLaunchRegs = (256 * kSoftmaxRegs + 128 * kControlRegs) / kThreads;
constexpr int kRowFloats = kHeadDim + 2;      // O and (m, l) of a query row in the workspace

struct Segment {
  int32_t unit, units;       // first unit and number of units
  int32_t row, rows;         // query rows
  int32_t table_row;         // whose table entries are read
  int32_t first_key, end_key;
  int32_t place;             // of its results among those of shared pages, in rows; ~place among those of the rows' own
};

// Where a row's partial results are: its segment of shared pages and its own, in units and as places among
// the results (units = 0: none).
struct RowPlan {
  int32_t tile_unit, tile_units, tile, in_tile;  // in_tile: the row's place in the segment
  int32_t own_unit, own_units, own, tile_rows;   // tile_rows: the segment's rows
};

// A slice: its units, the segment of the first one, and what all slices have alike.
struct Slice {
  int32_t u0, u1, segment;
  int32_t segments, units;  // of all slices
  int32_t pad[3];
};

struct SharedParams {
  int32_t hkv, hq, batch, groups, max_group_rows, bt_stride, max_seq_len;
  const int32_t* seq_lens;
  const int32_t* block_table;
  const int32_t* cu_group_rows;
  const int32_t* shared_pages;
  int64_t num_pages;
  float scale_log2;
  int32_t slices;       // CTAs per KV head
  int32_t tile_rows;    // most rows of a shared segment
  uint16_t* out;
  float* lse;
  int32_t* status;
  Slice* slice;            // [slices]
  Segment* segments;
  Segment* own_segments;   // [CTAs][kOwnPlanSegments]
  RowPlan* rows;           // [batch]
  // Partial results: of a piece of R rows [hkv][2 streams]([2 R][128], then (m, l) of each), where the results of
  // (slice, place) begin, in rows. A segment of shared pages with many rows has its first row for its place, one
  // with few rows that and `batch` (they come after all of those); a row's own segment, its number among those. Places
  // go up by a segment's rows from one to the next, and the slices' starts by tile_rows, so pieces, which go up in
  // both, do not overlap.
  float* tile_parts;       // slices * tile_rows + 2 * batch rows
  float* row_parts;        // slices + batch rows
};

constexpr int kPartFloats = 2 * 2 * kRowFloats;  // of a row and KV head: two streams, two query heads

// ---------------------------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;  // at most: four rows a thread

// Numbers of segments and their units travel as one word, segments above kShift bits of units.
template <int kGroups, int kRows, class Word, int kShift>
struct PlanSmem {
  using Packed = Word;
  static constexpr int kUnitBits = kShift;
  Packed warp_sums[3][kPlanThreads / 32];
  Packed totals[3];
  Slice own;  // of the CTA (a plan made by every CTA)
  // groups: first row, shared pages, first row that uses them; segments and units before the group's of
  // many rows, and before its one of few
  int32_t cu[kGroups + 1], shared[kGroups], first[kGroups];
  int32_t many_unit[kGroups], few_seg[kGroups], few_unit[kGroups];
  // rows: keys, last group that starts at or before the row (-1: none), pages that it shares; segments
  // and units of own pages before the row's
  int32_t len[kRows], group[kRows], start[kRows];
  int32_t own_seg[kRows + 1], own_unit[kRows + 1];
  int32_t unit[kGroups + kRows + kRows / kTileRows + 1];  // first unit of each segment
};
using PlanOfAll = PlanSmem<kMaxGroups, kMaxBatch, unsigned long long, 40>;
static_assert(sizeof(PlanOfAll) <= 232448, "shared memory over the 227 KB limit");

// A call of no more segments than this is planned by every CTA for itself, its slice's segments kept in its part
// of the workspace: that spares the launch of a plan kernel and the wait for it (4 rows over 1,000 keys 15.0 ->
// 13.8 us, 307 rows 102 -> 94, with the merge of then). Larger ones have the plan kernel.
constexpr int kOwnPlanSegments = 512;
using OwnPlan = PlanSmem<kOwnPlanSegments, kOwnPlanSegments, uint32_t, 20>;
static_assert(kOwnPlanSegments < 1 << 12 && kOwnPlanSegments * (kMaxKeys / kTileKeys) < 1 << 20, "fits in a word");

template <class T>
__device__ __forceinline__ T warp_scan_sum(T v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

// Exclusive prefix sums over the CTA of three packed numbers, and their totals.
template <class Smem>
__device__ __forceinline__ void plan_scan(Smem& s, typename Smem::Packed (&v)[3]) {
  using T = typename Smem::Packed;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    incl[k] = warp_scan_sum(v[k], lane);
    if (lane == 31) s.warp_sums[k][warp] = incl[k];
  }
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const T w = lane < static_cast<int>(blockDim.x >> 5) ? s.warp_sums[k][lane] : 0;
      const T x = warp_scan_sum(w, lane);
      s.warp_sums[k][lane] = x - w;
      if (lane == 31) s.totals[k] = x;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) v[k] = s.warp_sums[k][warp] + incl[k] - v[k];
}

__device__ __forceinline__ int units_of(int keys) { return (keys + kTileKeys - 1) / kTileKeys; }

// The slices' bounds U i / n and the slice of a unit by 32-bit divisions where they do (64-bit ones take
// several times as long, and the calls' starts and ends wait for them).
struct Divider {
  bool small;
  __device__ Divider(uint32_t U, uint32_t n) : small(U < 0xffffffffu / (n + 1)) {}
  __device__ __forceinline__ int operator()(uint64_t x, uint32_t d) const {  // x < U (n + 1)
    return small ? static_cast<int>(static_cast<uint32_t>(x) / d) : static_cast<int>(x / d);
  }
};

// Slice i, but for the segment of its first unit.
__device__ __forceinline__ Slice slice_of(const SharedParams& p, int2 plan, int i) {
  const Divider over(plan.y, p.slices);
  const int u0 = over(static_cast<uint64_t>(plan.y) * i, p.slices), u1 = over(static_cast<uint64_t>(plan.y) * (i + 1), p.slices);
  return Slice{u0, u1, 0, plan.x, plan.y, {0, 0, 0}};
}

// The segments (with kOwn those of slice `slice` alone) into `segments`, and where rows_out is set the rows' places
// into p.rows. Returns the number of segments and of units. Loops are not unrolled: this code runs once, and its time is what fetching it takes.
template <bool kOwn, class Smem>
__device__ __forceinline__ int2 make_plan(const SharedParams& p, Smem& s, Segment* segments, int slice, bool rows_out) {
  const int tid = threadIdx.x, threads = static_cast<int>(blockDim.x), G = p.groups, B = p.batch;
  int32_t* status = rows_out ? p.status : nullptr;  // (one CTA reports)
  bool bad = false;
  using Packed = typename Smem::Packed;
  constexpr Packed kOne = static_cast<Packed>(1) << Smem::kUnitBits;
  auto count_of = [](Packed v) { return static_cast<int>(v >> Smem::kUnitBits); };
  auto units_in = [](Packed v) { return static_cast<int>(v & (kOne - 1)); };
#pragma unroll 1
  for (int b = tid; b < B; b += threads) {
    int len = p.seq_lens[b];
    const int most = min(p.bt_stride * kPage, kMaxKeys);
    if (len < 0 || len > most || len > p.max_seq_len) flag_error(status, PA_DEV_ERR_LENGTH);
    s.len[b] = min(max(len, 0), most);
  }
#pragma unroll 1
  for (int g = tid; g < G; g += threads) {
    const int a = p.cu_group_rows[g], b = p.cu_group_rows[g + 1];
    int n = p.shared_pages[g];
    s.cu[g] = a;
    if (g == G - 1) s.cu[G] = b;
    bad |= a < 0 || b < a || b > B || b - a > p.max_group_rows;
    if (n < 0 || n > p.bt_stride) {
      flag_error(status, PA_DEV_ERR_LENGTH);
      n = 0;
    }
    s.shared[g] = n;
    s.first[g] = 0x7fffffff;
  }
  // groups that are not disjoint ranges of rows: no row shares anything
  bad = __syncthreads_or(bad);
  const bool grouped = G > 0 && !bad;
  if (bad && tid == 0) flag_error(status, PA_DEV_ERR_LENGTH);
#pragma unroll 1
  for (int b = tid; b < B; b += threads) {
    int lo = -1, start = 0;
    if (grouped && b >= s.cu[0]) {
      int hi = G;
      lo = 0;
#pragma unroll 1
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.cu[mid] <= b) lo = mid; else hi = mid;
      }
      // a row shorter than the shared pages reads its own keys alone
      if (b < s.cu[lo + 1] && s.shared[lo] > 0 && s.len[b] >= s.shared[lo] * kPage) {
        start = s.shared[lo];
        atomicMin(&s.first[lo], b);
      }
    }
    s.group[b] = lo;
    s.start[b] = start;
  }
  __syncthreads();
  // Segments, in this order: those of shared pages with many rows (a CTA never goes back to them from
  // those with few); then by row the rows' own pages, a group's shared pages with few rows before its
  // first row (short segments wait for memory more than they read, so they are spread over the slices).
  const int gper = (G + threads - 1) / threads, g0 = min(G, tid * gper), g1 = min(G, g0 + gper);
  const int per = (B + threads - 1) / threads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
  auto rows_of = [&](int g) { return grouped && s.first[g] != 0x7fffffff ? s.cu[g + 1] - s.cu[g] : 0; };
  auto few_of = [&](int rows) { return rows % kTileRows <= kFewRows ? rows % kTileRows : 0; };
  Packed at[3] = {0, 0, 0};  // many, few, own
#pragma unroll 1
  for (int g = g0; g < g1; ++g) {
    const int rows = rows_of(g), few = few_of(rows), units = units_of(s.shared[g] * kPage);
    const Packed many = (rows - few + kTileRows - 1) / kTileRows;
    at[0] += many * kOne + many * units;
    if (few > 0) at[1] += kOne + units;
  }
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int units = units_of(s.len[b] - s.start[b] * kPage);
    if (units > 0) at[2] += kOne + units;
  }
  plan_scan(s, at);
  const int many_tiles = count_of(s.totals[0]), many_units = units_in(s.totals[0]);
  const int count = many_tiles + count_of(s.totals[1]) + count_of(s.totals[2]);
  const int units_all = many_units + units_in(s.totals[1]) + units_in(s.totals[2]);
  const Slice own = slice_of(p, make_int2(count, units_all), slice);
  auto put = [&](int seg, const Segment& g) {
    if (!kOwn || (g.unit < own.u1 && g.unit + g.units > own.u0)) segments[seg] = g;
    s.unit[seg] = g.unit;
  };
  int few_seg = count_of(at[1]), few_unit = units_in(at[1]);
  {
    int seg = count_of(at[0]), unit = units_in(at[0]);
#pragma unroll 1
    for (int g = g0; g < g1; ++g) {
      const int rows = rows_of(g), few = few_of(rows), units = units_of(s.shared[g] * kPage);
      s.many_unit[g] = unit;
#pragma unroll 1
      for (int r = 0; r < rows - few; r += kTileRows) {
        put(seg, Segment{unit, units, s.cu[g] + r, min(kTileRows, rows - few - r), s.first[g], 0,
                         s.shared[g] * kPage, s.cu[g] + r});
        ++seg;
        unit += units;
      }
      s.few_seg[g] = few_seg;
      s.few_unit[g] = few_unit;
      if (few > 0) {
        ++few_seg;
        few_unit += units;
      }
    }
  }
  {
    int seg = count_of(at[2]), unit = units_in(at[2]);
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int units = units_of(s.len[b] - s.start[b] * kPage);
      s.own_seg[b] = seg;
      s.own_unit[b] = unit;
      if (units > 0) {
        ++seg;
        unit += units;
      }
    }
    if (tid == 0) {
      s.own_seg[B] = count_of(s.totals[2]);
      s.own_unit[B] = units_in(s.totals[2]);
      s.unit[count] = units_all;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int g = tid; g < G; g += threads) {
    const int rows = rows_of(g), few = few_of(rows);
    if (few == 0) continue;
    const int row = s.cu[g], seg = many_tiles + s.few_seg[g] + s.own_seg[row];
    const int unit = many_units + s.few_unit[g] + s.own_unit[row];
    put(seg, Segment{unit, units_of(s.shared[g] * kPage), row + rows - few, few, s.first[g], 0,
                     s.shared[g] * kPage, B + row + rows - few});
  }
#pragma unroll 1
  for (int b = tid; b < B; b += threads) {
    const int g = s.group[b], start = s.start[b], units = units_of(s.len[b] - start * kPage);
    RowPlan r{0, 0, 0, 0, 0, 0, 0, 0};
    int seg = many_tiles + s.own_seg[b], unit = many_units + s.own_unit[b];
    if (g >= 0) {
      const int rows = rows_of(g), few = few_of(rows), in_group = b - s.cu[g];
      seg += s.few_seg[g] + (few > 0 ? 1 : 0);
      unit += s.few_unit[g] + (few > 0 ? units_of(s.shared[g] * kPage) : 0);
      if (rows_out && start > 0) {
        const int tile = in_group / kTileRows;
        r.tile_units = units_of(start * kPage);
        r.in_tile = in_group % kTileRows;
        r.tile = b - r.in_tile;
        if (in_group < rows - few) {
          r.tile_rows = min(kTileRows, rows - few - tile * kTileRows);
          r.tile_unit = s.many_unit[g] + tile * r.tile_units;
        } else {
          r.tile += B;
          r.tile_rows = few;
          r.tile_unit = many_units + s.few_unit[g] + s.own_unit[s.cu[g]];
        }
      }
    }
    if (units > 0) {
      r.own = s.own_seg[b];
      r.own_unit = unit;
      r.own_units = units;
      put(seg, Segment{unit, units, b, 1, b, start * kPage, s.len[b], ~r.own});
    }
    if (rows_out) p.rows[b] = r;
  }
  __syncthreads();
  return make_int2(count, units_all);
}

__global__ void __launch_bounds__(kPlanThreads, 1) shared_plan_kernel(const SharedParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  PlanOfAll& s = *reinterpret_cast<PlanOfAll*>(smem_raw);
  launch_next();
  await_previous();
  const int2 plan = make_plan<false>(p, s, p.segments, 0, true);
#pragma unroll 1
  for (int i = threadIdx.x; i < p.slices; i += static_cast<int>(blockDim.x)) {
    Slice own = slice_of(p, plan, i);
    int lo = 0, hi = max(plan.x, 1);  // last segment with a first unit <= u0
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.unit[mid] <= own.u0) lo = mid; else hi = mid;
    }
    own.segment = lo;
    p.slice[i] = own;
  }
}

// ---------------------------------------------------------------------------------------------
// attention over the slices
// ---------------------------------------------------------------------------------------------
constexpr int kFirst = 1, kLast = 2;          // of this stream in the piece
constexpr int kPieceStart = 4, kPieceEnd = 8; // of the piece
constexpr int kQBuffer1 = 16;                 // else buffer 0
constexpr int kFewFlag = 32;                  // few rows: keys are the matrix's rows

struct UnitInfo {
  int64_t part;     // where stream 0's partial result goes, in floats; row r's O at + 128 r
  int32_t stats;    // (m, l) of row r at part + stats + 2 r; stream 1's result at part + stats / 128 * kRowFloats
  int32_t keys;
  int32_t flags;
  int32_t rows;     // query rows x heads
  int32_t is_tile;
  int32_t pad;
};

struct SharedSmem {
  uint8_t k[kStages][kTileBytes];
  uint8_t v[kStages][kTileBytes];
  uint8_t q[2 * kQBlockBytes];
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t info_full[kInfos];
  uint64_t s_full[2], p_full[2], p_free[2], o_ready[2], o_free[2];
  uint64_t few_ready[2][2], few_free[2][2];  // of a stream's two O with few rows
  uint64_t mma_done[2], met[2];
  uint32_t tmem_base;
  float exchange[2][3][4][kFew];  // of each stream: maxima (two, in turn) and sums, per warp and row
  UnitInfo info[kInfos];
};
static_assert(sizeof(SharedSmem) <= 232448, "shared memory over the 227 KB limit");
static_assert(sizeof(OwnPlan) <= 2 * kStages * kTileBytes, "an own plan fits in the ring");

__device__ __forceinline__ bool wait_or_flag(uint64_t* bar, uint32_t parity, int32_t* status) {
  if (mbar_wait_bounded(bar, parity)) return true;
  flag_error(status, PA_DEV_ERR_TIMEOUT);
  return false;
}

// The same for a whole warp, one lane of it polling: 32 lanes of eight warps at it slow every other
// thread's barrier operations down.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int lane, int32_t* status) {
  bool ok = true;
  if (lane == 0) ok = wait_or_flag(bar, parity, status);
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();  // (what the wait of one lane made visible is visible to the others)
  return ok;
}

// kOwnPlan: the CTA makes its plan itself.
template <bool kOwnPlan>
__global__ void __launch_bounds__(kThreads, 1)
shared_attention_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap v_map, const SharedParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  SharedSmem& s = *reinterpret_cast<SharedSmem*>(smem_raw);
  const int head = static_cast<int>(blockIdx.x) % p.hkv, slice = static_cast<int>(blockIdx.x) / p.hkv;
  if ((smem_addr(smem_raw) & 1023u) != 0) {  // not the layout this kernel was built for
    await_previous();
    if (threadIdx.x == 0) flag_error(p.status, PA_DEV_ERR_INTERNAL);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.k_full[i], 1);
      mbar_init(&s.k_empty[i], 1);
      mbar_init(&s.v_full[i], 1);
      mbar_init(&s.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.q_full[i], 1);
      mbar_init(&s.q_empty[i], 1);
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], 4);
      mbar_init(&s.p_free[i], 1);
      mbar_init(&s.mma_done[i], 1);
      mbar_init(&s.met[i], 4);
      mbar_init(&s.o_ready[i], 1);
      mbar_init(&s.o_free[i], 4);
      for (int k = 0; k < 2; ++k) {
        mbar_init(&s.few_ready[i][k], 1);
        mbar_init(&s.few_free[i][k], 4);
      }
    }
    for (int i = 0; i < kInfos; ++i) mbar_init(&s.info_full[i], 1);
    fence_mbar_init();
  }
  if (warp == kPvWarp) tc::tmem_alloc<512>(&s.tmem_base);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s.tmem_base;  // S_0 [0, 128), S_1 [128, 256), O_0 [256, 384), O_1 [384, 512); few rows:
                                      // S_t [0, 16) and two O_t of 32 columns at [64, 128) of the stream's S
  await_previous();
  Slice plan;
  Segment* own_segments = p.own_segments + static_cast<int64_t>(blockIdx.x) * kOwnPlanSegments;
  if (kOwnPlan) {
    OwnPlan& ps = *reinterpret_cast<OwnPlan*>(smem_raw);  // (in the ring, which is not in use yet)
    const int2 all = make_plan<true>(p, ps, own_segments, slice, blockIdx.x == 0);
    plan = slice_of(p, all, slice);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.slice[0] = plan;  // (for the merge)
    for (int i = threadIdx.x; i < all.x; i += kThreads)
      if (ps.unit[i] <= plan.u0 && plan.u0 < ps.unit[i + 1]) ps.own.segment = i;
    __syncthreads();
    plan.segment = ps.own.segment;
    tc::fence_proxy_async_smem();  // the ring's copies come after these accesses
    __syncthreads();
  } else {
    plan = p.slice[slice];
  }
  const int u0 = plan.u0, u1 = plan.u1, nt = u1 - u0;

  if (warp >= 8) {
    tc::regs_decrease<kControlRegs>();
  if (warp == kKProducerWarp || warp == kVProducerWarp) {
    // ------------------------------------------------------------------ producers
    // Both walk the slice's units; one loads Q and K and publishes the units, the other loads V. A copy
    // takes its issuing warp about 75 cycles, so a page is one copy, and K and V have a warp each (two
    // copies a page from one warp: 3,700 cycles a unit, whose bytes take 2,800 to arrive).
    const bool is_k = warp == kKProducerWarp;
    const CUtensorMap* map = is_k ? &k_map : &v_map;
    uint8_t(*ring)[kTileBytes] = is_k ? s.k : s.v;
    uint64_t* full = is_k ? s.k_full : s.v_full;
    uint64_t* empty = is_k ? s.k_empty : s.v_empty;
    bool ok = true;
    int it = 0, next_q = 0;
    uint32_t q_par = 0, q_used = 0;  // bit b: parity of Q buffer b's next load; whether it had one
    uint32_t st = 0, ph = 0, loads = 0;  // next ring stage, its parity, tiles loaded
    // Segments' records are read 32 at a time, a lane each; table entries 32 at a time (kBatch units), a
    // batch ahead, and those of the next segment's first units while this one's are loaded: an entry
    // read just before its copies would cost its latency in every unit.
    constexpr int kBatch = 32 / kTilePages;
    int seg = plan.segment, records = seg;
    Segment lane_record{};
    if (!kOwnPlan) lane_record = p.segments[max(0, min(seg + lane, plan.segments - 1))];
    auto record = [&](int i) {
      if (kOwnPlan) return own_segments[i];
      if (i >= records + 32) {
        records = i;
        lane_record = p.segments[min(i + lane, plan.segments - 1)];
      }
      const int from = i - records;
      Segment g;
      g.unit = __shfl_sync(0xffffffffu, lane_record.unit, from);
      g.units = __shfl_sync(0xffffffffu, lane_record.units, from);
      g.row = __shfl_sync(0xffffffffu, lane_record.row, from);
      g.rows = __shfl_sync(0xffffffffu, lane_record.rows, from);
      g.table_row = __shfl_sync(0xffffffffu, lane_record.table_row, from);
      g.first_key = __shfl_sync(0xffffffffu, lane_record.first_key, from);
      g.end_key = __shfl_sync(0xffffffffu, lane_record.end_key, from);
      g.place = __shfl_sync(0xffffffffu, lane_record.place, from);
      return g;
    };
    auto entries = [&](const Segment& g, int k) {
      const int key = g.first_key + k * kTileKeys + lane * kPage;
      return key < g.end_key ? p.block_table[static_cast<int64_t>(g.table_row) * p.bt_stride + key / kPage] : 0;
    };
    Segment g{};
    if (nt > 0) g = record(seg);
    int batch = nt > 0 ? entries(g, u0 - g.unit) : 0;
    while (it < nt && ok) {
      const int k0 = u0 + it - g.unit, k1 = min(u1 - g.unit, g.units);
      Segment next = g;
      int next_batch = 0;
      if (it + k1 - k0 < nt) {
        next = record(seg + 1);
        next_batch = entries(next, 0);
      }
      const bool few = g.rows <= kFewRows;
      const int qb = few ? next_q : 0;
      if (is_k) {
        // (the first segment of few rows takes the barrier of those of many: none of them is left)
        if (lane == 0) ok = wait_or_flag(&s.q_empty[qb], (q_par >> qb & 1) ^ 1u, p.status);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        const int boxes = (g.rows + kQBoxRows - 1) / kQBoxRows;
        uint8_t* to = s.q + (few ? qb * kFewQBytes : 0) + (lane & 1) * (few ? kFewHalfBytes : kQBlockBytes);
        if (lane == 0) mbar_arrive_expect_tx(&s.q_full[qb], boxes * 2 * (2 * kQBoxRows * 128));
        __syncwarp();
        if (lane < 2 * boxes)
          tc::tma_load_3d(to + (lane >> 1) * (2 * kQBoxRows * 128), &q_map, (lane & 1) * 64, 2 * head,
                          g.row + (lane >> 1) * kQBoxRows, &s.q_full[qb]);
        q_par ^= 1u << qb;
        q_used |= 1u << qb;
      }
      if (few) next_q = qb ^ 1;
      const bool is_tile = g.place >= 0;
      for (int kb = k0; kb < k1 && ok; kb += kBatch) {
        const int ahead = kb + kBatch < k1 ? entries(g, kb + kBatch) : 0;
        for (int k = kb; k < min(kb + kBatch, k1); ++k, ++it) {
          const int keys = min(kTileKeys, g.end_key - (g.first_key + k * kTileKeys));
          const int pages = (keys + kPage - 1) / kPage;
          // lane i copies the unit's page i
          int e = __shfl_sync(0xffffffffu, batch, (k - kb) * kTilePages + (lane & (kTilePages - 1)));
          if (lane < pages && (e < 0 || e >= p.num_pages)) {
            flag_error(p.status, PA_DEV_ERR_PAGE_OOB);
            e = 0;
          }
          if (lane == 0) ok = wait_or_flag(&empty[st], ph ^ 1u, p.status);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          // K's barrier hands the info on. The unit that its slot held last has been consumed: K's stage
          // was released by the scores of unit it - kStages, which were issued after P V of the unit two
          // before that one (it - 5; a slot serves every eighth).
          if (is_k && lane == 0) {
            UnitInfo& f = s.info[it % kInfos];
            const int from = is_tile ? slice * p.tile_rows + g.place : slice + ~g.place;  // (below 2^15)
            f.part = (static_cast<int64_t>(from) * p.hkv + head * g.rows) * kPartFloats;
            f.stats = 2 * g.rows * kHeadDim;
            f.keys = keys;
            f.flags = (k - k0 < 2 ? kFirst : 0) | (k1 - 1 - k < 2 ? kLast : 0) | (k == k0 ? kPieceStart : 0) |
                      (k == k1 - 1 ? kPieceEnd : 0) | (qb ? kQBuffer1 : 0) | (few ? kFewFlag : 0);
            f.rows = 2 * g.rows;
            f.is_tile = is_tile ? 1 : 0;
            mbar_arrive(&s.info_full[it % kInfos]);
          }
          if (lane == 0) mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(pages) * kPageBytes);
          __syncwarp();
          if (lane < pages) tc::tma_load_5d(ring[st] + lane * kPageBytes, map, 0, 0, 0, 2 * e, head, &full[st]);
          ++loads;
          if (++st == kStages) {
            st = 0;
            ph ^= 1u;
          }
        }
        batch = ahead;
      }
      ++seg;
      g = next;
      batch = next_batch;
    }
    // do not leave while copies into this CTA's shared memory may still be landing (only after a wait
    // that gave up: else all of them have been consumed)
    if (!ok && lane == 0) {
      for (uint32_t k = loads > kStages ? loads - kStages : 0; k < loads; ++k)
        wait_or_flag(&full[k % kStages], (k / kStages) & 1, p.status);
      for (int b = 0; b < 2; ++b)
        if (q_used >> b & 1) wait_or_flag(&s.q_full[b], (q_par >> b & 1) ^ 1u, p.status);
    }
    __syncwarp();
  } else if (warp == kScoreWarp) {
    // ------------------------------------------------------------------ S = Q K^T
    // Two warps issue the two products: every wait, group of instructions and commit takes an issuing
    // thread some hundred cycles (measured: a wait on a phase long complete 170 to 300, 8 instructions
    // 590, all of a 64-key unit 2,300 from one thread, 1.6 times what its bytes take to arrive).
    if (lane == 0) {
      const uint64_t dq = tc::smem_desc_sw128(smem_addr(s.q), 16, 1024);
      const uint64_t dk = tc::smem_desc_sw128(smem_addr(s.k[0]), 16, kGroupBytes);
      bool ok = true;
      uint32_t st = 0, ph = 0;
      // bits (an array indexed at run time would live in memory): of Q buffer b, the parity of its next
      // load; of stream t, the parity of its next unit and whether it had one
      uint32_t q_par = 0, par = 0, had = 0;
      for (int it = 0; it < nt; ++it) {
        ok = wait_or_flag(&s.k_full[st], ph, p.status);
        if (!ok) break;
        const volatile UnitInfo& f = s.info[it % kInfos];
        const int pages = (f.keys + kPage - 1) / kPage, flags = f.flags;
        const int t = it & 1, qb = flags & kQBuffer1 ? 1 : 0;
        // S takes the columns of the stream's last P
        if (had >> t & 1) ok = wait_or_flag(&s.p_free[t], (par >> t & 1) ^ 1u, p.status);
        had |= 1u << t;
        par ^= 1u << t;
        if (flags & kPieceStart) {
          ok = ok && wait_or_flag(&s.q_full[qb], q_par >> qb & 1, p.status);
          q_par ^= 1u << qb;
        }
        if (!ok) break;
        tc::fence_after_sync();
        const uint64_t k = dk + (st * kTileBytes >> 4);
        const uint32_t to = tmem + t * kTileKeys;
        if (flags & kFewFlag) {  // S^T = K Q^T, of all the tile's keys: those past the unit's are not used
          constexpr uint32_t id = tc::idesc_bf16(128, kFew, 0, 0);
          const uint64_t q = dq + (qb * kFewQBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t step = (kk & 3) * 32;
            const uint64_t qk = q + (((kk >> 2) * kFewHalfBytes + step) >> 4);
            const uint64_t kk_ = k + (((kk >> 2) * kHalfBytes + step) >> 4);
            if (kk == 0) tc::mma_ss_c<false>(to, kk_, qk, id);
            else tc::mma_ss_c<true>(to, kk_, qk, id);
          }
        } else {  // S = Q K^T; N = the unit's keys in whole pages
          const uint32_t id = tc::idesc_bf16(128, 0, 0, 0) | static_cast<uint32_t>(pages * kPage >> 3) << 17;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t step = (kk & 3) * 32;
            const uint64_t qk = dq + (((kk >> 2) * kQBlockBytes + step) >> 4);
            const uint64_t kk_ = k + (((kk >> 2) * kHalfBytes + step) >> 4);
            if (kk == 0) tc::mma_ss_c<false>(to, qk, kk_, id);
            else tc::mma_ss_c<true>(to, qk, kk_, id);
          }
        }
        tc::mma_commit(&s.s_full[t]);
        tc::mma_commit(&s.k_empty[st]);
        if (flags & kPieceEnd) tc::mma_commit(&s.q_empty[qb]);
        if (++st == kStages) {
          st = 0;
          ph ^= 1u;
        }
      }
      // every product must have finished before TMEM is released
      tc::mma_commit(&s.mma_done[0]);
      wait_or_flag(&s.mma_done[0], 0, p.status);
    }
    __syncwarp();
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------------ O += P V
    if (lane == 0) {
      const uint64_t dv = tc::smem_desc_sw128(smem_addr(s.v[0]), kHalfBytes, kGroupBytes);
      const uint64_t dp = tc::smem_desc_sw128(smem_addr(s.q) + kWeightsAt, 16, 1024);
      bool ok = true;
      uint32_t st = 0, ph = 0;
      uint32_t piece_par = 0, had = 0;  // bits of stream t: the parity of its next piece, whether it had one
      uint32_t few_pieces = 0;          // of stream t, 16 bits each
      for (int it = 0; it < nt; ++it) {
        const int t = it & 1;
        // (P's barrier hands the info on too)
        ok = wait_or_flag(&s.p_full[t], (it >> 1) & 1, p.status) && wait_or_flag(&s.v_full[st], ph, p.status);
        if (!ok) break;
        const volatile UnitInfo& f = s.info[it % kInfos];
        const int pages = (f.keys + kPage - 1) / kPage, flags = f.flags;
        const uint32_t piece = few_pieces >> 16 * t & 0xffffu, buf = piece & 1;
        if (flags & kFirst) {
          if (flags & kFewFlag) {
            if (piece >= 2) ok = wait_or_flag(&s.few_free[t][buf], ((piece >> 1) & 1) ^ 1u, p.status);
          } else {
            if (had >> t & 1) ok = wait_or_flag(&s.o_free[t], (piece_par >> t & 1) ^ 1u, p.status);
            had |= 1u << t;
            piece_par ^= 1u << t;
          }
          if (!ok) break;
        }
        tc::fence_after_sync();
        const uint32_t first = flags & kFirst ? 0u : 1u;
        const uint64_t v = dv + (st * kTileBytes >> 4);
        if (flags & kFewFlag) {  // O^T += V^T P^T
          constexpr uint32_t id = tc::idesc_bf16(128, 2 * kFew, 1, 0);
          const uint64_t w = dp + (t * kWeightBytes >> 4);
          const uint32_t o = tmem + t * kTileKeys + 64 + buf * 2 * kFew;
          tc::mma_ss(o, v, w, id, first);
          if (pages == kTilePages) {
#pragma unroll
            for (int kk = 1; kk < kTilePages; ++kk)
              tc::mma_ss_c<true>(o, v + kk * (kPageBytes >> 4), w + (((kk >> 2) * kWeightHalfBytes + (kk & 3) * 32) >> 4), id);
          } else {
            for (int kk = 1; kk < pages; ++kk)
              tc::mma_ss_c<true>(o, v + kk * (kPageBytes >> 4), w + (((kk >> 2) * kWeightHalfBytes + (kk & 3) * 32) >> 4), id);
          }
        } else {  // O += P V
          constexpr uint32_t id = tc::idesc_bf16(128, 128, 0, 1);
          const uint32_t w = tmem + t * kTileKeys, o = tmem + 256 + t * 128;
          tc::mma_ts(o, w, v, id, first);
          if (pages == kTilePages) {
#pragma unroll
            for (int kk = 1; kk < kTilePages; ++kk) tc::mma_ts_c<true>(o, w + kk * 8, v + kk * (kPageBytes >> 4), id);
          } else {
            for (int kk = 1; kk < pages; ++kk) tc::mma_ts_c<true>(o, w + kk * 8, v + kk * (kPageBytes >> 4), id);
          }
        }
        tc::mma_commit(&s.p_free[t]);
        tc::mma_commit(&s.v_empty[st]);
        if (flags & kLast) {
          tc::mma_commit(flags & kFewFlag ? &s.few_ready[t][buf] : &s.o_ready[t]);
          if (flags & kFewFlag) few_pieces = (few_pieces & ~(0xffffu << 16 * t)) | ((piece + 1) & 0xffffu) << 16 * t;
        }
        if (++st == kStages) {
          st = 0;
          ph ^= 1u;
        }
      }
      tc::mma_commit(&s.mma_done[1]);
      wait_or_flag(&s.mma_done[1], 0, p.status);
    }
    __syncwarp();
  }
  } else {
    // ------------------------------------------------------------------ softmax warps
    tc::regs_increase<kSoftmaxRegs>();
    const int stream = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_bits + stream * kTileKeys, t_o = tmem + lane_bits + 256 + stream * 128;
    bool ok = true;
    int it = stream;
    uint32_t n = 0, pieces = 0;  // units and pieces of this stream so far
    // The next unit's flags; false after the last one or a wait that gave up.
    auto next_flags = [&](int& flags) {
      if (it >= nt) return false;
      ok = warp_wait(&s.info_full[it % kInfos], (it / kInfos) & 1, lane, p.status);
      if (!ok) return false;
      const volatile UnitInfo& f = s.info[it % kInfos];
      flags = f.flags;
      return true;
    };
    // Slots of the unit's last page after its last key may hold anything, NaN too: their V rows meet
    // weights of 0 as zeros.
    auto clear_tail = [&](int keys) {
      const uint32_t vst = static_cast<uint32_t>(it) % kStages;
      ok = warp_wait(&s.v_full[vst], (static_cast<uint32_t>(it) / kStages) & 1, lane, p.status);
      if (!ok) return;
      const int end = (keys + kPage - 1) / kPage * kPage;
      for (int e = keys * 16 + r; e < end * 16; e += 128)  // 16 bytes of a key
        *reinterpret_cast<uint4*>(s.v[vst] + (e >> 7) * kGroupBytes + ((e >> 3) & 1) * kHalfBytes + ((e >> 4) & 7) * 128 +
                                  (e & 7) * 16) = make_uint4(0, 0, 0, 0);
      tc::fence_proxy_async_smem();
    };
    auto hand_over = [&](uint64_t* bar) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    int flags;
    bool more = next_flags(flags);

    // ------------------------------------------------------------------ softmax, a thread per row
    {
      const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
      float m_used = -CUDART_INF_F, l = 0.f;
      for (; more && !(flags & kFewFlag); it += 2, more = next_flags(flags)) {
        const volatile UnitInfo& f = s.info[it % kInfos];
        const int keys = f.keys, rows = f.rows, stats = f.stats;
        float* part = p.tile_parts + f.part + stream * (stats / kHeadDim * kRowFloats);
        const bool used = quarter * 32 < rows;  // some of this warp's rows are query rows
        ok = warp_wait(&s.s_full[stream], n & 1, lane, p.status);
        if (!ok) break;
        ++n;
        tc::fence_after_sync();
        if (flags & kFirst) {
          m_used = -CUDART_INF_F;
          l = 0.f;
        }
        if (used) {
          uint32_t sb[kTileKeys];
          float cm[4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            tc::tmem_ld32_max(t_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(sb + c * 32), cm[c]);
          tc::tmem_wait_ld();
          float mx = fmax3(cm[0], cm[1], fmaxf(cm[2], cm[3]));
          if (keys < kTileKeys) {  // keys past the segment's end (their scores are whatever TMEM held)
            mx = -CUDART_INF_F;
#pragma unroll
            for (int c = 0; c < kTileKeys; ++c) {
              if (c >= keys) sb[c] = 0xff800000u;
              mx = fmaxf(mx, __uint_as_float(sb[c]));
            }
          }
          const float mx2 = mx * p.scale_log2;
          const bool grow = mx2 > m_used + kRescaleThreshold;
          if (__any_sync(0xffffffffu, grow)) {
            const float m_new = grow ? mx2 : m_used;
            const float alpha = m_used == -CUDART_INF_F ? 0.f : fast_exp2(m_used - m_new);
            if (!(flags & kFirst)) {
              // O holds the stream's sum through its last unit: this unit's S was issued after that
              // product had completed
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint32_t o32[32];
                tc::tmem_ld32(t_o + c * 32, o32);
                tc::tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) o32[k] = __float_as_uint(__uint_as_float(o32[k]) * alpha);
                tc::tmem_st32(t_o + c * 32, o32);
              }
            }
            l *= alpha;
            m_used = m_new;
          }
          // The weights go to one bf16 for the product (their sum is of the unrounded ones): off by 2^-8 of each
          // at most, which averages out over the keys: 2.0e-3 of the output's norm against 1.7e-3 for two
          // bf16s as below. Those would cost twice the products and half as many instructions again here: 307
          // rows in 4 groups 85 -> 103 us.
          const float m_eff = m_used == -CUDART_INF_F ? 0.f : m_used;
          const float2 nm2 = make_float2(-m_eff, -m_eff);
          float2 ls[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) ls[k] = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float2 x = fma2(make_float2(__uint_as_float(sb[c * 64 + 2 * k]),
                                                __uint_as_float(sb[c * 64 + 2 * k + 1])), sc2, nm2);
              const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
              ls[k & 3] = add2(ls[k & 3], e);
              pk[k] = pack_bf16x2(e.x, e.y);
            }
            tc::tmem_st32(t_s + c * 32, pk);
          }
          const float2 sum = add2(add2(ls[0], ls[1]), add2(ls[2], ls[3]));
          l += sum.x + sum.y;
          tc::tmem_wait_st();
        }
        if (keys % kPage != 0) clear_tail(keys);
        if (!ok) break;
        hand_over(&s.p_full[stream]);
        if (flags & kLast) {
          ok = warp_wait(&s.o_ready[stream], pieces & 1, lane, p.status);
          if (!ok) break;
          ++pieces;
          tc::fence_after_sync();
          if (used) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tc::tmem_ld32(t_o + c * 32, o);
              tc::tmem_wait_ld();
              if (r < rows) {
                float4* dst = reinterpret_cast<float4*>(part + r * kHeadDim + c * 32);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  dst[k] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                       __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
              }
            }
            // (a NaN among the scores: any finite maximum hands the NaN on)
            if (r < rows) *reinterpret_cast<float2*>(part + stats + 2 * r) = make_float2(l == l ? m_used : 0.f, l);
          }
          hand_over(&s.o_free[stream]);
        }
      }
    }

    // ------------------------------------------------------------------ softmax, a thread per key
    // Lane c of every warp keeps row c's maximum; a row's maximum over the keys takes a reduction in each
    // warp and a meeting of the four, its sum is left in the threads until the piece's end.
    if (ok) {
      float m_used = -CUDART_INF_F;
      float l[kFew];  // this thread's keys' part of each row's sum
      uint32_t meetings = 0;
      // A piece's O is stored after the next unit's weights have been handed over, while its products run;
      // until then: where to, how many rows, and lane c's maximum and sum of row c.
      uint32_t few_pieces = 0;
      bool left = false;
      float* left_part = nullptr;
      int left_stats = 0, left_rows = 0;
      float left_m = 0.f, left_l = 0.f;
      auto store_left = [&] {
        const uint32_t piece = few_pieces - 1, buf = piece & 1;
        left = false;
        ok = warp_wait(&s.few_ready[stream][buf], (piece >> 1) & 1, lane, p.status);
        if (!ok) return;
        tc::fence_after_sync();
        uint32_t o[2 * kFew];
        tc::tmem_ld32(t_s + 64 + buf * 2 * kFew, o);
        tc::tmem_wait_ld();
        hand_over(&s.few_free[stream][buf]);
#pragma unroll
        for (int c = 0; c < kFew; ++c)
          if (c < left_rows) left_part[c * kHeadDim + r] = __uint_as_float(o[c]) + __uint_as_float(o[kFew + c]);
        // (a NaN among the scores: any finite maximum hands the NaN on)
        if (quarter == 0 && lane < left_rows)
          *reinterpret_cast<float2*>(left_part + left_stats + 2 * lane) = make_float2(left_l == left_l ? left_m : 0.f, left_l);
      };
      // all[w][c]: value of lane c of warp w
      auto meet = [&](float (*all)[kFew], float value) {
        if (lane < kFew) all[quarter][lane] = value;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.met[stream]);
        ok = warp_wait(&s.met[stream], meetings & 1, lane, p.status);
        ++meetings;
      };
      for (; more && ok; it += 2, more = ok && next_flags(flags)) {
        const volatile UnitInfo& f = s.info[it % kInfos];
        const int keys = f.keys, rows = f.rows, stats = f.stats;
        float* part = (f.is_tile ? p.tile_parts : p.row_parts) + f.part + stream * (stats / kHeadDim * kRowFloats);
        ok = warp_wait(&s.s_full[stream], n & 1, lane, p.status);
        if (!ok) break;
        ++n;
        tc::fence_after_sync();
        if (flags & kFirst) {
          m_used = -CUDART_INF_F;
#pragma unroll
          for (int c = 0; c < kFew; ++c) l[c] = 0.f;
        }
        uint32_t sb[kFew];
        tc::tmem_ld16(t_s, sb);
        tc::tmem_wait_ld();
        const bool seen = r < keys;
        int best = 0;  // lane c: the warp's largest score of row c, as an integer of the same order
#pragma unroll
        for (int c = 0; c < kFew; ++c) {
          if (c >= rows) break;
          const float x = __uint_as_float(sb[c]);
          int o = __float_as_int(seen && x == x ? x : -CUDART_INF_F);
          o ^= (o >> 31) & 0x7fffffff;
          o = __reduce_max_sync(0xffffffffu, o);
          if (lane == c) best = o;
        }
        best ^= (best >> 31) & 0x7fffffff;
        float (*all)[kFew] = s.exchange[stream][n & 1];
        meet(all, __int_as_float(best));
        if (!ok) break;
        float mx2 = -CUDART_INF_F;
        if (lane < rows)
          mx2 = fmax3(all[0][lane], all[1][lane], fmaxf(all[2][lane], all[3][lane])) * p.scale_log2;
        const bool grow = mx2 > m_used + kRescaleThreshold;
        if (__any_sync(0xffffffffu, grow)) {
          const float m_new = grow ? mx2 : m_used;
          const float alpha = m_used == -CUDART_INF_F ? 0.f : fast_exp2(m_used - m_new);
          m_used = m_new;
          if (!(flags & kFirst)) {
            const uint32_t t_few = t_s + 64 + (few_pieces & 1) * 2 * kFew;
            uint32_t o[2 * kFew];
            tc::tmem_ld32(t_few, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < kFew; ++c) {
              const float a = __shfl_sync(0xffffffffu, alpha, c);
              l[c] *= a;
              o[c] = __float_as_uint(__uint_as_float(o[c]) * a);
              o[kFew + c] = __float_as_uint(__uint_as_float(o[kFew + c]) * a);
            }
            tc::tmem_st32(t_few, o);
            tc::tmem_wait_st();
          }
        }
        const float m_eff = m_used == -CUDART_INF_F ? 0.f : m_used;
        // A weight is two bf16s: its high 16 bits, cut off, and the rest, rounded: 2^-8 of what is below 2^-7 of the
        // weight, so 2^-15 of it at most (one bf16 alone: 2^-8, 2.35e-3 of the output's norm, of which the output's own
        // rounding is 1.66e-3). The rest is taken of a weight 2^-20 larger, so that it is above 0 wherever the weight is:
        // times an infinity of V the two then agree. (Rows four at a time, to overlap their latencies: 2 us of 62 at 8
        // rows over 67,500 keys, which is what the second product had cost. Columns past the rows' are not used.)
        uint8_t* w = s.q + kWeightsAt + stream * kWeightBytes + (r >> 6) * kWeightHalfBytes + (r & 7) * 2;
#pragma unroll
        for (int c = 0; c < kFew; ++c) {
          if (c % 4 == 0 && c >= rows) break;
          const float m = __shfl_sync(0xffffffffu, m_eff, c);
          const float e = seen ? fast_exp2(fmaf(__uint_as_float(sb[c]), p.scale_log2, -m)) : 0.f;
          l[c] += e;
          const float high = __uint_as_float(__float_as_uint(e) & 0xffff0000u), rest = fmaf(e, 1.f + 0x1p-20f, -high);
          uint16_t* to = reinterpret_cast<uint16_t*>(w + c * 128 + ((((r >> 3) & 7) ^ (c & 7)) << 4));
          to[0] = static_cast<uint16_t>(__float_as_uint(e) >> 16);
          to[kFewHalfBytes / 2] = static_cast<uint16_t>(pack_bf16x2(rest, 0.f));
        }
        tc::fence_proxy_async_smem();
        if (keys % kPage != 0) clear_tail(keys);
        if (!ok) break;
        hand_over(&s.p_full[stream]);
        if (left) store_left();
        if (!ok) break;
        if (flags & kLast) {
          // lane c: the warp's sum of row c, then all four warps'
          float sum = 0.f;
#pragma unroll
          for (int c = 0; c < kFew; ++c) {
            if (c >= rows) break;
            float x = l[c];
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
            if (lane == c) sum = x;
          }
          all = s.exchange[stream][2];
          meet(all, sum);
          if (!ok) break;
          left = true;
          left_part = part;
          left_stats = stats;
          left_rows = rows;
          left_m = m_used;
          left_l = lane < kFew ? (all[0][lane] + all[1][lane]) + (all[2][lane] + all[3][lane]) : 0.f;
          ++few_pieces;
        }
      }
      if (ok && left) store_left();
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == kPvWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc<512>(tmem);
  }
}

// ---------------------------------------------------------------------------------------------
// merge: a CTA per row and KV head. Its threads find the row's partial results and weigh them, then its
// warps, half of them per query head, add a part of them each, four dims a lane, eight results' loads in flight.
// (A warp per query head alone, in a CTA per row, took 15 us for 8 rows of 38 results each.)
// The more rows, the fewer warps each: a row is a chain of four latencies however many, and rows that wait
// for an SM add theirs. The whole call with 16, 8 and 2 warps: 8 rows of up to 38 results 59.7, 60.9 and 67.7 us;
// 64 rows 159.7, 156.1 and 155.3; 307 rows 107, 94.7 and 84.9.
// ---------------------------------------------------------------------------------------------
constexpr int kMergeWarpsFewRows = 16;  // up to a CTA per SM
constexpr int kMergeWarps = 8;          // up to four
constexpr int kMergeWarpsManyRows = 2;

template <int kWarps>
__global__ void __launch_bounds__(kWarps * 32) shared_merge_kernel(const SharedParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  constexpr int kMergeThreads = kWarps * 32;
  const int max_parts = 4 * p.slices;  // two sets, two streams, every slice
  float4* stat = reinterpret_cast<float4*>(smem_raw);  // (m, l) of the row's two query heads
  const float** where = reinterpret_cast<const float**>(stat + max_parts);  // O of the first; the second's follows
  __shared__ float4 sums[kWarps][32];
  const int b = static_cast<int>(blockIdx.x) / p.hkv, head = static_cast<int>(blockIdx.x) % p.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  await_previous();
  const uint32_t n = static_cast<uint32_t>(p.slices), U = static_cast<uint32_t>(p.slice->units);
  const RowPlan row = p.rows[b];
  const Divider over(U, n);
  // slices [i0, i1] hold a set: slice i has units [U i / n, U (i + 1) / n)
  int i0[2] = {0, 0}, count[2] = {0, 0};
#pragma unroll
  for (int set = 0; set < 2; ++set) {
    const int unit = set == 0 ? row.tile_unit : row.own_unit, units = set == 0 ? row.tile_units : row.own_units;
    if (units == 0) continue;
    i0[set] = over((static_cast<uint64_t>(unit) + 1) * n - 1, U);
    count[set] = 2 * (over(static_cast<uint64_t>(unit + units) * n - 1, U) - i0[set] + 1);
  }
  const int total = count[0] + count[1];
  for (int c = tid; c < total; c += kMergeThreads) {
    const int set = c < count[0] ? 0 : 1, at = set == 0 ? c : c - count[0];
    const int i = (set == 0 ? i0[0] : i0[1]) + (at >> 1), stream = at & 1;
    const int unit = set == 0 ? row.tile_unit : row.own_unit, units = set == 0 ? row.tile_units : row.own_units;
    const int rows = set == 0 ? row.tile_rows : 1, r = set == 0 ? 2 * row.in_tile : 0;
    const int first = over(static_cast<uint64_t>(U) * i, n), end = over(static_cast<uint64_t>(U) * (i + 1), n);
    const int u0 = max(first, unit), u1 = min(end, unit + units);
    // units alternate between the streams, from the slice's first
    const bool there = u1 - u0 >= 2 || (u1 - u0 == 1 && ((u0 - first) & 1) == stream);
    const int from = set == 0 ? i * p.tile_rows + row.tile : i + row.own;
    const float* part = (set == 0 ? p.tile_parts : p.row_parts) +
                        (static_cast<int64_t>(from) * p.hkv + head * rows) * kPartFloats + stream * 2 * rows * kRowFloats;
    where[c] = there ? part + r * kHeadDim : nullptr;
    stat[c] = there ? *reinterpret_cast<const float4*>(part + 2 * rows * kHeadDim + 2 * r)
                    : make_float4(-CUDART_INF_F, 0.f, -CUDART_INF_F, 0.f);
  }
  __syncthreads();
  // each warp on its own: its first results' loads go out, then the row's maximum and sum over all results
  const int h = warp & 1;
  constexpr int kStride = kWarps / 2;
  float4 v[8];
  auto load = [&](int c0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + j * kStride;
      v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < total && where[c] != nullptr) v[j] = reinterpret_cast<const float4*>(where[c] + h * kHeadDim)[lane];
    }
  };
  load(warp >> 1);
  float top = -CUDART_INF_F, l = 0.f;
  for (int c = lane; c < total; c += 32) top = fmaxf(top, h == 0 ? stat[c].x : stat[c].z);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  auto weight = [&](int c) {
    const float m = h == 0 ? stat[c].x : stat[c].z;
    return m == -CUDART_INF_F ? 0.f : fast_exp2(m - top);
  };
  for (int c = lane; c < total; c += 32) l += weight(c) * (h == 0 ? stat[c].y : stat[c].w);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = warp >> 1; c0 < total; c0 += 8 * kStride) {
    if (c0 >= 8 * kStride) load(c0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + j * kStride;
      const float w = c < total ? weight(c) : 0.f;
      acc.x += w * v[j].x;
      acc.y += w * v[j].y;
      acc.z += w * v[j].z;
      acc.w += w * v[j].w;
    }
  }
  sums[warp][lane] = acc;
  __syncthreads();
  if (warp >= 2) return;
#pragma unroll
  for (int w = 1; w < kStride; ++w) {
    const float4 o = sums[2 * w + h][lane];
    acc.x += o.x;
    acc.y += o.y;
    acc.z += o.z;
    acc.w += o.w;
  }
  const float inv = 1.0f / l;
  uint2 out = make_uint2(0u, 0u);
  if (top != -CUDART_INF_F) {
    out.x = pack_bf16x2(acc.x * inv, acc.y * inv);
    out.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  }
  const int64_t at = static_cast<int64_t>(b) * p.hq + 2 * head + h;
  reinterpret_cast<uint2*>(p.out + at * kHeadDim)[lane] = out;
  if (lane == 0 && p.lse != nullptr) p.lse[at] = top == -CUDART_INF_F ? -CUDART_INF_F : (top + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------------
struct SharedLayout {
  int slices, tile_rows;
  bool own_plan;
  size_t slice, segments, own_segments, rows, tile_parts, row_parts, total;
};

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

bool shared_layout(SharedLayout& l, int hkv, int batch, int groups, int max_group_rows) {
  const int sms = sm_count_current_device();
  if (sms <= 0) return false;
  l.slices = std::min(kMaxSlices, std::max(1, sms / hkv));
  l.tile_rows = std::max(1, std::min({kTileRows, max_group_rows, batch}));
  // a group's segments: one, and one more for every kTileRows rows
  const size_t tiles = groups > 0 ? static_cast<size_t>(groups) + batch / kTileRows : 0;
  l.slice = 0;
  l.segments = align256(sizeof(Slice) * l.slices);
  l.own_plan = tiles + batch <= kOwnPlanSegments;
  l.own_segments = align256(l.segments + (l.own_plan ? 0 : sizeof(Segment) * (tiles + batch)));
  l.rows = align256(l.own_segments + (l.own_plan ? sizeof(Segment) * kOwnPlanSegments * l.slices * hkv : 0));
  l.tile_parts = align256(l.rows + sizeof(RowPlan) * batch);
  const size_t per_row = static_cast<size_t>(hkv) * kPartFloats * sizeof(float), slices = static_cast<size_t>(l.slices);
  l.row_parts = align256(l.tile_parts + (groups > 0 ? (slices * l.tile_rows + 2 * static_cast<size_t>(batch)) * per_row : 0));
  l.total = align256(l.row_parts + (slices + batch) * per_row);
  return true;
}

bool shared_sizes_valid(int batch, int groups, int max_group_rows) {
  return batch >= 0 && groups >= 0 && max_group_rows >= 0;
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_decode_shared_workspace_size(pa_dims dims, int32_t batch, int32_t groups,
                                                  int32_t max_group_rows) {
  using namespace pa;
  SharedLayout l;
  if (!gqa_dims_supported(dims) || !shared_sizes_valid(batch, groups, max_group_rows) || batch == 0 ||
      batch > kMaxBatch || groups > kMaxGroups || !shared_layout(l, dims.num_kv_heads, batch, groups, max_group_rows))
    return 0;
  return l.total;
}

extern "C" pa_status attn_decode_paged_shared(pa_dims dims, const void* q, const void* k_pool, const void* v_pool,
                                              int64_t num_pages, const int32_t* block_table, int32_t bt_stride,
                                              const int32_t* seq_lens, int32_t batch, const int32_t* cu_group_rows,
                                              const int32_t* shared_pages, int32_t groups, int32_t max_group_rows,
                                              int32_t max_seq_len, float softmax_scale, void* out, float* lse,
                                              void* workspace, size_t workspace_bytes, int32_t* status,
                                              pa_stream_t stream) {
  using namespace pa;
  if (!gqa_dims_supported(dims)) return PA_ERR_UNSUPPORTED;
  if (!shared_sizes_valid(batch, groups, max_group_rows) || num_pages <= 0 || bt_stride <= 0 ||
      bt_stride > 0x7fffffff / kPage || max_seq_len < 0 || max_seq_len > kMaxKeys ||
      !(softmax_scale > 0.f && softmax_scale < 1e30f))
    return PA_ERR_INVALID_ARG;
  if (batch > kMaxBatch || groups > kMaxGroups) {
    snprintf_error("attn_decode_paged_shared: at most %d rows and %d groups per call", kMaxBatch, kMaxGroups);
    return PA_ERR_UNSUPPORTED;
  }
  if (num_pages * kPage >= (int64_t(1) << 31)) return PA_ERR_UNSUPPORTED;
  if (batch == 0) return PA_OK;
  if (!q || !k_pool || !v_pool || !block_table || !seq_lens || !out || (groups > 0 && (!cu_group_rows || !shared_pages)))
    return PA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_pool) | reinterpret_cast<uintptr_t>(v_pool) |
       reinterpret_cast<uintptr_t>(out)) & 15u)
    return PA_ERR_INVALID_ARG;
  SharedLayout l;
  const int hkv = dims.num_kv_heads;
  if (!shared_layout(l, hkv, batch, groups, max_group_rows)) return PA_ERR_CUDA;
  if (workspace == nullptr || workspace_bytes < l.total) return PA_ERR_WORKSPACE_TOO_SMALL;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PA_ERR_INVALID_ARG;
  CUtensorMap qm, km, vm;
  if (!make_map_heads(&qm, q, static_cast<uint64_t>(batch), dims.num_q_heads, kGroup, kQBoxRows) ||
      !make_map_pages(&km, k_pool, static_cast<uint64_t>(num_pages), hkv) ||
      !make_map_pages(&vm, v_pool, static_cast<uint64_t>(num_pages), hkv)) {
    snprintf_error("cuTensorMapEncodeTiled failed for the decode's operands");
    return PA_ERR_CUDA;
  }
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    cudaError_t e = cudaFuncSetAttribute(shared_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(sizeof(PlanOfAll)));
    // same carveout for the merge: no reconfiguration between them
    for (auto* kernel : {&shared_merge_kernel<kMergeWarpsFewRows>, &shared_merge_kernel<kMergeWarps>,
                         &shared_merge_kernel<kMergeWarpsManyRows>})
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    for (auto* kernel : {&shared_attention_kernel<false>, &shared_attention_kernel<true>}) {
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(SharedSmem)));
      cudaFuncAttributes fa;
      if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kernel);
      if (e == cudaSuccess && fa.numRegs < kLaunchRegs) {  // (setmaxnreg.inc would wait forever)
        snprintf_error("shared_attention_kernel built with %d registers/thread, needs %d for its split", fa.numRegs,
                       kLaunchRegs);
        return PA_ERR_UNSUPPORTED;
      }
    }
    if (e != cudaSuccess) return record_cuda_error(e, "cudaFuncSetAttribute(decode_shared)");
    configured_device = dev;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SharedParams p;
  p.hkv = hkv;
  p.hq = dims.num_q_heads;
  p.batch = batch;
  p.groups = groups;
  p.max_group_rows = max_group_rows;
  p.bt_stride = bt_stride;
  p.max_seq_len = max_seq_len;
  p.seq_lens = seq_lens;
  p.block_table = block_table;
  p.cu_group_rows = cu_group_rows;
  p.shared_pages = shared_pages;
  p.num_pages = num_pages;
  p.scale_log2 = softmax_scale * kLog2e;
  p.slices = l.slices;
  p.tile_rows = l.tile_rows;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.status = status;
  p.slice = reinterpret_cast<Slice*>(ws + l.slice);
  p.segments = reinterpret_cast<Segment*>(ws + l.segments);
  p.own_segments = reinterpret_cast<Segment*>(ws + l.own_segments);
  p.rows = reinterpret_cast<RowPlan*>(ws + l.rows);
  p.tile_parts = reinterpret_cast<float*>(ws + l.tile_parts);
  p.row_parts = reinterpret_cast<float*>(ws + l.row_parts);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(l.slices * hkv);
  cudaError_t e = cudaSuccess;
  if (l.own_plan) {
    e = launch_dependent(shared_attention_kernel<true>, grid, kThreads, sizeof(SharedSmem), st, 0, qm, km, vm, p);
  } else {
    // a thread per row, group and slice, in whole warps
    const unsigned plan_threads = static_cast<unsigned>(
        std::min(kPlanThreads, (std::max({static_cast<int>(batch), static_cast<int>(groups), l.slices}) + 31) / 32 * 32));
    e = launch_dependent(shared_plan_kernel, 1, plan_threads, sizeof(PlanOfAll), st, 0, p);
    if (e == cudaSuccess)
      e = launch_dependent(shared_attention_kernel<false>, grid, kThreads, sizeof(SharedSmem), st, 0, qm, km, vm, p);
  }
  if (e == cudaSuccess) {
    const size_t smem = static_cast<size_t>(4 * l.slices) * (sizeof(float4) + sizeof(const float*));
    const unsigned ctas = static_cast<unsigned>(batch * hkv);
    auto merge = [&](auto* kernel, int warps) { return launch_dependent(kernel, ctas, 32 * warps, smem, st, 0, p); };
    // the widest whose CTAs all run at once
    e = batch <= l.slices       ? merge(shared_merge_kernel<kMergeWarpsFewRows>, kMergeWarpsFewRows)
        : batch <= 4 * l.slices ? merge(shared_merge_kernel<kMergeWarps>, kMergeWarps)
                                : merge(shared_merge_kernel<kMergeWarpsManyRows>, kMergeWarpsManyRows);
  }
  return e == cudaSuccess ? PA_OK : record_cuda_error(e, "attn_decode_paged_shared");
}
