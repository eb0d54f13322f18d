// paged_fork / paged_copy_pages: the paged cache follows the beams of a search (sm_103a).
//
// A group is W rows of the block table (one request's beams). After a selection, row b of the group
// continues the transcript of row parents[b], so it takes over that row's pages. Pages are shared, not
// copied: within a group a page may be in several rows' tables, and those tables are its reference
// count. Logical page j of all the group's rows is decided by one thread, which sees every holder at
// once, so nothing is counted in memory, no atomics order anything, and tables can change in place:
//   - a row without children gives a page back when no row with children, and no earlier row without,
//     holds it;
//   - the partly filled last page of a child is written by its next token, so all its holders but the
//     first child get a page of their own, and the copy is ordered in copies[];
//   - the leading pages that all rows in use have in common, and fill, are counted for the attention.
//
// Bound by latency and, in large batches, by the table's bytes. Two launches: the first counts what
// each block of pages gives back and each group copies, and saves what the second overwrites (lengths,
// the end of the free list); the second sums the counts before its own, and changes the tables, the
// list and the lengths. If anything is wrong (a parent outside the group, a length past the table,
// too few free pages) it changes nothing: that has to be known before the first store, hence two.
// Measured on a GB300 (calls of a graph that also restore the table and the list by two copies): 4 rows of
// 1,000 tokens 12 us, 512 rows of 2,000 to 67,500 tokens 22 us: each launch is a chain of loads (group and page
// entries, counts, the end of the list).
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
constexpr int kMaxRows = 4096;
constexpr int kNone = 0x7fffffff;
// Blocks of pages per call that the second launch sums over, at most about this many.
constexpr int kMaxBlocks = 2048;

struct ForkParams {
  const int32_t* parents;
  const int32_t* seq_lens;
  int32_t groups, beams;
  int32_t* block_table;
  int32_t bt_stride;
  int32_t* free_pages;
  int32_t free_capacity;
  const int32_t* free_count;
  int64_t num_pages;
  int32_t* free_count_out;
  int32_t* seq_lens_out;
  int32_t* copies;
  int32_t* shared_pages;
  int32_t* status;
  int32_t blocks, span;  // page blocks per group, and pages in each (a multiple of kThreads)
  // workspace
  int32_t* freed;    // [groups][blocks] pages that a block gives back; -1: nothing in it changes
  int32_t* differ;   // [groups][blocks] its first page that the rows do not have in common
  int32_t* copied;   // [groups] copies; -1: the group's parents or lengths are not valid
  int32_t* copy_of;  // [rows] the page that the row's last page is copied from, or -1
  int32_t* old_lens; // [rows]
  int32_t* tail;     // [rows] the free list from its end
  int32_t* count;    // the free count as used
};

// What a CTA needs to know of its group.
struct Group {
  int32_t parent[kMaxBeams];  // -1: the row becomes empty
  int32_t old_len[kMaxBeams], len[kMaxBeams];
  int32_t old_pages[kMaxBeams], pages[kMaxBeams];
  uint32_t has_child[2];      // rows that some child continues
  uint32_t live[2];           // children that are not empty
  int32_t max_pages[2];       // of the old rows, by half
};

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kPage - 1) / kPage; }
__device__ __forceinline__ bool bit(const uint32_t (&m)[2], int i) { return m[i >> 5] >> (i & 31) & 1; }

// The group from this thread's row of it (rows are the first threads'); false if a parent or a length is
// not valid. Every thread of the CTA takes part.
__device__ __forceinline__ bool make_group(const ForkParams& p, int parent, int len, Group& s) {
  const int W = p.beams, t = threadIdx.x;
  const bool mine = t < W;
  if (mine) {
    s.parent[t] = parent;
    s.old_len[t] = len;
  }
  const bool bad = mine && (parent < -1 || parent >= W || len < 0 || len > p.bt_stride * kPage);
  if (__syncthreads_or(bad)) return false;
  if (t < 64) {
    bool child = false;
    for (int b = 0; b < W; ++b) child |= mine && s.parent[b] == t;
    const int now = mine && parent >= 0 ? s.old_len[parent] : 0;
    if (mine) {
      s.len[t] = now;
      s.old_pages[t] = pages_of(len);
      s.pages[t] = pages_of(now);
    }
    const uint32_t children = __ballot_sync(0xffffffffu, child), live = __ballot_sync(0xffffffffu, now > 0);
    const int pages = __reduce_max_sync(0xffffffffu, mine ? pages_of(len) : 0);
    if ((t & 31) == 0) {
      s.has_child[t >> 5] = children;
      s.live[t >> 5] = live;
      s.max_pages[t >> 5] = pages;
    }
  }
  __syncthreads();
  return true;
}

// Logical page j of the group's rows, read into this thread's column of `col`.
__device__ __forceinline__ void read_column(const ForkParams& p, const int32_t* rows, int j, int32_t* col) {
#pragma unroll 8
  for (int r = 0; r < p.beams; ++r)
    col[r * kThreads] = j < p.bt_stride ? rows[static_cast<int64_t>(r) * p.bt_stride + j] : -1;
}

// What logical page j of the group's rows comes to.
struct Verdict {
  uint64_t gives;  // rows without children that give their page back: no row with a child holds it, and no
                   // earlier row (it may lie outside the pool: it is then flagged and goes nowhere)
  bool common;     // the rows in use have it in common, filled
  bool changes;    // some entry may change (a partly filled last page may be copied)
};

// Up to 8 rows, unrolled: entries in registers, one round of shared-memory reads, pairs as bits. (The loops
// below took 5 us for 8 rows, one read waiting for the other.)
constexpr int kFewBeams = 8;

__device__ __forceinline__ Verdict judge_few(const ForkParams& p, const Group& s, const int32_t* col, int j) {
  int32_t e[kFewBeams], now[kFewBeams];
  uint32_t held = 0, holds = 0, live = 0, same = 0;  // holds: after the fork; same: the entry stays
  bool common = true;
#pragma unroll
  for (int b = 0; b < kFewBeams; ++b) {
    const bool mine = b < p.beams;
    e[b] = mine ? col[b * kThreads] : -1;
    now[b] = mine ? col[max(s.parent[b], 0) * kThreads] : -1;
    if (mine && j < s.old_pages[b]) held |= 1u << b;
    if (mine && j < s.pages[b]) holds |= 1u << b;
    if (mine && s.len[b] > 0) live |= 1u << b;
    if (mine && j < s.len[b] / kPage && now[b] >= 0) same |= 1u << b;  // (filled, for now)
  }
  common = live != 0 && (same & live) == live;
  const int32_t one = live != 0 ? __ffs(live) - 1 : 0;
  int32_t first = -1;
#pragma unroll
  for (int b = 0; b < kFewBeams; ++b)
    if (b == one) first = now[b];
  uint32_t moved = held ^ holds, gives = 0;
#pragma unroll
  for (int b = 0; b < kFewBeams; ++b) {
    common &= !(live >> b & 1) || now[b] == first;
    // filled entries that stay do not change; a partly filled one may be copied
    if ((holds >> b & 1) && (e[b] != now[b] || !(j < s.len[b] / kPage))) moved |= 1u << b;
    uint32_t equal = 0;
#pragma unroll
    for (int o = 0; o < kFewBeams; ++o)
      if (o != b && e[o] == e[b]) equal |= 1u << o;
    if ((held >> b & 1) && e[b] >= 0 && (equal & held & (s.has_child[0] | ((1u << b) - 1u))) == 0) gives |= 1u << b;
  }
  return Verdict{gives & ~s.has_child[0], common, moved != 0};
}

__device__ __forceinline__ Verdict judge_many(const ForkParams& p, const Group& s, const int32_t* col, int j) {
  Verdict v{0, true, false};
  int32_t one = -1;
  for (int b = 0; b < p.beams; ++b) {
    const int len = s.len[b];
    const bool held = j < s.old_pages[b];
    if (len == 0) {
      v.changes |= held;
      continue;
    }
    const int32_t e = col[s.parent[b] * kThreads];
    if (one < 0) one = e;
    v.common &= e >= 0 && e == one && j < len / kPage;
    v.changes |= j < s.pages[b] ? e != col[b * kThreads] || j >= len / kPage : held;
  }
  v.common &= one >= 0;
  for (int r = 0; v.changes && r < p.beams; ++r) {
    const int32_t e = col[r * kThreads];
    if (bit(s.has_child, r) || j >= s.old_pages[r] || e < 0) continue;
    bool kept = false;
    for (int o = 0; o < p.beams && !kept; ++o)
      kept = o != r && (o < r || bit(s.has_child, o)) && col[o * kThreads] == e && j < s.old_pages[o];
    if (!kept) v.gives |= 1ull << r;
  }
  return v;
}

__device__ __forceinline__ Verdict judge(const ForkParams& p, const Group& s, const int32_t* col, int j) {
  return p.beams <= kFewBeams ? judge_few(p, s, col, j) : judge_many(p, s, col, j);
}

// Sums of n values over the CTA.
template <int n>
__device__ __forceinline__ void block_sums(int (&v)[n], int32_t (*scratch)[kWarps]) {
#pragma unroll
  for (int k = 0; k < n; ++k) {
    v[k] = __reduce_add_sync(0xffffffffu, v[k]);
    if ((threadIdx.x & 31) == 0) scratch[k][threadIdx.x >> 5] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < n; ++k) {
    v[k] = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v[k] += scratch[k][w];
  }
}

__global__ void __launch_bounds__(kThreads) fork_count_kernel(const ForkParams p) {
  extern __shared__ int32_t columns[];  // [beams][kThreads]
  __shared__ Group s;
  __shared__ int32_t scratch[3][kWarps], first;
  const int tid = threadIdx.x, W = p.beams;
  const int g = static_cast<int>(blockIdx.y), block = static_cast<int>(blockIdx.x), at = g * p.blocks + block;
  int32_t* col = columns + tid;
  int32_t* rows = p.block_table + static_cast<int64_t>(g) * W * p.bt_stride;
  const int j0 = block * p.span;
  if (tid == 0) first = kNone;
  launch_next();
  await_previous();
  // everything that does not depend on anything is asked for first
  const int i = g * W + tid;
  const int parent = tid < W ? p.parents[i] : 0, len = tid < W ? p.seq_lens[i] : 0;
  int count = block == 0 ? *p.free_count : 0;
  read_column(p, rows, j0 + tid, col);
  // the end of the free list, from which copies take their pages, and the lengths: both may be
  // overwritten by the second launch
  if (block == 0) {
    if (count < 0 || count > p.free_capacity) {
      if (g == 0 && tid == 0) flag_error(p.status, PA_DEV_ERR_LENGTH);
      count = count < 0 ? 0 : p.free_capacity;
    }
    if (g == 0 && tid == 0) *p.count = count;
    if (tid < W) {
      p.old_lens[i] = len;
      p.tail[i] = i < count ? p.free_pages[count - 1 - i] : -1;
    }
  }
  const bool good = make_group(p, parent, len, s);
  int sums[3] = {0, 0, 0};  // pages given back, entries that change, copies
  int32_t from = -1;
  if (good) {
    const int end = min(j0 + p.span, max(s.max_pages[0], s.max_pages[1]));
    for (int j = j0 + tid; j < end; j += kThreads) {
      if (j >= j0 + kThreads) read_column(p, rows, j, col);
      const Verdict v = judge(p, s, col, j);
      if (!v.common) atomicMin(&first, j);
      if (!v.changes) continue;
      sums[1] = 1;
      for (uint64_t m = v.gives; m != 0; m &= m - 1) {
        if (col[(__ffsll(static_cast<long long>(m)) - 1) * kThreads] < p.num_pages) ++sums[0];
        else flag_error(p.status, PA_DEV_ERR_PAGE_OOB);
      }
    }
    // the children whose last page is copied: partly filled, and held by another child that comes
    // first or has it filled
    if (block == 0 && tid < W && s.len[tid] % kPage != 0) {
      const int last = s.len[tid] / kPage;
      const int32_t e = rows[static_cast<int64_t>(s.parent[tid]) * p.bt_stride + last];
      if (e < 0 || e >= p.num_pages) {
        flag_error(p.status, PA_DEV_ERR_PAGE_OOB);
      } else {
#pragma unroll 4
        for (int b = 0; b < W; ++b)
          if (b != tid && last < pages_of(s.len[b]) && (b < tid || s.len[b] >= (last + 1) * kPage) &&
              rows[static_cast<int64_t>(s.parent[b]) * p.bt_stride + last] == e)
            from = e;
      }
    }
  }
  if (block == 0 && tid < W) p.copy_of[i] = from;
  sums[2] = from >= 0 ? 1 : 0;
  block_sums(sums, scratch);
  if (tid == 0) {
    p.freed[at] = sums[1] != 0 ? sums[0] : -1;
    p.differ[at] = first;
    if (block == 0) p.copied[g] = good ? sums[2] : -1;
  }
}

__global__ void __launch_bounds__(kThreads) fork_apply_kernel(const ForkParams p) {
  extern __shared__ int32_t columns[];
  __shared__ Group s;
  __shared__ int32_t scratch[5][kWarps], fresh[kMaxBeams], warp_freed[kWarps], differs[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = p.beams;
  const int g = static_cast<int>(blockIdx.y), block = static_cast<int>(blockIdx.x), at = g * p.blocks + block;
  int32_t* rows = p.block_table + static_cast<int64_t>(g) * W * p.bt_stride;
  int32_t* col = columns + tid;
  const int j0 = block * p.span, i = g * W + tid;
  await_previous();
  const bool still = p.freed[at] < 0;  // nothing in this block changes
  if (block != 0 && still) return;
  const int parent = tid < W ? p.parents[i] : 0, len = tid < W ? p.old_lens[i] : 0;
  const int from = tid < W ? p.copy_of[i] : -1, count = *p.count;
  // counts before this block, and of all
  int sums[5] = {0, 0, 0, 0, 0};  // given back: before, all; copies: before, all; groups that are not valid
  for (int k = tid; k < p.groups * p.blocks; k += kThreads) {
    const int n = max(p.freed[k], 0);
    sums[1] += n;
    if (k < at) sums[0] += n;
  }
  for (int k = tid; k < p.groups; k += kThreads) {
    const int n = p.copied[k];
    if (n < 0) sums[4] = 1;
    sums[3] += max(n, 0);
    if (k < g) sums[2] += max(n, 0);
  }
  int differ = kNone;
  if (block == 0)
    for (int k = tid; k < p.blocks; k += kThreads) differ = min(differ, p.differ[g * p.blocks + k]);
  block_sums(sums, scratch);
  const int before = sums[0], freed = sums[1], copies_before = sums[2], copies = sums[3];
  const bool bad = sums[4] != 0, short_of = !bad && copies > count;
  const bool full = static_cast<int64_t>(count) - copies + freed > p.free_capacity;
  if (at == 0 && tid == 0) {
    if (bad || full) flag_error(p.status, PA_DEV_ERR_LENGTH);
    if (short_of) flag_error(p.status, PA_DEV_ERR_NO_PAGES);
    *p.free_count_out = bad || full || short_of ? count : count - copies + freed;
  }
  if (bad || full || short_of) {  // nothing changes
    if (block == 0 && tid < W) {
      p.seq_lens_out[i] = len;
      p.copies[3 * i] = p.copies[3 * i + 1] = -1;
      p.copies[3 * i + 2] = 0;
    }
    if (block == 0 && tid == 0) p.shared_pages[g] = 0;
    return;
  }
  // the pages that the group's copies get: the list's last ones, in row order
  if (tid < W) fresh[tid] = from;
  make_group(p, parent, len, s);
  int32_t page = kNone;
  if (tid < W && from >= 0) {
    int k = copies_before;
    for (int b = 0; b < tid; ++b) k += fresh[b] >= 0 ? 1 : 0;
    page = p.tail[k];
  }
  __syncthreads();
  if (tid < W) fresh[tid] = page;
  if (block == 0) {
    if (tid < W && s.len[tid] > 0) differ = min(differ, s.len[tid] / kPage);
    differ = __reduce_min_sync(0xffffffffu, differ);
    if (lane == 0) differs[warp] = differ;
  }
  __syncthreads();
  if (block == 0) {
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) differ = min(differ, differs[w]);
      p.shared_pages[g] = (s.live[0] | s.live[1]) == 0 ? 0 : differ;
    }
    if (tid < W) {
      p.seq_lens_out[i] = s.len[tid];
      int32_t src = -1, dst = -1, n = 0;
      if (page != kNone) {
        if (page < 0 || page >= p.num_pages) {
          flag_error(p.status, PA_DEV_ERR_PAGE_OOB);
        } else {
          src = from;
          dst = page;
          n = s.len[tid] % kPage;
        }
      }
      p.copies[3 * i] = src;
      p.copies[3 * i + 1] = dst;
      p.copies[3 * i + 2] = n;
    }
    if (still) return;
  }
  int to0 = count - copies + before;
  const int j1 = min(j0 + p.span, max(s.max_pages[0], s.max_pages[1]));
  for (int jb = j0; jb < j1; jb += kThreads) {
    const int j = jb + tid;
    int n = 0;
    Verdict v{0, true, false};
    if (j < j1) {
      read_column(p, rows, j, col);
      v = judge(p, s, col, j);
      if (!v.changes) v.gives = 0;
      for (uint64_t m = v.gives; m != 0; m &= m - 1) {
        const int r = __ffsll(static_cast<long long>(m)) - 1;
        if (col[r * kThreads] < p.num_pages) ++n;
        else v.gives &= ~(1ull << r);
      }
    }
    // places of the pages given back: by page, then row
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_freed[warp] = incl;
    __syncthreads();
    int to = to0 + incl - n;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) to += warp_freed[w];
      to0 += warp_freed[w];
    }
    __syncthreads();
    if (!v.changes) continue;
    for (uint64_t m = v.gives; m != 0; m &= m - 1)
      p.free_pages[to++] = col[(__ffsll(static_cast<long long>(m)) - 1) * kThreads];
#pragma unroll 8
    for (int b = 0; b < W; ++b) {
      const int32_t e = col[b * kThreads];
      int32_t now = e;
      if (j < s.pages[b])
        now = fresh[b] != kNone && j == s.len[b] / kPage ? fresh[b] : col[s.parent[b] * kThreads];
      else if (j < s.old_pages[b])
        now = -1;
      if (now != e) rows[static_cast<int64_t>(b) * p.bt_stride + j] = now;
    }
  }
}

// ---------------------------------------------------------------------------------------------
// paged_copy_pages: the first n tokens of a page, 16 bytes a thread and load, for every row of
// copies[] and every pool: a CTA per pair. Bound by HBM (each byte read once and written once): 512 rows,
// half of them copied, in 56 pools, 503 MB in 76.4 us (6.6 TB/s, 0.97 of a copy's rate); 3 pages 2.9 us.
// ---------------------------------------------------------------------------------------------
constexpr int kPoolsPerLaunch = 128;

struct CopyParams {
  const int32_t* copies;
  int64_t num_pages;
  int32_t vectors;  // 16-byte units of a token in a pool
  int32_t* status;
  uint4* pools[kPoolsPerLaunch];
};

__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const __grid_constant__ CopyParams p) {
  await_previous();
  const int row = static_cast<int>(blockIdx.x);
  const int src = p.copies[3 * row], dst = p.copies[3 * row + 1], tokens = p.copies[3 * row + 2];
  if (src < 0 && tokens == 0) return;  // no copy
  if (src < 0 || dst < 0 || src >= p.num_pages || dst >= p.num_pages || tokens < 0 || tokens > kPage) {
    if (blockIdx.y == 0 && threadIdx.x == 0)
      flag_error(p.status, tokens < 0 || tokens > kPage ? PA_DEV_ERR_LENGTH : PA_DEV_ERR_PAGE_OOB);
    return;
  }
  if (src == dst) return;
  uint4* pool = p.pools[blockIdx.y];
  const uint4* from = pool + static_cast<int64_t>(src) * kPage * p.vectors;
  uint4* to = pool + static_cast<int64_t>(dst) * kPage * p.vectors;
  const int n = tokens * p.vectors;  // at most 2,048
  uint4 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (threadIdx.x + k * kThreads < n) v[k] = from[threadIdx.x + k * kThreads];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (threadIdx.x + k * kThreads < n) to[threadIdx.x + k * kThreads] = v[k];
}

struct ForkLayout {
  int blocks, span;
  size_t freed, differ, copied, copy_of, old_lens, tail, count, total;
};

ForkLayout fork_layout(int32_t groups, int32_t beams, int32_t bt_stride) {
  ForkLayout l;
  const int64_t units = (static_cast<int64_t>(bt_stride) + kThreads - 1) / kThreads;
  // pages of a block: kThreads, or as many more as keep the blocks of all groups near kMaxBlocks
  const int64_t per = std::max<int64_t>(1, std::min(units, units * groups / kMaxBlocks));
  l.span = static_cast<int>(per) * kThreads;
  l.blocks = static_cast<int>((units + per - 1) / per);
  const size_t rows = static_cast<size_t>(groups) * beams, all = static_cast<size_t>(groups) * l.blocks;
  l.freed = 0;
  l.differ = l.freed + all;
  l.copied = l.differ + all;
  l.copy_of = l.copied + groups;
  l.old_lens = l.copy_of + rows;
  l.tail = l.old_lens + rows;
  l.count = l.tail + rows;
  l.total = (l.count + 1) * sizeof(int32_t);
  return l;
}

bool fork_sizes_valid(int32_t groups, int32_t beams, int32_t bt_stride) {
  return groups >= 0 && beams > 0 && bt_stride > 0 && bt_stride <= 0x7fffffff / kPage;
}

bool fork_sizes_supported(int32_t groups, int32_t beams) {
  return beams <= kMaxBeams && static_cast<int64_t>(groups) * beams <= kMaxRows;
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_fork_workspace_size(int32_t groups, int32_t beams, int32_t bt_stride) {
  using namespace pa;
  if (!fork_sizes_valid(groups, beams, bt_stride) || !fork_sizes_supported(groups, beams)) return 0;
  return (fork_layout(groups, beams, bt_stride).total + 255) / 256 * 256;
}

extern "C" pa_status paged_fork(const int32_t* parents, const int32_t* seq_lens, int32_t groups, int32_t beams,
                                int32_t* block_table, int32_t bt_stride, int32_t* free_pages,
                                int32_t free_capacity, const int32_t* free_count, int64_t num_pages,
                                int32_t* free_count_out, int32_t* seq_lens_out, int32_t* copies,
                                int32_t* shared_pages, void* workspace, size_t workspace_bytes, int32_t* status,
                                pa_stream_t stream) {
  using namespace pa;
  if (!fork_sizes_valid(groups, beams, bt_stride) || free_capacity < 0 || num_pages <= 0) return PA_ERR_INVALID_ARG;
  if (!fork_sizes_supported(groups, beams)) {
    snprintf_error("paged_fork: at most %d rows in a group and %d rows per call", kMaxBeams, kMaxRows);
    return PA_ERR_UNSUPPORTED;
  }
  if (!free_count || !free_count_out || (free_capacity > 0 && !free_pages)) return PA_ERR_INVALID_ARG;
  if (groups > 0 && (!parents || !seq_lens || !block_table || !seq_lens_out || !copies || !shared_pages))
    return PA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (groups == 0) {
    if (free_count_out == free_count) return PA_OK;
    const cudaError_t e = cudaMemcpyAsync(free_count_out, free_count, sizeof(int32_t), cudaMemcpyDeviceToDevice, st);
    return e == cudaSuccess ? PA_OK : record_cuda_error(e, "paged_fork");
  }
  const ForkLayout l = fork_layout(groups, beams, bt_stride);
  if (workspace == nullptr || workspace_bytes < l.total) return PA_ERR_WORKSPACE_TOO_SMALL;
  if (reinterpret_cast<uintptr_t>(workspace) & 3u) return PA_ERR_INVALID_ARG;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    const int most = kMaxBeams * kThreads * static_cast<int>(sizeof(int32_t));
    cudaError_t e = cudaFuncSetAttribute(fork_count_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fork_apply_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return record_cuda_error(e, "cudaFuncSetAttribute(fork)");
    configured_device = dev;
  }
  int32_t* w = static_cast<int32_t*>(workspace);
  const ForkParams p{parents, seq_lens, groups, beams, block_table, bt_stride, free_pages, free_capacity, free_count,
                     num_pages, free_count_out, seq_lens_out, copies, shared_pages, status, l.blocks, l.span,
                     w + l.freed, w + l.differ, w + l.copied, w + l.copy_of, w + l.old_lens, w + l.tail, w + l.count};
  const dim3 grid(static_cast<unsigned>(l.blocks), static_cast<unsigned>(groups));  // (groups <= kMaxRows)
  const size_t smem = static_cast<size_t>(beams) * kThreads * sizeof(int32_t);
  cudaError_t e = launch_dependent(fork_count_kernel, grid, kThreads, smem, st, 0, p);
  if (e == cudaSuccess) e = launch_dependent(fork_apply_kernel, grid, kThreads, smem, st, 0, p);
  return e == cudaSuccess ? PA_OK : record_cuda_error(e, "paged_fork");
}

extern "C" pa_status paged_copy_pages(pa_dims dims, const int32_t* copies, int32_t rows, void* const* pools,
                                      int32_t num_pools, int64_t num_pages, int32_t* status, pa_stream_t stream) {
  using namespace pa;
  if (!gqa_dims_supported(dims)) return PA_ERR_UNSUPPORTED;
  if (rows < 0 || num_pools < 0 || num_pages <= 0) return PA_ERR_INVALID_ARG;
  if (rows == 0 || num_pools == 0) return PA_OK;
  if (!copies || !pools) return PA_ERR_INVALID_ARG;
  for (int32_t i = 0; i < num_pools; ++i)
    if (!pools[i] || (reinterpret_cast<uintptr_t>(pools[i]) & 15u)) return PA_ERR_INVALID_ARG;
  CopyParams p;
  p.copies = copies;
  p.num_pages = num_pages;
  p.vectors = dims.num_kv_heads * kHeadDim * 2 / 16;
  p.status = status;
  for (int32_t i0 = 0; i0 < num_pools; i0 += kPoolsPerLaunch) {
    const int32_t n = std::min(kPoolsPerLaunch, num_pools - i0);
    for (int32_t i = 0; i < kPoolsPerLaunch; ++i) p.pools[i] = i < n ? static_cast<uint4*>(pools[i0 + i]) : nullptr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows), static_cast<unsigned>(n));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, copy_pages_kernel, p);
    if (e != cudaSuccess) return record_cuda_error(e, "copy_pages_kernel");
  }
  return PA_OK;
}
