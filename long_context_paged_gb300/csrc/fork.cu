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
  int32_t* freed;    // [groups][blocks] pages that a block gives back
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
  uint64_t has_child;         // rows that some child continues
  uint64_t live;              // children that are not empty
  int32_t max_pages;          // of the old rows
  int32_t bad;
};

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kPage - 1) / kPage; }

// One warp's worth of threads would do; every thread of the CTA takes part in the barriers.
__device__ __forceinline__ void read_group(const ForkParams& p, const int32_t* lens, int g, Group& s) {
  const int W = p.beams, t = threadIdx.x;
  if (t == 0) {
    s.has_child = s.live = 0;
    s.max_pages = s.bad = 0;
  }
  __syncthreads();
  if (t < W) {
    const int parent = p.parents[g * W + t], len = lens[g * W + t];
    if (parent < -1 || parent >= W || len < 0 || len > p.bt_stride * kPage) s.bad = 1;
    s.parent[t] = parent;
    s.old_len[t] = len;
    if (len > 0) atomicMax(&s.max_pages, pages_of(min(len, p.bt_stride * kPage)));
  }
  __syncthreads();
  if (t < W && !s.bad) {
    const int parent = s.parent[t];
    s.len[t] = parent < 0 ? 0 : s.old_len[parent];
    if (parent >= 0)
      atomicOr(reinterpret_cast<unsigned long long*>(&s.has_child), 1ull << parent);
    if (s.len[t] > 0) atomicOr(reinterpret_cast<unsigned long long*>(&s.live), 1ull << t);
  }
  __syncthreads();
}

// Logical page j of the group's rows, read into this thread's column of `col`.
__device__ __forceinline__ void read_column(const ForkParams& p, const int32_t* rows, int j, int32_t* col) {
#pragma unroll 8
  for (int r = 0; r < p.beams; ++r)
    col[r * kThreads] = j < p.bt_stride ? rows[static_cast<int64_t>(r) * p.bt_stride + j] : -1;
}

// Whether row r, which has no child, gives back its page j: a page of the pool that no row with a
// child holds, and no earlier row.
__device__ __forceinline__ bool gives_back(const ForkParams& p, const Group& s, const int32_t* col, int j, int r) {
  if (s.has_child >> r & 1 || j >= pages_of(s.old_len[r])) return false;
  const int32_t e = col[r * kThreads];
  if (e < 0 || e >= p.num_pages) return false;
  for (int o = 0; o < p.beams; ++o)
    if (o != r && (o < r || s.has_child >> o & 1) && col[o * kThreads] == e && j < pages_of(s.old_len[o])) return false;
  return true;
}

// Whether all rows in use have page j in common, filled.
__device__ __forceinline__ bool common(const ForkParams& p, const Group& s, const int32_t* col, int j) {
  int32_t one = -1;
  for (uint64_t m = s.live; m != 0; m &= m - 1) {
    const int b = __ffsll(static_cast<long long>(m)) - 1;
    const int32_t e = col[s.parent[b] * kThreads];
    if (one < 0) one = e;
    if (e < 0 || e != one || j >= s.len[b] / kPage) return false;
  }
  return one >= 0;
}

__device__ __forceinline__ int block_sum(int v, int32_t* scratch) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += scratch[w];
  __syncthreads();
  return sum;
}

__global__ void __launch_bounds__(kThreads) fork_count_kernel(const ForkParams p) {
  extern __shared__ int32_t columns[];  // [beams][kThreads]
  __shared__ Group s;
  __shared__ int32_t scratch[kWarps], first;
  const int tid = threadIdx.x, W = p.beams;
  const int g = static_cast<int>(blockIdx.x) / p.blocks, block = static_cast<int>(blockIdx.x) % p.blocks;
  await_previous();
  // the end of the free list, from which copies take their pages, and the lengths: both may be
  // overwritten by the second launch
  int count = *p.free_count;
  if (count < 0 || count > p.free_capacity) {
    if (blockIdx.x == 0 && tid == 0) flag_error(p.status, PA_DEV_ERR_LENGTH);
    count = count < 0 ? 0 : p.free_capacity;
  }
  if (blockIdx.x == 0 && tid == 0) *p.count = count;
  if (block == 0 && tid < W) {
    const int i = g * W + tid;
    p.old_lens[i] = p.seq_lens[i];
    p.tail[i] = i < count ? p.free_pages[count - 1 - i] : -1;
  }
  if (tid == 0) first = kNone;
  read_group(p, p.seq_lens, g, s);
  int32_t* col = columns + tid;
  const int32_t* rows = p.block_table + static_cast<int64_t>(g) * W * p.bt_stride;
  int freed = 0;
  const int j0 = block * p.span;
  if (!s.bad) {
    for (int j = j0 + tid; j < min(j0 + p.span, s.max_pages); j += kThreads) {
      read_column(p, rows, j, col);
      for (int r = 0; r < W; ++r) {
        if (gives_back(p, s, col, j, r)) ++freed;
        if (col[r * kThreads] >= p.num_pages && !(s.has_child >> r & 1) && j < pages_of(s.old_len[r]))
          flag_error(p.status, PA_DEV_ERR_PAGE_OOB);
      }
      if (!common(p, s, col, j)) atomicMin(&first, j);
    }
  }
  freed = block_sum(freed, scratch);
  if (tid == 0) {
    p.freed[blockIdx.x] = freed;
    p.differ[blockIdx.x] = first;
  }
  if (block != 0) return;
  // the children whose last page is copied: partly filled, and held by another child that comes
  // first or has it filled
  int32_t from = -1;
  if (tid < W) {
    if (!s.bad && s.len[tid] % kPage != 0) {
      const int last = s.len[tid] / kPage;
      const int32_t e = rows[static_cast<int64_t>(s.parent[tid]) * p.bt_stride + last];
      if (e < 0 || e >= p.num_pages) {
        flag_error(p.status, PA_DEV_ERR_PAGE_OOB);
      } else {
        for (int b = 0; b < W; ++b)
          if (b != tid && last < pages_of(s.len[b]) && (b < tid || s.len[b] >= (last + 1) * kPage) &&
              rows[static_cast<int64_t>(s.parent[b]) * p.bt_stride + last] == e)
            from = e;
      }
    }
    p.copy_of[g * W + tid] = from;
  }
  const int copied = block_sum(from >= 0 ? 1 : 0, scratch);
  if (tid == 0) p.copied[g] = s.bad ? -1 : copied;
}

__global__ void __launch_bounds__(kThreads) fork_apply_kernel(const ForkParams p) {
  extern __shared__ int32_t columns[];
  __shared__ Group s;
  __shared__ int32_t scratch[kWarps], fresh[kMaxBeams], warp_freed[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = p.beams;
  const int g = static_cast<int>(blockIdx.x) / p.blocks, block = static_cast<int>(blockIdx.x) % p.blocks;
  await_previous();
  // counts before this block, and of all
  int before = 0, freed = 0, copies_before = 0, copies = 0, bad = 0;
  for (int i = tid; i < p.groups * p.blocks; i += kThreads) {
    const int n = p.freed[i];
    freed += n;
    if (i < static_cast<int>(blockIdx.x)) before += n;
  }
  for (int i = tid; i < p.groups; i += kThreads) {
    const int n = p.copied[i];
    if (n < 0) bad = 1;
    copies += max(n, 0);
    if (i < g) copies_before += max(n, 0);
  }
  before = block_sum(before, scratch);
  freed = block_sum(freed, scratch);
  copies_before = block_sum(copies_before, scratch);
  copies = block_sum(copies, scratch);
  bad = block_sum(bad, scratch);
  const int count = *p.count;
  const bool short_of = copies > count;
  const bool full = static_cast<int64_t>(count) - copies + freed > p.free_capacity;
  if (blockIdx.x == 0 && tid == 0) {
    if (bad || full) flag_error(p.status, PA_DEV_ERR_LENGTH);
    if (short_of) flag_error(p.status, PA_DEV_ERR_NO_PAGES);
    *p.free_count_out = bad || full || short_of ? count : count - copies + freed;
  }
  if (bad || full || short_of) {  // nothing changes
    if (block == 0 && tid < W) {
      const int i = g * W + tid;
      p.seq_lens_out[i] = p.old_lens[i];
      p.copies[3 * i] = p.copies[3 * i + 1] = -1;
      p.copies[3 * i + 2] = 0;
    }
    if (block == 0 && tid == 0) p.shared_pages[g] = 0;
    return;
  }
  read_group(p, p.old_lens, g, s);
  // the pages that the group's copies get: the list's last ones, in row order
  if (tid < W) {
    int i = copies_before;
    for (int b = 0; b < tid; ++b) i += p.copy_of[g * W + b] >= 0 ? 1 : 0;
    fresh[tid] = p.copy_of[g * W + tid] >= 0 ? p.tail[i] : kNone;
  }
  __syncthreads();
  int32_t* rows = p.block_table + static_cast<int64_t>(g) * W * p.bt_stride;
  int32_t* col = columns + tid;
  if (block == 0) {
    int differ = kNone;
    for (int i = tid; i < p.blocks; i += kThreads) differ = min(differ, p.differ[g * p.blocks + i]);
    if (tid < W && s.len[tid] > 0) differ = min(differ, s.len[tid] / kPage);
    differ = __reduce_min_sync(0xffffffffu, differ);
    if (lane == 0) scratch[warp] = differ;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) differ = min(differ, scratch[w]);
      p.shared_pages[g] = s.live == 0 ? 0 : differ;
    }
    if (tid < W) {
      const int i = g * W + tid, page = fresh[tid];
      p.seq_lens_out[i] = s.len[tid];
      int32_t src = -1, dst = -1, n = 0;
      if (page != kNone) {
        if (page < 0 || page >= p.num_pages) {
          flag_error(p.status, PA_DEV_ERR_PAGE_OOB);
        } else {
          src = p.copy_of[i];
          dst = page;
          n = s.len[tid] % kPage;
        }
      }
      p.copies[3 * i] = src;
      p.copies[3 * i + 1] = dst;
      p.copies[3 * i + 2] = n;
    }
  }
  int at = count - copies + before;
  const int j0 = block * p.span, j1 = min(j0 + p.span, s.max_pages);
  for (int jb = j0; jb < j1; jb += kThreads) {
    const int j = jb + tid;
    int n = 0;
    if (j < j1) {
      read_column(p, rows, j, col);
      for (int r = 0; r < W; ++r) n += gives_back(p, s, col, j, r) ? 1 : 0;
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
    int to = at + incl - n;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) to += warp_freed[w];
      at += warp_freed[w];
    }
    __syncthreads();
    if (j < j1) {
      for (int r = 0; n > 0 && r < W; ++r)
        if (gives_back(p, s, col, j, r)) {
          p.free_pages[to++] = col[r * kThreads];
          --n;
        }
      for (int b = 0; b < W; ++b) {
        const int32_t e = col[b * kThreads];
        int32_t now = e;
        if (j < pages_of(s.len[b]))
          now = fresh[b] != kNone && j == s.len[b] / kPage ? fresh[b] : col[s.parent[b] * kThreads];
        else if (j < pages_of(s.old_len[b]))
          now = -1;
        if (now != e) rows[static_cast<int64_t>(b) * p.bt_stride + j] = now;
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// paged_copy_pages: the first n tokens of a page, 16 bytes a thread and load, for every row of
// copies[] and every pool: a CTA per pair. Bound by HBM (each byte read once and written once).
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
  const unsigned grid = static_cast<unsigned>(groups) * static_cast<unsigned>(l.blocks);
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
