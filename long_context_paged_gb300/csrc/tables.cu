// paged_step_plan / paged_release: block tables, positions and slot maps from request lengths,
// on the GPU (sm_103a).
//
// With c_b cached and n_b new tokens, request b holds ceil(c_b / 16) pages and needs
//     need_b = ceil((c_b + n_b) / 16) - ceil(c_b / 16)
// more. With cum_b = need_0 + .. + need_b, it is served when need_b = 0 or cum_b <= free pages:
// the served needs are then a prefix of all needs, so request b's k-th new page is
// free[count - 1 - (cum_b - need_b) - k] whatever the other requests got, and the assignment is a
// pair of prefix sums, the same on every run. Packed row t of request b (cu_b <= t < cu_{b+1}) is
// position p = c_b + t - cu_b in slot page(p / 16) * 16 + p % 16.
//
// The work is a few KB of lengths in and 12 bytes per row out: bound by latency (a launch, one
// round of loads, a block-wide scan, one round of stores), not by bandwidth. So one launch does it
// all: every CTA scans all the lengths by itself (4 per
// thread at most) and then writes its share of the rows, so that nothing is exchanged between
// CTAs. Where an output is an input's buffer (lengths or free count updated in place), the grid is one
// cluster of at most 8 CTAs, whose barrier orders the reads before the writes; else any grid does
// (57,000 rows: 8.8 us, in place 11.9 us).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "cluster_common.cuh"
#include "dependent_launch.cuh"
#include "pa_common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBatch = 4096;
constexpr int kMaxCluster = 8;
// A call has a CTA for every so many rows (or requests), up to one per SM, in place up to kMaxCluster. A CTA
// writes 4 consecutive rows a thread, 4,096 of them at a pass, so from 1,024 on the rows need no more CTAs
// than 4,096 each would give: 57,000 rows take 8.9 us at 1,024 to 4,096 and 11.8 at 8,192, 4,127 rows 5.1
// and 6.2. The requests' own work (a new page's search and table entry) is spread over all of them: 4,096
// requests of a token each, all with a new page, 9.3 us at 512, 9.4 at 1,024, 10.8 at 2,048, 14.1 at 4,096.
constexpr int kRowsPerCta = 1024;

struct PlanParams {
  const int32_t* cached;
  const int32_t* fresh;
  int32_t batch;
  int32_t* block_table;
  int32_t bt_stride;
  const int32_t* free_pages;
  int32_t free_capacity;
  const int32_t* free_count;
  int64_t num_pages;
  int32_t total_rows;
  int32_t* free_count_out;
  int32_t* cu;
  int32_t* seq_lens;
  int32_t* positions;
  int64_t* slots;
  int32_t* status;
  bool vector_rows;  // positions and slots are 16-byte aligned
  bool in_place;     // an output is an input's buffer: the grid is one cluster
};

struct PlanSmem {
  long long warp_rows[kWarps], warp_need[kWarps];
  int32_t cu[kMaxBatch + 1];   // first packed row of each request
  int32_t need[kMaxBatch + 1]; // pages needed by the requests before
  int32_t cached[kMaxBatch];   // cached tokens; ~tokens (negative) of a request that is not served
};

__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

// Last i in [0, n) with a[i] <= x (a non-decreasing, a[0] <= x).
__device__ __forceinline__ int last_at_most(const int32_t* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int pages_of(long long tokens) {
  return static_cast<int>((tokens + kPage - 1) / kPage);
}

// The free list's page count as the kernels use it: within [0, capacity], flagged if it was not.
__device__ __forceinline__ int read_free_count(const int32_t* count, int capacity, int32_t* status,
                                               bool report) {
  const int n = *count;
  if (n >= 0 && n <= capacity) return n;
  if (report) flag_error(status, PA_DEV_ERR_LENGTH);
  return n < 0 ? 0 : capacity;
}

__global__ void __launch_bounds__(kThreads, 1) step_plan_kernel(const PlanParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  PlanSmem& s = *reinterpret_cast<PlanSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
  const bool report = rank == 0;
  const int capacity = p.bt_stride * kPage;  // < 2^31: checked on the host

  await_previous();
  const int free_count = read_free_count(p.free_count, p.free_capacity, p.status, report && tid == 0);
  const int per = (p.batch + kThreads - 1) / kThreads;  // <= 4
  const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  int c[4], n[4], need[4], len[4];  // len: tokens after the step
  bool valid[4];
  long long rows = 0, pages = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    c[k] = n[k] = need[k] = len[k] = 0;
    valid[k] = false;
    if (b0 + k < b1) {
      c[k] = p.cached[b0 + k];
      n[k] = p.fresh[b0 + k];
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (b0 + k < b1) {
      valid[k] = c[k] >= 0 && n[k] >= 0 && static_cast<long long>(c[k]) + n[k] <= capacity;
      if (!valid[k] && report) flag_error(p.status, PA_DEV_ERR_LENGTH);
      n[k] = max(n[k], 0);  // a request that does not fit keeps its rows in the packing
      if (valid[k]) need[k] = pages_of(c[k] + n[k]) - pages_of(c[k]);
      rows += n[k];
      pages += need[k];
    }
  }
  if (p.batch == 0 && tid == 0) s.cu[0] = s.need[0] = 0;
  const long long rows_in = warp_scan(rows, lane), pages_in = warp_scan(pages, lane);
  if (lane == 31) {
    s.warp_rows[warp] = rows_in;
    s.warp_need[warp] = pages_in;
  }
  __syncthreads();
  if (warp == 0) {
    const long long r = s.warp_rows[lane], q = s.warp_need[lane];
    s.warp_rows[lane] = warp_scan(r, lane) - r;
    s.warp_need[lane] = warp_scan(q, lane) - q;
  }
  __syncthreads();
  const long long kMax = 0x7fffffffll;
  long long r_run = s.warp_rows[warp] + rows_in - rows, q_run = s.warp_need[warp] + pages_in - pages;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (b0 + k < b1) {
      const bool served = valid[k] && (need[k] == 0 || q_run + need[k] <= free_count);
      if (report && valid[k] && !served) flag_error(p.status, PA_DEV_ERR_NO_PAGES);
      s.cu[b0 + k] = static_cast<int32_t>(min(r_run, kMax));
      s.need[b0 + k] = static_cast<int32_t>(min(q_run, kMax));
      c[k] = min(max(c[k], 0), capacity);
      s.cached[b0 + k] = served ? c[k] : ~c[k];
      len[k] = served ? c[k] + n[k] : c[k];
      r_run += n[k];
      q_run += need[k];
      if (b0 + k == p.batch - 1) {
        s.cu[p.batch] = static_cast<int32_t>(min(r_run, kMax));
        s.need[p.batch] = static_cast<int32_t>(min(q_run, kMax));
      }
    }
  }
  if (p.in_place && ctas > 1) cluster_sync_all(); else __syncthreads();

  // ---- per request: length after the step (from the lengths themselves: the packed offsets end at
  //      2^31 - 1; by the last CTA, which has the fewest rows), packed offset, new table entries
  if (rank == ctas - 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (b0 + k < b1) p.seq_lens[b0 + k] = len[k];
  }
  const int all = ctas * kThreads, id = rank * kThreads + tid;
  for (int b = id; b <= p.batch; b += all) p.cu[b] = s.cu[b];
  const int total = s.cu[p.batch], rows_end = min(total, p.total_rows);
  // the served needs are a prefix of all needs: everything up to the free count, cut back to
  // where the last served request ends
  int used = s.need[p.batch];
  if (used > free_count) {
    const int b = last_at_most(s.need, p.batch + 1, free_count);
    used = s.need[b];
  }
  for (int64_t i0 = id; i0 < used; i0 += all) {
    const int i = static_cast<int>(i0);
    const int b = last_at_most(s.need, p.batch, i);
    const int lp = pages_of(s.cached[b]) + (i - s.need[b]);
    const int page = p.free_pages[free_count - 1 - i];
    if (page < 0 || page >= p.num_pages) flag_error(p.status, PA_DEV_ERR_PAGE_OOB);
    p.block_table[static_cast<int64_t>(b) * p.bt_stride + lp] = page;
  }
  if (id == 0) {
    *p.free_count_out = free_count - used;
    if (total > p.total_rows) flag_error(p.status, PA_DEV_ERR_LENGTH);
  }
  // ---- per row: position and slot; rows of requests that wait, and rows past the last request,
  //      are (0, -1). Four consecutive rows a thread: one search (the next rows are mostly the same
  //      request's or the next one's), four page loads in flight, 16-byte stores.
  for (int64_t t0 = 4ll * id; t0 < p.total_rows; t0 += 4ll * all) {
    int pos[4], page[4];
    const int32_t* entry[4];
    int b = t0 < rows_end ? last_at_most(s.cu, p.batch, static_cast<int>(t0)) : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t t = t0 + k;
      pos[k] = 0;
      entry[k] = nullptr;
      if (t < rows_end) {
        if (t >= s.cu[b + 1]) {
          ++b;
          if (t >= s.cu[b + 1]) b = last_at_most(s.cu, p.batch, static_cast<int>(t));
        }
        const int cb = s.cached[b];
        if (cb >= 0) {
          pos[k] = cb + static_cast<int>(t) - s.cu[b];
          const int lp = pos[k] / kPage, held = pages_of(cb);
          entry[k] = lp < held ? p.block_table + static_cast<int64_t>(b) * p.bt_stride + lp
                               : p.free_pages + (free_count - 1 - (s.need[b] + lp - held));
        }
      }
    }
    int64_t slot[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = entry[k] != nullptr ? *entry[k] : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      slot[k] = -1;
      if (entry[k] != nullptr) {
        if (page[k] < 0 || page[k] >= p.num_pages) flag_error(p.status, PA_DEV_ERR_PAGE_OOB);
        else slot[k] = static_cast<int64_t>(page[k]) * kPage + pos[k] % kPage;
      }
    }
    if (p.vector_rows && t0 + 4 <= p.total_rows) {
      *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      reinterpret_cast<longlong2*>(p.slots + t0)[0] = make_longlong2(slot[0], slot[1]);
      reinterpret_cast<longlong2*>(p.slots + t0)[1] = make_longlong2(slot[2], slot[3]);
    } else {
      for (int k = 0; k < 4 && t0 + k < p.total_rows; ++k) {
        p.positions[t0 + k] = pos[k];
        p.slots[t0 + k] = slot[k];
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// paged_release: the valid entries of each request's page range go back on the free list, in
// (request, page) order, and become -1 in the table. Two passes over the ranges: count (a warp
// per request, four rounds of loads in flight), a scan of the counts, then the pushes at their
// final places. CTA r of the cluster takes the r-th share of the requests; the CTAs' totals are
// exchanged through distributed shared memory.
// ---------------------------------------------------------------------------------------------
struct ReleaseParams {
  const int32_t* begin;
  const int32_t* end;
  int32_t batch;
  int32_t* block_table;
  int32_t bt_stride;
  int32_t* free_pages;
  int32_t free_capacity;
  const int32_t* free_count;
  int64_t num_pages;
  int32_t* free_count_out;
  int32_t* status;
};

// The page range of request b, cut to its table row, flagged if pages outside the row were named. (Any
// begin past the row, up to INT32_MAX, is cut too, so that stepping on from it stays within 32 bits.)
__device__ __forceinline__ void release_range(const ReleaseParams& p, int b, bool report, int& lo, int& hi) {
  lo = p.begin[b];
  hi = p.end[b];
  if (lo < 0 || hi > p.bt_stride) {
    if (report) flag_error(p.status, PA_DEV_ERR_LENGTH);
    lo = max(lo, 0);
    hi = min(hi, p.bt_stride);
  }
  lo = min(lo, p.bt_stride);
}

__global__ void __launch_bounds__(kThreads, 1) release_kernel(const ReleaseParams p) {
  __shared__ int32_t warp_count[kWarps];
  __shared__ int32_t cta_count[kMaxCluster];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_nctarank());
  if (ctas > 1) cluster_sync_all();  // every CTA has started before any writes to another's shared memory
  await_previous();
  const int free_count = read_free_count(p.free_count, p.free_capacity, p.status, rank == 0 && tid == 0);
  // this warp's requests: a contiguous share, so that the pushes of all warps are in order
  const int w = rank * kWarps + warp, all = ctas * kWarps;
  const int b0 = static_cast<int>(static_cast<int64_t>(w) * p.batch / all);
  const int b1 = static_cast<int>(static_cast<int64_t>(w + 1) * p.batch / all);
  auto usable = [&](int e) { return e >= 0 && e < p.num_pages; };

  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    int lo, hi;
    release_range(p, b, lane == 0, lo, hi);
    const int32_t* row = p.block_table + static_cast<int64_t>(b) * p.bt_stride;
    for (int i = lo + lane; i < hi; i += 128) {
      int e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = i + 32 * k < hi ? row[i + 32 * k] : -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        mine += usable(e[k]) ? 1 : 0;
        if (e[k] >= p.num_pages) flag_error(p.status, PA_DEV_ERR_PAGE_OOB);
      }
    }
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) warp_count[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    const int v = warp_count[lane];
    const int incl = static_cast<int>(warp_scan(v, lane));
    warp_count[lane] = incl - v;
    const int sum = __shfl_sync(0xffffffffu, incl, 31);
    if (lane < ctas) {
      if (ctas == 1) cta_count[0] = sum;
      else
        asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(map_to_rank(&cta_count[rank], lane)), "r"(sum)
                     : "memory");
    }
  }
  if (ctas > 1) cluster_sync_all(); else __syncthreads();
  int before = 0;
  long long total = 0;
  for (int r = 0; r < ctas; ++r) {
    if (r < rank) before += cta_count[r];
    total += cta_count[r];
  }
  // more pages than the list has room for: nothing is released
  if (free_count + total > p.free_capacity) {
    if (rank == 0 && tid == 0) {
      flag_error(p.status, PA_DEV_ERR_LENGTH);
      *p.free_count_out = free_count;
    }
    return;
  }
  if (rank == 0 && tid == 0) *p.free_count_out = free_count + static_cast<int>(total);
  int at = free_count + before + warp_count[warp];
  for (int b = b0; b < b1; ++b) {
    int lo, hi;
    release_range(p, b, false, lo, hi);
    int32_t* row = p.block_table + static_cast<int64_t>(b) * p.bt_stride;
    for (int i0 = lo; i0 < hi; i0 += 128) {
      int e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + 32 * k + lane;
        e[k] = i < hi ? row[i] : -1;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + 32 * k + lane;
        const bool push = usable(e[k]);
        const uint32_t votes = __ballot_sync(0xffffffffu, push);
        if (push) p.free_pages[at + __popc(votes & ((1u << lane) - 1u))] = e[k];
        if (i < hi) row[i] = -1;
        at += __popc(votes);
      }
    }
  }
}

// One cluster over `work` items, kRowsPerCta each, of 1, 2, 4 or 8 CTAs.
int cluster_of(int64_t work, int64_t per_cta) {
  int c = 1;
  while (c < kMaxCluster && c * per_cta < work) c *= 2;
  return c;
}

template <class Params>
pa_status launch_cluster(void (*kernel)(Params), const Params& p, int ctas, size_t smem,
                         cudaStream_t stream, const char* name) {
  const cudaError_t e = launch_dependent(kernel, static_cast<unsigned>(ctas), kThreads, smem, stream, ctas, p);
  return e == cudaSuccess ? PA_OK : record_cuda_error(e, name);
}

}  // namespace
}  // namespace pa

extern "C" pa_status paged_step_plan(const int32_t* cached_lens, const int32_t* new_lens, int32_t batch,
                                     int32_t* block_table, int32_t bt_stride,
                                     const int32_t* free_pages, int32_t free_capacity,
                                     const int32_t* free_count, int64_t num_pages,
                                     int32_t total_rows, int32_t* free_count_out,
                                     int32_t* cu_new_lens, int32_t* seq_lens, int32_t* positions,
                                     int64_t* slot_map, int32_t* status, pa_stream_t stream) {
  using namespace pa;
  if (batch < 0 || bt_stride <= 0 || bt_stride > 0x7fffffff / kPage || free_capacity < 0 ||
      num_pages <= 0 || total_rows < 0)
    return PA_ERR_INVALID_ARG;
  if (batch > kMaxBatch) {
    snprintf_error("paged_step_plan: at most %d requests per call", kMaxBatch);
    return PA_ERR_UNSUPPORTED;
  }
  // (an empty batch still gets its offsets, free count and padding rows)
  if (!free_count || !free_count_out || !cu_new_lens ||
      (batch > 0 && (!cached_lens || !new_lens || !block_table || !seq_lens)) ||
      (free_capacity > 0 && !free_pages) || (total_rows > 0 && (!positions || !slot_map)))
    return PA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(slot_map) & 7u) return PA_ERR_INVALID_ARG;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    const cudaError_t e = cudaFuncSetAttribute(step_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(sizeof(PlanSmem)));
    if (e != cudaSuccess) return record_cuda_error(e, "cudaFuncSetAttribute(step_plan)");
    configured_device = dev;
  }
  PlanParams p{cached_lens, new_lens, batch, block_table, bt_stride, free_pages, free_capacity, free_count,
               num_pages, total_rows, free_count_out, cu_new_lens, seq_lens, positions, slot_map, status,
               ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(slot_map)) & 15u) == 0,
               free_count_out == free_count || seq_lens == cached_lens};
  const int64_t work = std::max(total_rows, batch);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p.in_place)
    return launch_cluster(step_plan_kernel, p, cluster_of(work, kRowsPerCta), sizeof(PlanSmem), st, "step_plan_kernel");
  const int sms = sm_count_current_device();
  if (sms <= 0) return PA_ERR_CUDA;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(sms, std::max<int64_t>(1, (work + kRowsPerCta - 1) / kRowsPerCta)));
  const cudaError_t e = launch_dependent(step_plan_kernel, grid, kThreads, sizeof(PlanSmem), st, 0, p);
  return e == cudaSuccess ? PA_OK : record_cuda_error(e, "step_plan_kernel");
}

extern "C" pa_status paged_release(const int32_t* begin_pages, const int32_t* end_pages, int32_t batch,
                                   int32_t* block_table, int32_t bt_stride, int32_t* free_pages,
                                   int32_t free_capacity, const int32_t* free_count,
                                   int64_t num_pages, int32_t* free_count_out, int32_t* status,
                                   pa_stream_t stream) {
  using namespace pa;
  if (batch < 0 || bt_stride <= 0 || bt_stride > 0x7fffffff / kPage || free_capacity < 0 || num_pages <= 0)
    return PA_ERR_INVALID_ARG;
  if (batch > kMaxBatch) {
    snprintf_error("paged_release: at most %d requests per call", kMaxBatch);
    return PA_ERR_UNSUPPORTED;
  }
  if (static_cast<int64_t>(batch) * bt_stride > 0x7fffffff) {  // the pages are counted in 32 bits
    snprintf_error("paged_release: a table of %d x %d entries (2^31 and more are not supported)", batch, bt_stride);
    return PA_ERR_UNSUPPORTED;
  }
  if (!free_count || !free_count_out || (batch > 0 && (!begin_pages || !end_pages || !block_table)) ||
      (free_capacity > 0 && !free_pages))
    return PA_ERR_INVALID_ARG;
  ReleaseParams p{begin_pages, end_pages, batch, block_table, bt_stride, free_pages, free_capacity, free_count,
                  num_pages, free_count_out, status};
  return launch_cluster(release_kernel, p, cluster_of(batch, kWarps), 0, reinterpret_cast<cudaStream_t>(stream),
                        "release_kernel");
}
