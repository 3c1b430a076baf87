// Block tables, row offsets, slot map and the free-page stack of one ragged
// step over a paged cache, from the requests' lengths.
//
// Mathematics: with held the pages a request has (ceil(cache / 64), or more
// where a cache was cut back behind its last step) and need = max(ceil((cache +
// new) / 64) - held, 0), three prefix sums over the requests (new rows, needed pages, pages
// given back) place everything: request b's rows start at its row prefix, its
// i-th new page is number (its page prefix + i) off the top of the stack, and
// a page given back lands above the old top in request order.  All of it is a
// pure function of the inputs, so every CTA computes the whole scan (a few
// thousand lengths at most) and then writes its share of the outputs; a page
// number is never read back from a table entry this call writes.
//
// Bound: latency.  The outputs are 4 bytes a row and the inputs 8 bytes a
// request; what takes time is the chain of lengths, scan, table entry, store.
// One CTA holds small steps; from kPlanWide rows on the slot map is shared by
// as many CTAs as have four rows a thread (one CTA against the grid: 2085 rows
// 5.4 and 5.2 us, 3237 rows 6.8 and 5.5, 4133 rows 7.1 and 5.6, 12837 rows 13.2
// and 5.7).  Where kv_len or free_count_out is the input array, or held_len is
// updated, every CTA's reads have to come before the first write: then the CTAs
// are one cluster of eight and meet at its barrier (144000 rows of 512
// requests: 27 us, against 8 us for a grid of 71; 165 rows of 8 requests 6 to 7
// us, against 5.3).
#include "ptx.cuh"
#include "step.h"

namespace dvlm {

namespace {
constexpr int kPlanThreads = 512;
constexpr int kPlanPer = kPlanMaxBatch / kPlanThreads;  // requests per thread of the scan
constexpr int kPlanCtas = 8;
constexpr int kPlanWide = 4096;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanNoPage = (1 << 25) - 1;  // past every store; its slot numbers still fit 31 bits

// Inclusive scan over the warp.
__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Last b with pre[b] <= i (pre ascending, pre[0] = 0): the request owning
// item i of a prefix-summed list.
__device__ __forceinline__ int owner_of(const int* pre, int n, int i) {
  int lo = 0, hi = n;  // pre[lo] <= i < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}
}  // namespace

__global__ void __launch_bounds__(kPlanThreads, 1) page_plan_kernel(const PagePlanArgs a) {
  extern __shared__ int sm[];
  int* s_row = sm;                          // [n + 1] first row of each request
  int* s_need = s_row + a.n_batch + 1;      // [n + 1] first new page
  int* s_free = s_need + a.n_batch + 1;     // [n + 1] first page given back
  int* s_cache = s_free + a.n_batch + 1;    // [n] cached lengths
  int* s_held = s_cache + a.n_batch;        // [n] pages held
  __shared__ long long w_sum[3][kPlanWarps];
  __shared__ int s_rows, s_pages;           // admitted rows and pages

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, n_cta = gridDim.x, n = a.n_batch;
  const long long cap = static_cast<long long>(a.max_pages) * 64;
  int err = 0;
  int count = *a.free_count;
  if (count < 0 || count > a.n_pages) {
    err = DVLM_ERR_BOUNDS;
    count = count < 0 ? 0 : a.n_pages;
  }

  // each thread takes kPlanPer consecutive requests (as few as n needs)
  const int per = (n + kPlanThreads - 1) / kPlanThreads;
  int want[kPlanPer], need[kPlanPer], freed[kPlanPer], cache[kPlanPer], held[kPlanPer];
  bool live[kPlanPer], part[kPlanPer];
  long long t0 = 0, t1 = 0, t2 = 0;
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    const int b = tid * per + i;
    want[i] = need[i] = freed[i] = cache[i] = held[i] = 0;
    live[i] = true;
    part[i] = false;
    if (i >= per || b >= n) continue;
    const int c = a.cache_len[b], m = a.new_len[b], hl = a.held_len ? max(a.held_len[b], c) : c;
    if (c < 0 || hl > cap || m < -1) {
      err = DVLM_ERR_BOUNDS;  // such a request takes no part
      continue;
    }
    part[i] = true;
    cache[i] = c;
    held[i] = (hl + 63) >> 6;
    if (m < 0) {
      live[i] = false;
      freed[i] = held[i];
    } else if (c + static_cast<long long>(m) > cap) {
      err = DVLM_ERR_BOUNDS;
    } else {
      want[i] = m;
      need[i] = max(((c + m + 63) >> 6) - held[i], 0);
    }
    t0 += want[i];
    t1 += need[i];
    t2 += freed[i];
  }
  const long long i0 = warp_scan(t0, lane), i1 = warp_scan(t1, lane), i2 = warp_scan(t2, lane);
  if (lane == 31) {
    w_sum[0][warp] = i0;
    w_sum[1][warp] = i1;
    w_sum[2][warp] = i2;
  }
  if (tid == 0) s_rows = s_pages = 0;
  __syncthreads();
  const int wl = lane & (kPlanWarps - 1);
  const long long x0 = lane < kPlanWarps ? w_sum[0][wl] : 0, x1 = lane < kPlanWarps ? w_sum[1][wl] : 0;
  const long long x2 = lane < kPlanWarps ? w_sum[2][wl] : 0;
  const long long y0 = warp_scan(x0, lane), y1 = warp_scan(x1, lane), y2 = warp_scan(x2, lane);
  long long r0 = __shfl_sync(0xffffffffu, y0 - x0, warp) + i0 - t0;  // exclusive prefixes of this thread
  long long r1 = __shfl_sync(0xffffffffu, y1 - x1, warp) + i1 - t1;
  long long r2 = __shfl_sync(0xffffffffu, y2 - x2, warp) + i2 - t2;
  const long long total_freed = __shfl_sync(0xffffffffu, y2, 31);
  const long long avail = count + total_freed;

  // Admission: requests are served in order while their pages and rows fit;
  // both prefixes ascend, so the first that does not fit and all behind it
  // wait (their rows and pages count 0).  Offsets past the admitted totals
  // are cut to them below.
  bool fits[kPlanPer];
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    const int b = tid * per + i;
    fits[i] = false;
    if (i >= per || b >= n) continue;
    s_cache[b] = cache[i];
    s_held[b] = held[i];
    s_row[b] = static_cast<int>(r0 < a.max_rows ? r0 : a.max_rows);
    s_need[b] = static_cast<int>(r1 < avail ? r1 : avail);
    s_free[b] = static_cast<int>(r2);
    r0 += want[i];
    r1 += need[i];
    r2 += freed[i];
    fits[i] = r0 <= a.max_rows && r1 <= avail;
    if (fits[i]) {
      if (want[i] > 0) {
        atomicMax(&s_rows, static_cast<int>(r0));
        if (need[i] > 0) atomicMax(&s_pages, static_cast<int>(r1));
      }
    } else if (want[i] > 0 && err == 0) {
      err = DVLM_ERR_CACHE_OVERFLOW;
    }
  }
  if (rank == 0 && err) record_error(a.status, err);
  __syncthreads();
  const int rows = s_rows, pages = s_pages;
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    const int b = tid * per + i;
    if (i >= per || b >= n) continue;
    s_row[b] = min(s_row[b], rows);
    s_need[b] = min(s_need[b], pages);
  }
  if (tid == 0) {
    s_row[n] = rows;
    s_need[n] = pages;
    s_free[n] = static_cast<int>(total_freed);
  }
  // the scan is complete, and in place every CTA has read the inputs
  if (a.in_place) cluster_sync();
  else __syncthreads();

  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      const int b = tid * per + i;
      if (i >= per || b >= n) continue;
      // (in place, the length of a request that takes no part is not lost: its pages can still be given back)
      if (part[i] || a.kv_len != a.cache_len) a.kv_len[b] = live[i] ? cache[i] + (fits[i] ? want[i] : 0) : 0;
      a.cu_rows[b] = s_row[b];
      if (a.held_len && part[i]) a.held_len[b] = live[i] ? max(a.held_len[b], cache[i] + (fits[i] ? want[i] : 0)) : 0;
    }
    if (tid == 0) {
      a.cu_rows[n] = rows;
      *a.free_count_out = static_cast<int>(min(avail - pages, static_cast<long long>(a.n_pages)));
    }
  }

  // page number `r` of those given back, and the page at `i` from the top
  auto returned = [&](int r) -> int {
    const int b = owner_of(s_free, n, r);
    return a.block_table[static_cast<size_t>(b) * a.max_pages + (r - s_free[b])];
  };
  auto taken = [&](int i) -> int {
    const long long at = avail - 1 - i;
    return at < count ? a.free_pages[at] : returned(static_cast<int>(at - count));
  };
  const int gtid = rank * kPlanThreads + tid, gsize = n_cta * kPlanThreads;
  for (int i = gtid; i < pages; i += gsize) {
    const int b = owner_of(s_need, n, i);
    a.block_table[static_cast<size_t>(b) * a.max_pages + s_held[b] + (i - s_need[b])] = taken(i);
  }
  for (long long r = gtid; r < total_freed - pages; r += gsize) {
    if (count + r < a.n_pages) a.free_pages[count + r] = returned(static_cast<int>(r));
    else record_error(a.status, DVLM_ERR_BOUNDS);
  }

  // four consecutive rows per thread: one search, one 16-byte store
  const bool vec = (reinterpret_cast<uintptr_t>(a.slot_map) & 15u) == 0;
  for (long long i4 = static_cast<long long>(gtid) * 4; i4 < a.max_rows; i4 += static_cast<long long>(gsize) * 4) {
    const int i = static_cast<int>(i4);
    int v[4] = {-1, -1, -1, -1};
    if (i < rows) {
      int b = owner_of(s_row, n, i), last = -1, page = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (i + e >= rows) break;
        while (i + e >= s_row[b + 1]) {
          ++b;
          last = -1;
        }
        const int slot = s_cache[b] + (i + e - s_row[b]), p = slot >> 6, held = s_held[b];
        if (p != last) {
          page = p < held ? a.block_table[static_cast<size_t>(b) * a.max_pages + p] : taken(s_need[b] + p - held);
          // a wild number's slots must not wrap into the store, and -1's must not
          // reach slot -1, which means padding
          page = page == -1 ? -2 : max(-kPlanNoPage, min(page, kPlanNoPage));
          last = p;
        }
        v[e] = page * 64 + (slot & 63);
      }
    }
    if (vec && i + 3 < a.max_rows) {
      *reinterpret_cast<int4*>(a.slot_map + i) = make_int4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < a.max_rows) a.slot_map[i + e] = v[e];
    }
  }
}

cudaError_t launch_page_plan(const PagePlanArgs& a, cudaStream_t s) {
  const int smem = (5 * a.n_batch + 3) * 4;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (5 * kPlanMaxBatch + 3) * 4);
    if (e != cudaSuccess) return e;
  }
  const bool in_place = a.in_place != 0;
  const int per = kPlanThreads * 4, wide = (a.max_rows + per - 1) / per;
  const int n_cta = a.max_rows < kPlanWide ? 1 : in_place ? kPlanCtas : (wide < device_sm_count() ? wide : device_sm_count());
  if (!in_place) {  // (a plain launch costs the host half of one with attributes)
    page_plan_kernel<<<n_cta, kPlanThreads, smem, s>>>(a);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(n_cta);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = n_cta;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, page_plan_kernel, a);
}

}  // namespace dvlm
