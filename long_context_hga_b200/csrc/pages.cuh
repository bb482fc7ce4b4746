// Pages of a cache: taking, sharing, returning, gathering together and copying
// them, with the bookkeeping (page table, lengths, reference counts) on the
// device, so that a captured step can do it.
//
// Every operation is a plan and, where bytes move, a copy.  The plan is one
// block: a page always goes to the lowest free index, in the order of the
// call's list, so results do not depend on timing.  Bound of the copies: HBM,
// 2 x bytes moved: compacting 110 MB takes 36 us (6.1 TB/s) after a plan of 6;
// 128 copies of 16 pages in 36 planes (340 MB written, 42 MB read) about 60 us.
#pragma once
#include "common.cuh"

namespace hga {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;

struct PoolArgs {
  char* data;
  int64_t page_bytes, plane_stride;
  int n_pages, n_planes, page_tokens, n_rows, row_pages;
  int32_t *table, *len, *ref;
  // workspace (int32): count[8], wa, wb, wc [max(n_pages, n_rows)] each,
  // claim [2 n_rows], need [n_rows]
  int32_t *count, *wa, *wb, *wc, *claim, *need;
};

// Exclusive prefix sum of v over the block; *total receives the sum.
__device__ __forceinline__ int block_scan(int v, int* total) {
  __shared__ int warp_sums[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                       // earlier reads of warp_sums are done
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int w = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return (warp ? before : 0) + x - v;
}

// Lists the pages in [lo, hi) whose use (ref != 0) equals `used`, ascending,
// into out[0 .. most); returns how many were listed.
__device__ __forceinline__ int list_pages(const int32_t* ref, int lo, int hi, bool used,
                                          int32_t* out, int most) {
  int found = 0;
  for (int base = lo; base < hi && found < most; base += 4 * kPlanThreads) {
    const int i0 = base + 4 * threadIdx.x;
    bool hit[4];
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hit[j] = i0 + j < hi && (ref[i0 + j] != 0) == used;
      n += hit[j];
    }
    int total;
    int at = found + block_scan(n, &total);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (hit[j]) {
        if (at < most) out[at] = i0 + j;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  return min(found, most);
}

// ---------------------------------------------------------------- free

// One block per listed row.  atomicExch takes each entry exactly once, so a
// row listed twice is freed once.
__global__ void __launch_bounds__(kCopyThreads) pages_free_kernel(PoolArgs a,
                                                                  const int32_t* rows) {
  griddep_wait();
  const int r = rows[blockIdx.x];
  if (r < 0) return;                      // padding of a fixed-size list
  if (r >= a.n_rows) {
    if (threadIdx.x == 0) report(HGA_ERR_DEVICE_CHECK);
    return;
  }
  int32_t* row = a.table + (int64_t)r * a.row_pages;
  for (int c = threadIdx.x; c < a.row_pages; c += kCopyThreads) {
    if (row[c] < 0) continue;
    const int pg = atomicExch(&row[c], -1);
    if (pg < 0) continue;
    if (pg >= a.n_pages) {
      report(HGA_ERR_DEVICE_CHECK);
      continue;
    }
    if (atomicSub(&a.ref[pg], 1) <= 0) {  // was free already: the table is broken
      atomicAdd(&a.ref[pg], 1);
      report(HGA_ERR_DEVICE_CHECK);
    }
  }
  if (threadIdx.x == 0) a.len[r] = 0;
}

// ---------------------------------------------------------------- reserve and fork: plans

// The pages that entry i of the list gets are ranks [before, before + need) of
// the free pages in ascending order.  When they run out, that entry and every
// later one that needs a page gets none.
__device__ __forceinline__ int pages_needed(const PoolArgs& a, int32_t tokens) {
  return (int)(((int64_t)tokens + a.page_tokens - 1) / a.page_tokens);
}

// claim[row] = lowest list index that names it.
__device__ __forceinline__ void claim_rows(const PoolArgs& a, const int32_t* rows, int n) {
  for (int i = threadIdx.x; i < a.n_rows; i += kPlanThreads) a.claim[i] = 0x7fffffff;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int r = rows[i];
    if (r >= 0 && r < a.n_rows) atomicMin(&a.claim[r], i);
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kPlanThreads) pages_reserve_kernel(PoolArgs a,
                                                                     const int32_t* rows,
                                                                     const int32_t* new_len,
                                                                     int n) {
  griddep_wait();
  claim_rows(a, rows, n);
  // need[i] = -1: nothing to do or refused
  int sum = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    int need = -1;
    if (i < n && rows[i] >= 0) {
      const int r = rows[i];
      if (r < a.n_rows && a.claim[r] == i && new_len[i] >= a.len[r] && a.len[r] >= 0 &&
          new_len[i] <= (int64_t)a.row_pages * a.page_tokens)
        need = pages_needed(a, new_len[i]) - pages_needed(a, a.len[r]);
      else
        report(HGA_ERR_DEVICE_CHECK);
    }
    int total;
    const int before = sum + block_scan(max(need, 0), &total);
    if (i < n) {
      a.need[i] = need;
      a.claim[a.n_rows + i] = before;     // prefix, kept beside the claims
    }
    sum += total;
  }
  const int have = list_pages(a.ref, 0, a.n_pages, false, a.wa, min(sum, a.n_pages));
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int need = a.need[i], before = a.claim[a.n_rows + i];
    if (need < 0) continue;
    const int r = rows[i];
    if (need > 0 && before + need > have) {
      report(HGA_ERR_DEVICE_CHECK);
      continue;
    }
    const int at = pages_needed(a, a.len[r]);
    int32_t* row = a.table + (int64_t)r * a.row_pages;
    for (int j = 0; j < need; ++j) {
      const int pg = a.wa[before + j];
      row[at + j] = pg;
      a.ref[pg] = 1;
    }
    a.len[r] = new_len[i];
  }
}

// wa: free pages, wb[i] = page of pair i that is copied from (or -1), wc[i] =
// where to; need[i] = -1 refused, 0 shares only, 1 shares and copies.
__global__ void __launch_bounds__(kPlanThreads) pages_fork_plan_kernel(PoolArgs a,
                                                                       const int32_t* parents,
                                                                       const int32_t* children,
                                                                       int n) {
  griddep_wait();
  claim_rows(a, children, n);
  int sum = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    int need = -1;
    if (i < n && children[i] >= 0) {
      const int c = children[i], p = parents[i];
      // the child is empty, named once, and no child of this call is a parent
      if (c < a.n_rows && p >= 0 && p < a.n_rows && a.claim[c] == i &&
          a.claim[p] == 0x7fffffff && a.len[c] == 0 && a.len[p] >= 0 &&
          a.len[p] <= (int64_t)a.row_pages * a.page_tokens)
        need = a.len[p] % a.page_tokens > 0;
      else
        report(HGA_ERR_DEVICE_CHECK);
    }
    int total;
    const int before = sum + block_scan(max(need, 0), &total);
    if (i < n) {
      a.need[i] = need;
      a.claim[a.n_rows + i] = before;
    }
    sum += total;
  }
  __syncthreads();
  const int have = list_pages(a.ref, 0, a.n_pages, false, a.wa, min(sum, a.n_pages));
  if (threadIdx.x == 0) a.count[0] = 0;
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    int need = a.need[i];
    const int before = a.claim[a.n_rows + i];
    if (need > 0) {
      const int p = parents[i];
      const int src = a.table[(int64_t)p * a.row_pages + a.len[p] / a.page_tokens];
      if (before >= have || src < 0 || src >= a.n_pages) {
        report(HGA_ERR_DEVICE_CHECK);
        a.need[i] = need = -1;
      } else {
        a.wb[i] = src;
        a.wc[i] = a.wa[before];
        a.ref[a.wa[before]] = 1;
      }
    }
    if (need <= 0) a.wb[i] = a.wc[i] = -1;
  }
  griddep_launch();
}

// Copies of whole pages over every plane.  Copy j (j < n) moves page src[j] to
// dst[j]; pairs with a negative entry are skipped.  A block's turn is 16 KB of a
// page (four 16-byte vectors of a thread in flight) of GROUP neighbouring
// copies: those from one source (a parent's children) read it once.
template <int GROUP>
__device__ __forceinline__ void copy_pages(const PoolArgs& a, const int32_t* src,
                                           const int32_t* dst, int n, int64_t block,
                                           int64_t n_blocks) {
  const int64_t vecs = a.page_bytes / 16;
  constexpr int kPiece = kCopyThreads * 4;
  const int64_t pieces = (vecs + kPiece - 1) / kPiece;
  const int groups = (n + GROUP - 1) / GROUP;
  const int64_t total = pieces * a.n_planes * groups;
  for (int64_t w = block; w < total; w += n_blocks) {
    const int64_t pp = w / pieces, piece = w - pp * pieces;
    const int plane = (int)(pp / groups), j0 = (int)(pp - (int64_t)plane * groups) * GROUP;
    char* base = a.data + plane * a.plane_stride;
    const int64_t at = piece * kPiece + threadIdx.x;
    uint4 v[4];
    int have = -1;
    for (int j = j0; j < j0 + GROUP && j < n; ++j) {
      const int s = src[j], d = dst[j];
      if (s < 0 || d < 0) continue;
      if (s != have) {
        const uint4* from = reinterpret_cast<const uint4*>(base + s * a.page_bytes);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (at + k * kCopyThreads < vecs) v[k] = from[at + k * kCopyThreads];
        have = s;
      }
      uint4* to = reinterpret_cast<uint4*>(base + d * a.page_bytes);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (at + k * kCopyThreads < vecs) __stcs(to + at + k * kCopyThreads, v[k]);
    }
  }
}

// Shares and copies of a planned fork: block i < n fills child i's table row.
template <int GROUP>
__global__ void __launch_bounds__(kCopyThreads) pages_fork_kernel(PoolArgs a,
                                                                  const int32_t* parents,
                                                                  const int32_t* children, int n) {
  griddep_wait();
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    if (a.need[i] < 0) continue;
    const int p = parents[i], c = children[i];
    const int len = a.len[p], full = len / a.page_tokens;
    const int32_t* from = a.table + (int64_t)p * a.row_pages;
    int32_t* to = a.table + (int64_t)c * a.row_pages;
    for (int j = threadIdx.x; j < a.row_pages; j += kCopyThreads) {
      int pg = -1;
      if (j < full) {
        pg = from[j];
        if (pg < 0 || pg >= a.n_pages) {
          report(HGA_ERR_DEVICE_CHECK);
          pg = -1;
        } else {
          atomicAdd(&a.ref[pg], 1);
        }
      } else if (j == full && a.need[i] > 0) {
        pg = a.wc[i];
      }
      to[j] = pg;
    }
    if (threadIdx.x == 0) a.len[c] = len;
  }
  copy_pages<GROUP>(a, a.wb, a.wc, n, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------- compact

// wa: used pages at or above the used count, wb: free pages below it (as many,
// both ascending), wc[page] = where a page at or above the count goes, -1 for a
// free one.  The counts move here; the table follows wc.
__global__ void __launch_bounds__(kPlanThreads) pages_compact_plan_kernel(PoolArgs a) {
  griddep_wait();
  int used = 0;
  for (int base = 0; base < a.n_pages; base += 4 * kPlanThreads) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = base + 4 * threadIdx.x + j;
      n += i < a.n_pages && a.ref[i] != 0;
    }
    int total;
    block_scan(n, &total);
    used += total;
  }
  const int moves = list_pages(a.ref, used, a.n_pages, true, a.wa, a.n_pages);
  list_pages(a.ref, 0, used, false, a.wb, a.n_pages);
  if (threadIdx.x == 0) {
    a.count[0] = moves;
    a.count[1] = used;
  }
  for (int i = used + threadIdx.x; i < a.n_pages; i += kPlanThreads) a.wc[i] = -1;
  __syncthreads();
  for (int j = threadIdx.x; j < moves; j += kPlanThreads) {
    const int from = a.wa[j], to = a.wb[j];
    a.wc[from] = to;
    a.ref[to] = a.ref[from];
    a.ref[from] = 0;
  }
  griddep_launch();
}

__global__ void __launch_bounds__(kCopyThreads) pages_compact_kernel(PoolArgs a) {
  griddep_wait();
  const int moves = a.count[0], used = a.count[1];
  const int64_t tid = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
  const int64_t nthr = (int64_t)gridDim.x * kCopyThreads;
  for (int64_t i = tid; i < (int64_t)a.n_rows * a.row_pages; i += nthr) {
    const int pg = a.table[i];
    if (pg < used) continue;
    const int to = pg < a.n_pages ? a.wc[pg] : -1;
    if (to >= 0) a.table[i] = to;
    else report(HGA_ERR_DEVICE_CHECK);    // no page of the pool, or a free one
  }
  copy_pages<1>(a, a.wa, a.wb, moves, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------- copy

// Refuses a pair whose page is outside the pool, whose target an earlier pair
// has, or whose target is a source of the call (wa: claims of the targets, wb
// and wc: the accepted pairs).
__global__ void __launch_bounds__(kPlanThreads) pages_copy_plan_kernel(PoolArgs a,
                                                                       const int32_t* src,
                                                                       const int32_t* dst, int n) {
  griddep_wait();
  for (int i = threadIdx.x; i < a.n_pages; i += kPlanThreads) a.wa[i] = 0x7fffffff;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    if (dst[i] >= 0 && dst[i] < a.n_pages) atomicMin(&a.wa[dst[i]], i);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads)
    if (src[i] >= 0 && src[i] < a.n_pages && dst[i] >= 0) atomicMin(&a.wa[src[i]], -1);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int s = src[i], d = dst[i];
    const bool skip = s < 0 && d < 0;     // padding of a fixed-size list
    const bool ok = s >= 0 && s < a.n_pages && d >= 0 && d < a.n_pages && a.wa[d] == i;
    if (!ok && !skip) report(HGA_ERR_DEVICE_CHECK);
    a.wb[i] = ok ? s : -1;
    a.wc[i] = ok ? d : -1;
  }
  griddep_launch();
}

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(PoolArgs a, int n) {
  griddep_wait();
  copy_pages<1>(a, a.wb, a.wc, n, blockIdx.x, gridDim.x);
}

}  // namespace hga
