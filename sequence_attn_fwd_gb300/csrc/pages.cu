// Page management of a paged K/V cache: reserving, freeing, forking, copying
// and compacting pages, on tables with reference counts that stay on the
// device. A page is free when no table entry holds it, so the reference
// counts are the only allocator state; new pages are always the lowest free
// ones in the order of the rows that need them, which makes every result a
// function of the tables alone.
//
// The searches read the counts (4 bytes a page) and are bound by latency; the
// copies move whole pages and are bound by DRAM. Measured (GB300): freeing 100
// forks of a 4,096-page pool, forking them again (26 MB of last pages over 16
// layer pools) and reserving their next tokens, four kernels, 22 us of the device in
// a chain of such cycles (the three calls, one after the other, 27 to 30 us: their
// host side); making a pool of 8 layers dense, 0.52 GB of pages moved, 168 us = 6.1
// TB/s of the 6.8 that a copy reaches.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "ptx.cuh"

namespace seqattn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kStatusNoPages = 1, kStatusTooLong = 2, kStatusInUse = 3;

// Exclusive prefix sum of one int per thread over the CTA; *total is the sum.
// `warp_sums` has 33 ints of shared memory.
__device__ __forceinline__ int block_scan(int x, int *warp_sums, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  __syncthreads();  // warp_sums may still be read from an earlier call
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = lane < warps ? warp_sums[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[warps - 1];
  return incl - x + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// The free ones of this thread's eight pages from `at` on, one bit each.
constexpr int kPagesPerThread = 8;
__device__ __forceinline__ unsigned free_mask(const int *refs, int n_pages, int at) {
  unsigned mask = 0;
#pragma unroll
  for (int i = 0; i < kPagesPerThread; ++i)
    if (at + i < n_pages && refs[at + i] == 0) mask |= 1u << i;
  return mask;
}

// Finds the `want` lowest free pages and calls give(rank, page) for each, until
// they run out; returns how many there were (the same on every thread).
// `ready`: free_mask of the first kPlanThreads * kPagesPerThread pages, which a
// caller loads along with what it needs first.
template <typename Give>
__device__ int find_free(const int *refs, int n_pages, int want, unsigned ready, int *warp_sums, Give give) {
  int found = 0;
  for (int base = 0; base < n_pages && found < want; base += kPlanThreads * kPagesPerThread) {
    const int at = base + threadIdx.x * kPagesPerThread;
    unsigned mask = base == 0 ? ready : free_mask(refs, n_pages, at);
    int total;
    int rank = found + block_scan(__popc(mask), warp_sums, &total);
    while (mask && rank < want) {
      give(rank, at + __ffs(mask) - 1);
      mask &= mask - 1;
      ++rank;
    }
    found += total;
  }
  return found < want ? found : want;
}

// Rank r among the needs of rows whose exclusive prefix sums are prefix[0..n]:
// the row i with prefix[i] <= r < prefix[i + 1].
__device__ __forceinline__ int row_of_rank(const int *prefix, int n, int r) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int pages_for(long long tokens, int page_log2) {
  return static_cast<int>((tokens + (1ll << page_log2) - 1) >> page_log2);
}

// prefix[0..n]: exclusive sums of the needs that prefix[i] holds at the start, n <= kPagedMaxRows.
__device__ void scan_needs(int *prefix, int n, int *warp_sums) {
  __syncthreads();
  const int per = (n + kPlanThreads - 1) / kPlanThreads;
  const int i0 = min(n, static_cast<int>(threadIdx.x) * per), i1 = min(n, i0 + per);
  int sum = 0;
  for (int i = i0; i < i1; ++i) sum += prefix[i];
  int total;
  int at = block_scan(sum, warp_sums, &total);
  for (int i = i0; i < i1; ++i) {
    const int need = prefix[i];
    prefix[i] = at;
    at += need;
  }
  if (threadIdx.x == 0) prefix[n] = total;
  __syncthreads();
}

// One CTA: needs, prefix sums, then one walk over the reference counts that
// gives rank r to the row whose range holds it. A row that the pool cannot
// serve whole (only the last one reached can have got some pages) gives them
// back. Bound by latency: lengths and the first counts are loaded together.
__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(PageTables t, const int *n_new, int *status, int *guard) {
  __shared__ int prefix[kPagedMaxRows + 1];
  __shared__ int length[kPagedMaxRows];  // -1: the row's table has no room
  __shared__ int warp_sums[33];
  launch_dependents();
  wait_prerequisites();
  const long long room = static_cast<long long>(t.max_pages) << t.page_log2;
  const unsigned ready = free_mask(t.page_refs, t.n_pages, threadIdx.x * kPagesPerThread);
  for (int b = threadIdx.x; b < t.B; b += kPlanThreads) {
    const long long len = max(t.kv_lens[b], 0), want = len + max(n_new[b], 0);
    const bool fits = want <= room;
    length[b] = fits ? static_cast<int>(len) : -1;
    // a sum of more than the pool has is never served
    prefix[b] = fits ? min(pages_for(want, t.page_log2) - pages_for(len, t.page_log2), t.n_pages + 1) : 0;
  }
  scan_needs(prefix, t.B, warp_sums);
  const int got = find_free(t.page_refs, t.n_pages, prefix[t.B], ready, warp_sums, [&](int rank, int page) {
    const int b = row_of_rank(prefix, t.B, rank);
    t.page_table[b * t.table_stride + pages_for(length[b], t.page_log2) + rank - prefix[b]] = page;
    t.page_refs[page] = 1;
  });
  __syncthreads();
  for (int b = threadIdx.x; b < t.B; b += kPlanThreads) {
    const int n = prefix[b + 1] - prefix[b];
    int st = length[b] >= 0 ? 0 : kStatusTooLong;
    if (n > 0 && prefix[b + 1] > got) {
      st = kStatusNoPages;
      const int have = pages_for(length[b], t.page_log2);
      for (int i = 0; i < got - prefix[b]; ++i) {
        int *e = &t.page_table[b * t.table_stride + have + i];
        t.page_refs[*e] = 0;
        *e = -1;
      }
    }
    const int asked = max(n_new[b], 0);
    if (guard != nullptr && asked > 0) {
      const int len = static_cast<int>(min(static_cast<long long>(max(t.kv_lens[b], 0)), room));
      RowGuard(guard, t.B).request(b, len, st == 0 ? len + asked : len, st != 0);
    }
    if (st == 0) t.kv_lens[b] = length[b] + asked;
    status[b] = st;
  }
}

// blockIdx.x: row of the list.
__global__ void free_kernel(PageTables t, const __grid_constant__ PageList rows) {
  launch_dependents();
  wait_prerequisites();
  const int b = rows.a[blockIdx.x];
  int *row = t.page_table + b * t.table_stride;
  for (int i = threadIdx.x; i < t.max_pages; i += blockDim.x) {
    const int e = row[i];
    if (e >= 0 && e < t.n_pages) atomicSub(&t.page_refs[e], 1);  // integers: any order, one result
    row[i] = -1;
  }
  if (threadIdx.x == 0) t.kv_lens[b] = 0;
}

// Whether a row of `len` tokens ends in a partly filled page that is there: the
// one that a fork copies. (An evicted last page is shared like the others: as the
// entry that it is.)
__device__ __forceinline__ bool copies_last(const PageTables &t, const int *row, int len) {
  if ((len & ((1 << t.page_log2) - 1)) == 0) return false;
  const int e = row[len >> t.page_log2];
  return e >= 0 && e < t.n_pages;
}

// Fork, first part (one CTA): checks the pairs and hands out the pages for
// their partly filled last ones.
__global__ void __launch_bounds__(kPlanThreads)
    fork_plan_kernel(PageTables t, const __grid_constant__ PageList pairs, int *status) {
  __shared__ int prefix[kPageListMax + 1];
  __shared__ int warp_sums[33];
  __shared__ int *entry[kPageListMax];  // where the target's own page goes
  launch_dependents();
  wait_prerequisites();
  const unsigned ready = free_mask(t.page_refs, t.n_pages, threadIdx.x * kPagesPerThread);
  const int i = threadIdx.x;  // kPageListMax pairs at most: one a thread
  bool in_use = false;
  if (i < pairs.n) {
    const long long room = static_cast<long long>(t.max_pages) << t.page_log2;
    const int dst = pairs.b[i];
    in_use = t.kv_lens[dst] != 0;
    const int len = static_cast<int>(min(static_cast<long long>(max(t.kv_lens[pairs.a[i]], 0)), room));
    prefix[i] = !in_use && copies_last(t, t.page_table + pairs.a[i] * t.table_stride, len);
    entry[i] = t.page_table + dst * t.table_stride + (len >> t.page_log2);
  }
  scan_needs(prefix, pairs.n, warp_sums);
  const int got = find_free(t.page_refs, t.n_pages, prefix[pairs.n], ready, warp_sums, [&](int rank, int page) {
    *entry[row_of_rank(prefix, pairs.n, rank)] = page;
    t.page_refs[page] = 1;
  });
  if (i < pairs.n)
    status[i] = in_use ? kStatusInUse : (prefix[i + 1] > got && prefix[i + 1] > prefix[i] ? kStatusNoPages : 0);
}
static_assert(kPageListMax <= kPlanThreads, "one pair a thread");

// Copies `bytes` (a multiple of 16) with the CTA's threads, four 16-byte loads in flight each.
__device__ __forceinline__ void copy_bytes(unsigned char *dst, const unsigned char *src, long long bytes) {
  const uint4 *s = reinterpret_cast<const uint4 *>(src);
  uint4 *d = reinterpret_cast<uint4 *>(dst);
  const long long n = bytes / 16;
  const int step = blockDim.x;
  for (long long i = threadIdx.x; i < n; i += 4 * step) {
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * step < n) x[k] = __ldcs(s + i + k * step);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * step < n) __stcs(d + i + k * step, x[k]);
  }
}

constexpr int kCopyThreads = 256;
constexpr long long kCopyChunk = 16384;  // bytes a CTA copies at a time: kCopyThreads x 4 x 16

// Copies page `src` over page `dst` in layer `layer` of the pools (layers of
// all pools counted through), chunk `chunk` of it.
__device__ __forceinline__ void copy_page(const PoolList &pools, int layer, int src, int dst, long long chunk) {
  int i = 0;
  while (layer >= pools.pool[i].n_layers) layer -= pools.pool[i++].n_layers;
  const PoolView &v = pools.pool[i];
  const long long at = chunk * kCopyChunk;
  if (at >= v.page_bytes) return;
  unsigned char *base = v.base + layer * v.layer_stride + at;
  const long long n = v.page_bytes - at < kCopyChunk ? v.page_bytes - at : kCopyChunk;
  copy_bytes(base + dst * v.page_stride, base + src * v.page_stride, n);
}

// Fork, second part. blockIdx.y: pair; blockIdx.x 0: its table row, references
// and length; the others: (layer, chunk) of its last page.
__global__ void __launch_bounds__(kCopyThreads)
    fork_copy_kernel(PageTables t, const __grid_constant__ PoolList pools, const __grid_constant__ PageList pairs,
                     const int *status, int chunks) {
  const int i = blockIdx.y, src = pairs.a[i], dst = pairs.b[i];
  launch_dependents();
  wait_prerequisites();
  if (status[i] != 0) return;
  const int room = static_cast<int>(min(static_cast<long long>(t.max_pages) << t.page_log2, 0x7fffffffll));
  const int len = min(max(t.kv_lens[src], 0), room);
  const int *from = t.page_table + src * t.table_stride;
  int *to = t.page_table + dst * t.table_stride;
  const bool ends_inside = (len & ((1 << t.page_log2) - 1)) != 0;
  const int last = ends_inside ? len >> t.page_log2 : 0;
  const int page = ends_inside ? from[last] : -1, own = ends_inside ? to[last] : -1;  // both loads at once
  const bool part = page >= 0 && page < t.n_pages;  // copies_last
  const int whole = part ? last : pages_for(len, t.page_log2);  // entries that are shared
  if (blockIdx.x == 0) {
    for (int c = threadIdx.x; c < t.max_pages; c += kCopyThreads) {
      if (c < whole) {
        const int e = from[c];
        to[c] = e;
        if (e >= 0 && e < t.n_pages) atomicAdd(&t.page_refs[e], 1);
      } else if (c > whole || !part) {
        to[c] = -1;
      }
    }
    if (threadIdx.x == 0) t.kv_lens[dst] = len;
  } else if (part) {
    const int item = blockIdx.x - 1;
    if (own >= 0 && own < t.n_pages)
      copy_page(pools, item / chunks, page, own, item % chunks);
  }
}

// blockIdx.y: pair; blockIdx.x: (layer, chunk).
__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(const __grid_constant__ PoolList pools, const __grid_constant__ PageList pairs, int chunks) {
  launch_dependents();
  wait_prerequisites();
  copy_page(pools, blockIdx.x / chunks, pairs.a[blockIdx.y], pairs.b[blockIdx.y], blockIdx.x % chunks);
}

// ---------------------------------------------------------------- compaction
// Pages are counted in blocks of kBlockPages. Workspace (ints): the number of
// moves, live counts of the blocks, per page its rank (as a hole below n_live
// or as a page to move from above, else -1), then holes, movers and the
// movers' references by rank.
constexpr int kBlockPages = 4096;

__global__ void __launch_bounds__(kPlanThreads) count_kernel(const int *refs, int n_pages, int *counts) {
  __shared__ int warp_sums[33];
  launch_dependents();
  wait_prerequisites();
  int live = 0;
#pragma unroll
  for (int k = 0; k < kBlockPages / kPlanThreads; ++k) {
    const int i = blockIdx.x * kBlockPages + k * kPlanThreads + threadIdx.x;
    live += i < n_pages && refs[i] > 0;
  }
  int total;
  block_scan(live, warp_sums, &total);
  if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

// Live pages before page `at`, by the whole CTA: the counts of whole blocks and
// a look into the block of `at`.
__device__ int live_before(const int *refs, const int *counts, int at, int *warp_sums) {
  const int block = at / kBlockPages;
  int live = 0;
  for (int i = threadIdx.x; i < block; i += kPlanThreads) live += counts[i];
  for (int i = block * kBlockPages + threadIdx.x; i < at; i += kPlanThreads) live += refs[i] > 0;
  int total;
  block_scan(live, warp_sums, &total);
  return total;
}

__global__ void __launch_bounds__(kPlanThreads)
    rank_kernel(const int *refs, int n_pages, const int *counts, int n_blocks, int *n_live_out, int *n_moves, int *rank,
                int *holes, int *movers, int *mover_refs) {
  __shared__ int warp_sums[33];
  launch_dependents();
  wait_prerequisites();
  int sum = 0;
  for (int i = threadIdx.x; i < n_blocks; i += kPlanThreads) sum += counts[i];
  int n_live;
  block_scan(sum, warp_sums, &n_live);
  const int below = live_before(refs, counts, n_live, warp_sums);  // live pages that stay
  const int before = live_before(refs, counts, blockIdx.x * kBlockPages, warp_sums);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *n_live_out = n_live;
    *n_moves = n_live - below;  // as many pages to move as holes to fill
  }
  constexpr int kPer = kBlockPages / kPlanThreads;
  const int at = blockIdx.x * kBlockPages + threadIdx.x * kPer;
  int r[kPer], live = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    r[k] = at + k < n_pages ? refs[at + k] : 0;
    live += r[k] > 0;
  }
  int total;
  int seen = before + block_scan(live, warp_sums, &total);  // live pages before this thread's
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = at + k;
    if (i < n_pages) {
      int mine = -1;
      if (i < n_live && r[k] <= 0) {
        mine = i - seen;
        holes[mine] = i;
      } else if (i >= n_live && r[k] > 0) {
        mine = seen - below;
        movers[mine] = i;
        mover_refs[mine] = r[k];
      }
      rank[i] = mine;
    }
    seen += r[k] > 0;
  }
}

// Table entries, references and the page data, each dealt over the whole grid.
__global__ void __launch_bounds__(kCopyThreads)
    move_kernel(const __grid_constant__ PoolList pools, const int *page_table, int *out_table, long long table_stride,
                const int *page_refs, int *out_refs, int B, int max_pages, int n_pages, const int *n_live_in,
                const int *n_moves_in, const int *rank, const int *holes, const int *movers, const int *mover_refs,
                int chunks) {
  launch_dependents();
  wait_prerequisites();
  const int n_live = *n_live_in;
  const long long tid = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x;
  const long long threads = static_cast<long long>(gridDim.x) * kCopyThreads;
  for (long long i = tid; i < static_cast<long long>(B) * max_pages; i += threads) {
    const long long at = i / max_pages * table_stride + i % max_pages;
    const int e = page_table[at];
    // an entry of a page that no reference counts (not a state these calls make) stays
    const bool moved = e >= n_live && e < n_pages && rank[e] >= 0;
    out_table[at] = moved ? holes[rank[e]] : e;
  }
  for (long long i = tid; i < n_pages; i += threads) {
    const int r = page_refs[i];
    out_refs[i] = i >= n_live ? 0 : (r > 0 ? r : mover_refs[rank[i]]);
  }
  const long long items = static_cast<long long>(*n_moves_in) * pools.total_layers * chunks;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const long long per = static_cast<long long>(pools.total_layers) * chunks;
    const int m = static_cast<int>(it / per), rest = static_cast<int>(it % per);
    copy_page(pools, rest / chunks, movers[m], holes[m], rest % chunks);
  }
}

int chunks_of(const PoolList &pools) {
  long long most = 0;
  for (int i = 0; i < pools.n; ++i) most = pools.pool[i].page_bytes > most ? pools.pool[i].page_bytes : most;
  return static_cast<int>((most + kCopyChunk - 1) / kCopyChunk);
}

}  // namespace

cudaError_t launch_reserve(const PageTables &t, const int *n_new, int *status, int *guard, cudaStream_t stream) {
  return launch_dependent(reserve_kernel, dim3(1), dim3(kPlanThreads), 0, stream, t, n_new, status, guard);
}

cudaError_t launch_free(const PageTables &t, const PageList &rows, cudaStream_t stream) {
  return launch_dependent(free_kernel, dim3(rows.n), dim3(256), 0, stream, t, rows);
}

cudaError_t launch_fork(const PageTables &t, const PoolList &pools, const PageList &pairs, int *status,
                        cudaStream_t stream) {
  cudaError_t e = launch_dependent(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, t, pairs, status);
  if (e != cudaSuccess) return e;
  const int chunks = chunks_of(pools);
  const dim3 grid(1 + static_cast<unsigned>(pools.total_layers) * chunks, pairs.n);
  return launch_dependent(fork_copy_kernel, grid, dim3(kCopyThreads), 0, stream, t, pools, pairs, status,
                          chunks > 0 ? chunks : 1);
}

cudaError_t launch_copy(const PoolList &pools, const PageList &pairs, cudaStream_t stream) {
  const int chunks = chunks_of(pools);
  const dim3 grid(static_cast<unsigned>(pools.total_layers) * chunks, pairs.n);
  return launch_dependent(copy_kernel, grid, dim3(kCopyThreads), 0, stream, pools, pairs, chunks);
}

cudaError_t launch_compact(const PoolList &pools, const int *page_table, int *out_table, long long table_stride,
                           const int *page_refs, int *out_refs, int *n_live, int *workspace, int B, int max_pages,
                           int n_pages, cudaStream_t stream) {
  const int n_blocks = (n_pages + kBlockPages - 1) / kBlockPages;
  int *n_moves = workspace, *counts = n_moves + 1, *rank = counts + n_blocks, *holes = rank + n_pages,
      *movers = holes + n_pages, *mover_refs = movers + n_pages;  // compact_workspace_ints in all
  cudaError_t e = launch_dependent(count_kernel, dim3(n_blocks), dim3(kPlanThreads), 0, stream, page_refs, n_pages, counts);
  if (e != cudaSuccess) return e;
  e = launch_dependent(rank_kernel, dim3(n_blocks), dim3(kPlanThreads), 0, stream, page_refs, n_pages, counts, n_blocks,
                       n_live, n_moves, rank, holes, movers, mover_refs);
  if (e != cudaSuccess) return e;
  const int chunks = chunks_of(pools);
  return launch_dependent(move_kernel, dim3(device_sm_count() * 8), dim3(kCopyThreads), 0, stream, pools, page_table,
                          out_table, table_stride, page_refs, out_refs, B, max_pages, n_pages, n_live, n_moves, rank,
                          holes, movers, mover_refs, chunks > 0 ? chunks : 1);
}

size_t compact_workspace_ints(int n_pages) {
  return 1 + (static_cast<size_t>(n_pages) + kBlockPages - 1) / kBlockPages + 4 * static_cast<size_t>(n_pages);
}

}  // namespace seqattn
