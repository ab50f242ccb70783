// Drafts: the masks of their trees, the path that the model accepts, and giving
// the rejected ones back.
//
// A step's new tokens of a sequence are a tree: each has a parent among those
// before it, or none. Everything here is small (a few ints a token, a few slots a
// layer) and bound by latency: few dependent loads, few launches. Measured (GB300):
// masks, path and keeping for 4 sequences of up to 12 drafts in 4 layers 9.4 us on the
// device in a chain of such steps (the four kernels and a copy of the tables), for 64
// sequences of up to 60 in 32 layers of an e4m3 cache 20 us; the three calls take
// the host 64 to 82.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "ptx.cuh"

namespace seqattn {
namespace {

constexpr int kStatusBadPath = 4, kStatusShared = 5, kStatusRefused = 6;

// A sequence's packed rows, clamped.
struct Rows {
  int q0, n;
};
__device__ __forceinline__ Rows rows_of(const int *cu, int b, int total) {
  const int q0 = min(max(cu[b], 0), total);
  return {q0, min(max(cu[b + 1], q0), total) - q0};
}

// ---------------------------------------------------------------- masks
// One CTA a sequence, a thread a token. A token's ancestors by doubling: with
// mask[t] the tokens on the way from t up to but not including up[t],
//   mask[t] |= mask[up[t]],  up[t] = up[up[t]]
// doubles the way, so a tree of depth d takes ceil(log2(d + 1)) rounds. The depth
// is the number of ancestors. A sequence of more tokens than the masks have bits is
// no tree (its masks 0, its depths the tokens' places).
constexpr int kTreeThreads = 256;  // tokens of the largest tree: 64 kDraftWords

__global__ void __launch_bounds__(kTreeThreads)
    tree_kernel(const int *parents, const int *cu, unsigned long long *masks, int *depths, int total, int words) {
  __shared__ unsigned long long mask[kDraftWords][kTreeThreads];
  __shared__ int up[kTreeThreads];
  launch_dependents();
  wait_prerequisites();
  const Rows s = rows_of(cu, blockIdx.x, total);
  const int t = threadIdx.x;
  if (s.n > 64 * words) {
    for (int i = t; i < s.n; i += kTreeThreads) {
      for (int w = 0; w < words; ++w) masks[static_cast<size_t>(s.q0 + i) * words + w] = 0;
      depths[s.q0 + i] = i;
    }
    return;
  }
  int u = t < s.n ? parents[s.q0 + t] : -1;
  if (u < 0 || u >= t) u = -1;  // a parent that is not an earlier token is none
  up[t] = u;
#pragma unroll
  for (int w = 0; w < kDraftWords; ++w) mask[w][t] = t >> 6 == w ? 1ull << (t & 63) : 0ull;
  while (__syncthreads_or(u >= 0)) {
    unsigned long long more[kDraftWords];
    int next = -1;
#pragma unroll
    for (int w = 0; w < kDraftWords; ++w) more[w] = u >= 0 && w < words ? mask[w][u] : 0ull;
    if (u >= 0) next = up[u];
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kDraftWords; ++w) mask[w][t] |= more[w];
    up[t] = u = next;
  }
  if (t >= s.n) return;
  int depth = -1;
#pragma unroll
  for (int w = 0; w < kDraftWords; ++w)
    if (w < words) {
      masks[static_cast<size_t>(s.q0 + t) * words + w] = mask[w][t];
      depth += __popcll(mask[w][t]);
    }
  depths[s.q0 + t] = depth;
}

// ---------------------------------------------------------------- the accepted path
// One CTA a sequence; its first warp goes down the tree: the lowest child of the
// current token that is what the model chose after it. Children are behind their
// parents, so the search goes on from the token that was found. A sequence of more
// tokens than the masks of `words` words have bits (0: no masks) was attended as a
// chain, so it is one here: each token's only child is the next.
constexpr int kAcceptThreads = 128;
constexpr int kStaged = 1024;  // tokens from the last given one on that are brought to shared memory

__global__ void __launch_bounds__(kAcceptThreads)
    accept_kernel(const int *parents, const int *cu, const int *tokens, const int *choices, const int *given, int *path,
                  int *n_keep, int *last, int total, int words) {
  __shared__ int staged[3][kStaged];
  __shared__ int kept;
  launch_dependents();
  wait_prerequisites();
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const Rows s = rows_of(cu, b, total);
  if (s.n == 0) {
    if (threadIdx.x == 0) {
      n_keep[b] = 0;
      last[b] = -1;
    }
    return;
  }
  const int sure = given ? min(max(given[b], 1), s.n) : 1;
  const bool chain = words > 0 && s.n > 64 * words;
  const int from = sure - 1, rest = s.n - from;  // tokens from the last given one on
  const int *parent = parents + s.q0 + from, *token = tokens + s.q0 + from, *choice = choices + s.q0 + from;
  int *out = path + s.q0;
  for (int i = threadIdx.x; i < sure; i += kAcceptThreads) out[i] = i;
  if (rest <= kStaged) {
    for (int i = threadIdx.x; i < rest; i += kAcceptThreads) {
      staged[0][i] = parent[i];
      staged[1][i] = token[i];
      staged[2][i] = choice[i];
    }
    parent = staged[0];
    token = staged[1];
    choice = staged[2];
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int at = 0, n = sure;
    for (bool found = true; found;) {
      const int want = choice[at];
      found = false;
      const int end = chain ? min(rest, at + 2) : rest;
      for (int c0 = at + 1; c0 < end && !found; c0 += 32) {
        const int c = c0 + lane;
        const unsigned hit = __ballot_sync(0xffffffffu, c < end && (chain || parent[c] == at + from) && token[c] == want);
        if (hit != 0) {
          found = true;
          at = c0 + __ffs(hit) - 1;
          if (lane == 0) out[n] = at + from;
          ++n;
        }
      }
    }
    if (lane == 0) {
      n_keep[b] = n;
      last[b] = choice[at];
      kept = n;
    }
  }
  __syncthreads();
  for (int i = kept + threadIdx.x; i < s.n; i += kAcceptThreads) out[i] = -1;
}

// ---------------------------------------------------------------- keeping the path
// First kernel. blockIdx.y: row; blockIdx.x: share of the lines, a line being 16
// bytes (or one, of slots that are no multiple) of a slot in one (pool, layer,
// head): a thread takes its line of every kept slot, eight at a time, loaded before
// they are stored. Slot i is filled from path[i] >= i, and what later slots come
// from lies behind it, so going up in place is safe. Every CTA of a row finds the
// same verdict from the same tables; the first writes it down for the second kernel,
// which changes the tables.
constexpr int kKeepThreads = 256;

struct Verdict {
  int status, base, n, first;  // n kept slots from base on; `first`: the first one that moves
};

__device__ Verdict verdict(const KeepParams &p, int b) {
  const Rows s = rows_of(p.cu, b, p.total);
  const int len = p.t.kv_lens[b], n = p.n_keep[b], base = len - s.n;
  const int ps_log2 = p.t.page_log2;
  const bool room = len <= (static_cast<long long>(p.t.max_pages) << ps_log2);
  if (s.n == 0) return {0, len, 0, 0};
  const bool refused = p.guard != nullptr && RowGuard(p.guard, p.t.B).refuses(b, len, s.n);
  const bool sizes = base >= 0 && room && n >= 0 && n <= s.n;
  int first = n;
  bool bad = false, shared = false;
  if (!refused && sizes) {
    const int *path = p.path + s.q0, *row = p.t.page_table + b * p.t.table_stride;
    for (int i = threadIdx.x; i < n; i += kKeepThreads) {
      const int from = path[i], before = i > 0 ? path[i - 1] : -1;
      bad |= from <= before || from >= s.n;
      if (from != i) {
        first = min(first, i);
        if (from > i && from < s.n) {
          const int to = row[(base + i) >> ps_log2], src = row[(base + from) >> ps_log2];
          const bool there = to >= 0 && to < p.t.n_pages;
          shared |= there && p.t.page_refs[to] > 1;
          bad |= there && (src < 0 || src >= p.t.n_pages);
        }
      }
    }
  }
  // the page that the row then ends in takes its next tokens: no other row may have it
  if (threadIdx.x == 0 && !refused && sizes && n < s.n) {
    const int left = base + n;
    if ((left & ((1 << ps_log2) - 1)) != 0) {
      const int e = p.t.page_table[b * p.t.table_stride + (left >> ps_log2)];
      shared |= e >= 0 && e < p.t.n_pages && p.t.page_refs[e] > 1;
    }
  }
  __shared__ int firsts[kKeepThreads / 32];
  first = __reduce_min_sync(0xffffffffu, first);
  if ((threadIdx.x & 31) == 0) firsts[threadIdx.x >> 5] = first;
  bad = __syncthreads_or(bad);
  shared = __syncthreads_or(shared);
#pragma unroll
  for (int i = 0; i < kKeepThreads / 32; ++i) first = min(first, firsts[i]);
  const int status = refused ? kStatusRefused : (!sizes || bad ? kStatusBadPath : (shared ? kStatusShared : 0));
  return {status, base, n, first};
}

template <typename T>
__device__ __forceinline__ void move_line(const KeepParams &p, const Verdict &v, int b, int q0, const SlotPool &pool,
                                          int layer, int head, int at) {
  const int *path = p.path + q0, *row = p.t.page_table + b * p.t.table_stride;
  const int mask = (1 << p.t.page_log2) - 1;
  const long long head_at = (static_cast<long long>(head) << p.t.page_log2) * pool.slot_bytes + at;
  unsigned char *base = pool.base + layer * pool.layer_stride + head_at;
  auto place = [&](int slot) -> unsigned char * {
    const int page = row[slot >> p.t.page_log2];
    return page >= 0 && page < p.t.n_pages ? base + page * pool.page_stride + static_cast<long long>(slot & mask) * pool.slot_bytes
                                           : nullptr;
  };
  for (int i0 = v.first; i0 < v.n; i0 += 8) {
    T x[8];
    unsigned char *to[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      to[k] = i0 + k < v.n ? place(v.base + i0 + k) : nullptr;
      if (to[k] != nullptr) x[k] = *reinterpret_cast<const T *>(place(v.base + path[i0 + k]));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (to[k] != nullptr) *reinterpret_cast<T *>(to[k]) = x[k];
  }
}

__global__ void __launch_bounds__(kKeepThreads) keep_move_kernel(const __grid_constant__ KeepParams p) {
  launch_dependents();
  wait_prerequisites();
  const int b = blockIdx.y;
  const Verdict v = verdict(p, b);
  if (blockIdx.x == 0 && threadIdx.x == 0) p.status[b] = v.status;
  if (v.status != 0 || v.first >= v.n) return;
  const int q0 = rows_of(p.cu, b, p.total).q0;
  for (int line = blockIdx.x * kKeepThreads + threadIdx.x; line < p.lines; line += gridDim.x * kKeepThreads) {
    int i = 0, rest = line;
    while (rest >= p.pool[i].lines) rest -= p.pool[i++].lines;
    const SlotPool &pool = p.pool[i];
    const int unit = pool.slot_bytes % 16 == 0 ? 16 : 1, per_slot = pool.slot_bytes / unit;
    const int at = rest % per_slot * unit, head = rest / per_slot % pool.heads, layer = rest / per_slot / pool.heads;
    if (unit == 16) move_line<uint4>(p, v, b, q0, pool, layer, head, at);
    else move_line<unsigned char>(p, v, b, q0, pool, layer, head, at);
  }
}

// Second kernel: the tables. One CTA a row.
__global__ void __launch_bounds__(128) keep_tables_kernel(const __grid_constant__ KeepParams p) {
  launch_dependents();
  wait_prerequisites();
  const int b = blockIdx.x;
  const Rows s = rows_of(p.cu, b, p.total);
  if (p.status[b] != 0 || s.n == 0) return;
  const int len = p.t.kv_lens[b], left = len - s.n + p.n_keep[b], ps_log2 = p.t.page_log2;
  const int round = (1 << ps_log2) - 1;
  int *row = p.t.page_table + b * p.t.table_stride;
  const int end = static_cast<int>((static_cast<long long>(len) + round) >> ps_log2);
  for (int i = static_cast<int>((static_cast<long long>(left) + round) >> ps_log2) + threadIdx.x; i < end; i += 128) {
    const int e = row[i];
    if (e >= 0 && e < p.t.n_pages) atomicSub(&p.t.page_refs[e], 1);  // integers: any order, one result
    row[i] = -1;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    p.t.kv_lens[b] = left;
    if (p.guard != nullptr) RowGuard(p.guard, p.t.B).held[b] = 0;
  }
}

}  // namespace

cudaError_t launch_draft_tree(const int *parents, const int *cu, long long *masks, int *depths, int B, int total, int words,
                              cudaStream_t stream) {
  return launch_dependent(tree_kernel, dim3(B), dim3(kTreeThreads), 0, stream, parents, cu,
                          reinterpret_cast<unsigned long long *>(masks), depths, total, words);
}

cudaError_t launch_draft_accept(const int *parents, const int *cu, const int *tokens, const int *choices, const int *given,
                                int *path, int *n_keep, int *last, int B, int total, int words, cudaStream_t stream) {
  return launch_dependent(accept_kernel, dim3(B), dim3(kAcceptThreads), 0, stream, parents, cu, tokens, choices, given, path,
                          n_keep, last, total, words);
}

cudaError_t launch_keep(const KeepParams &p, cudaStream_t stream) {
  // enough CTAs for a few waves, whatever the rows
  const long long want = (static_cast<long long>(p.lines) + kKeepThreads - 1) / kKeepThreads;
  const long long most = static_cast<long long>(device_sm_count()) * 16 / p.t.B + 1;
  const long long x = want < 1 ? 1 : (want < most ? want : most);
  cudaError_t e = launch_dependent(keep_move_kernel, dim3(static_cast<unsigned>(x), p.t.B), dim3(kKeepThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_dependent(keep_tables_kernel, dim3(p.t.B), dim3(128), 0, stream, p);
}

}  // namespace seqattn
