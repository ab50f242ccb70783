// Attention of new tokens over a paged K/V cache (included by attn_kernel.cu).
//
// For row (token, head) of a sequence: softmax(scale q K^T) V over the keys of
// its sequence that the row sees, K and V gathered page by page through the
// page table. With few rows per sequence the cost is reading K and V once; with
// many it is the two products.
//
// How. The G = Hq / Hkv query heads of a KV head share its keys, so they are
// rows of one tile: row r of a tile is token r / G, head r % G, `tok` whole
// tokens per 128-row tile (one TMA box of a 4-D view lays them out). A work
// item is two such tiles of one (sequence, KV head); its cost is the number
// of 128-key tiles its last token sees and a constant. The costs of all items,
// put end to end, are cut into equal ranges, one per CTA, whatever the lengths:
// every CTA has the same work to within one tile. An item inside one range is
// written directly; an item that ranges cut leaves one fp32 partial per range
// (normalised, with its log-sum-exp) in the workspace, at most two per CTA,
// and a second kernel merges them in the order of the keys. The cuts follow
// from the lengths alone, so results do not depend on timing. Each CTA finds
// its range from prefix sums over the sequences that it forms itself: no
// planning launch, and a captured graph follows the lengths it finds.
//
// Inside a CTA the roles are those of the dense forward: a TMA producer warp,
// an MMA issuer per query tile taking turns, a softmax warpgroup per query
// tile. The producer reads the page table, a window of 32 entries ahead, and
// issues a key tile as 128 / page_size boxes, or one box inside a larger page; 16
// keys a page cost no more than 128 (319 us against 318 for the batch below).
//
// Measured (GB300): 1,024 new tokens behind 65,536 keys, 32 heads over 8 KV heads
// of 128, 0.75 ms = 1,470 TFLOP/s in a chain of 15 calls and 0.86 ms = 1,290 under
// sustained load (power), 3,000 clocks a pair of tiles (the dense forward's share;
// the tensor pipe's own time is 2,048); six sequences of up to 600 new tokens behind
// up to 12,400 keys 162 us, and 11 more for the merge: the tiles at that rate, 12,000 clocks until the first scores of a CTA and about as
// many from an item to the next, most of it the epilogue of the softmax warps.
//
// This is the wide form. Sequences of at most 64 rows per KV head are the narrow
// form's (attn_paged_narrow.cuh): their items make a line of their own, and the
// CTAs are dealt to the two lines by their costs. Every CTA finds that out for
// itself, along with its range. (63 single tokens and a prompt piece of 512, 2.1 GB
// of cache: 356 us, with every item in the wide form 496.)
#pragma once

namespace seqattn {
namespace paged {

using namespace detail;

constexpr int kThreads = 352;
constexpr int kMmaWarp = 8, kTmaWarp = 9, kMmaWarp1 = 10;

template <int D>
struct Cfg {
  static constexpr int kColBlocks = D / 64;
  static constexpr int kTileBytes = kRowsPerTile * D * 2;
  static constexpr int kStages = 131072 / kTileBytes;
  static constexpr int kNumBarriers = 2 + 2 * kStages + 7;
  // tiles of the wide form (Q, ring, epilogue) or of the narrow one (ring, P, Q), then
  // barriers, three words, four segments, the narrow form's reductions (before
  // them, in the same place, the sums over warps). The prefix sums over the
  // sequences are needed before the tiles arrive only: they lie where the ring of
  // either form will be.
  static constexpr int kAreaBytes = 196608 + kRowsPerTile * 128 + 64 * D * 2;
  static_assert(2 * kTileBytes + kStages * kTileBytes + 8 * 2560 <= kAreaBytes, "wide layout");
  static constexpr int kItemBarrier = 2 * (196608 / kTileBytes) + 11;  // behind those of either form
  static constexpr int kMaxBarriers = kItemBarrier + 8;
  static constexpr int kRedFloats = 2 * 6 * 32;
  static constexpr int kPrefixAt = 65536;
  static_assert(kPrefixAt >= 2 * kTileBytes && kPrefixAt + 4 * (kPagedMaxSeqs + 1) <= 2 * kTileBytes + kStages * kTileBytes,
                "prefix sums inside either ring");
  static constexpr int kSmemBytes = 1024 + kAreaBytes + 8 * kMaxBarriers + 16 + 4 * 48 + 4 * kRedFloats;
};
static_assert(Cfg<128>::kSmemBytes <= 232448 && Cfg<64>::kSmemBytes <= 232448, "shared memory per CTA");

// A sequence's rows and keys, clamped so that every access stays in range.
struct Seq {
  int q0, q_len, kv_len;
};
__device__ __forceinline__ Seq sequence(const PagedAttnParams &p, int b) {
  const int q0 = min(max(p.cache.cu_seqlens[b], 0), p.total_q);
  const int q1 = min(max(p.cache.cu_seqlens[b + 1], q0), p.total_q);
  const int max_keys = p.cache.max_pages << p.page_log2;  // at most 2^30
  return {q0, q1 - q0, min(max(p.cache.kv_lens[b], 0), max_keys)};
}

__device__ __forceinline__ int row_blocks(const PagedAttnParams &p, const Seq &s) {
  return (s.q_len + 2 * p.tok - 1) / (2 * p.tok);
}

// Key tiles seen by the tokens before `end` of a sequence (end > 0).
__device__ __forceinline__ int tiles_seen(const PagedAttnParams &p, const Seq &s, int end) {
  const int keys = p.causal ? s.kv_len - s.q_len + min(end, s.q_len) : s.kv_len;
  return keys <= 0 ? 0 : (keys + kRowsPerTile - 1) / kRowsPerTile;
}
__device__ __forceinline__ int item_tiles(const PagedAttnParams &p, const Seq &s, int rb) {
  return tiles_seen(p, s, (rb + 1) * 2 * p.tok);
}

// sum_{i=0}^{n-1} floor((a i + b) / m), a and m at most 256 (the lattice points
// under a line, by the Euclidean algorithm on a and m). Divisions of 32 bits
// wherever the numbers have no more: with 64 throughout, the sums over a batch of
// prompt pieces took 3,800 clocks of every CTA's start.
__device__ __forceinline__ long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  long long sum = 0;
  while (n > 0) {
    const unsigned whole_a = a / m, whole_b = b / m;
    sum += static_cast<long long>(n) * (n - 1) / 2 * whole_a + static_cast<long long>(n) * whole_b;
    a -= whole_a * m;
    b -= whole_b * m;
    const unsigned long long top = static_cast<unsigned long long>(a) * n + b;
    if (top < m) break;
    n = top >> 32 ? static_cast<unsigned>(top / m) : static_cast<unsigned>(top) / m;
    b = static_cast<unsigned>(top - static_cast<unsigned long long>(n) * m);
    const unsigned t = m;
    m = a;
    a = t;
  }
  return sum;
}

// The cost of an item is its key tiles and kItemCost more, for what comes once
// per item: Q, the first scores' and the last product's way through the empty
// pipeline, the epilogue (about 12,000 clocks, of 3,000 a tile; with 2, 4, 6, 8 a
// batch of prompt pieces took 190, 174, 173, 177 us and a small cross attention
// 37.0, 36.4, 37.5, 39.3). An item that sees no key costs nothing.
constexpr int kItemCost = 4;
// Cost of a narrow tile in wide ones, as the two share the machine. Five mixes of
// 31 to 200 single tokens with prompt pieces took in all, at 0.5, 0.6, 0.65, 0.7,
// 0.75, 1: 1,138, 1,085, 1,074, 1,080, 1,127, 1,345 us with heads of 128; at 0.4,
// 0.55, 0.65, 0.75, 1: 933, 855, 833, 878, 1,027 us with heads of 64.
constexpr float kNarrowUnit = 0.65f;
__device__ __forceinline__ int item_cost(int tiles) { return tiles > 0 ? tiles + kItemCost : 0; }

// Cost of the items before row block `rb` of one KV head of a sequence.
__device__ __forceinline__ long long cost_before(const PagedAttnParams &p, const Seq &s, int rb) {
  if (rb <= 0 || s.kv_len <= 0) return 0;
  const int rbs = row_blocks(p, s);
  rb = min(rb, rbs);
  if (rbs == 1) return item_cost(tiles_seen(p, s, s.q_len));
  if (!p.causal) return static_cast<long long>(rb) * item_cost(tiles_seen(p, s, s.q_len));
  // row block i < rbs - 1 sees ceil((c + i w) / 128) tiles, w = 2 tok rows, where c + i w > 0
  const int w = 2 * p.tok, n = min(rb, rbs - 1);
  const int c = s.kv_len - s.q_len + w;
  long long sum = 0;
  const int first = c > 0 ? 0 : (-c) / w + 1;  // first block that sees a key
  if (first < n)
    sum = floor_sum(n - first, kRowsPerTile, w, c + first * w + kRowsPerTile - 1) + static_cast<long long>(n - first) * kItemCost;
  if (rb == rbs) sum += item_cost(tiles_seen(p, s, s.q_len));
  return sum;
}

// The line of costs that a CTA works on: the narrow form's or the wide one's.
struct Line {
  bool narrow;
  int total, n_ctas, first_cta;  // its cost, and its CTAs
  int rows;                      // most rows of a narrow sequence
};

// Rows per KV head up to which a sequence is the narrow form's.
constexpr int kNarrowRows = 64;
__device__ __forceinline__ bool is_narrow(const PagedAttnParams &p, const Seq &s) {
  return s.q_len <= kNarrowRows && s.q_len * p.G <= kNarrowRows && gridDim.x > 1;
}

// Deals the grid's CTAs, the first ones to the narrow form, so that the later of
// the two ends as early as it can.
__device__ __forceinline__ Line line_of(int narrow_total, int wide_total, int rows) {
  const int n = gridDim.x;
  if (wide_total <= 0 || narrow_total <= 0) return {wide_total <= 0, max(wide_total, narrow_total), n, 0, rows};
  const float a = static_cast<float>(narrow_total) * kNarrowUnit, b = static_cast<float>(wide_total);
  int wide = max(1, min(n - 1, static_cast<int>(n * (b / (a + b)))));
  if (wide < n - 1 && fmaxf(a / (n - wide), b / wide) > fmaxf(a / (n - wide - 1), b / (wide + 1))) ++wide;
  const bool narrow = static_cast<int>(blockIdx.x) < n - wide;
  return {narrow, narrow ? narrow_total : wide_total, narrow ? n - wide : wide, narrow ? 0 : n - wide, rows};
}

// The CTA's line, and prefix[0 .. B]: cost in it of all KV heads of the sequences
// before each; by every thread of the CTA. sums has 36 entries.
__device__ __forceinline__ Line prefix_costs(const PagedAttnParams &p, int *prefix, int *sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int B = p.cache.B, per = (B + kThreads - 1) / kThreads;
  const int b0 = min(B, static_cast<int>(threadIdx.x) * per), b1 = min(B, b0 + per);
  int narrow = 0, wide = 0, rows = 0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = sequence(p, b);
    const int cost = s.q_len > 0 ? static_cast<int>(cost_before(p, s, row_blocks(p, s))) * p.cache.Hkv : 0;
    if (is_narrow(p, s)) {
      rows = max(rows, s.q_len * p.G);
      narrow += cost;
      prefix[b] = cost;
    } else {
      wide += cost;
      prefix[b] = -cost;
    }
  }
  int narrow_incl = narrow, wide_incl = wide;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, narrow_incl, off), y = __shfl_up_sync(0xffffffffu, wide_incl, off);
    if (lane >= off) {
      narrow_incl += x;
      wide_incl += y;
    }
  }
  rows = __reduce_max_sync(0xffffffffu, rows);
  if (lane == 31) {
    sums[warp] = narrow_incl;
    sums[12 + warp] = wide_incl;
    sums[24 + warp] = rows;
  }
  __syncthreads();
  const bool one = lane < kThreads / 32;
  const int of_narrow = one ? sums[lane] : 0, of_wide = one ? sums[12 + lane] : 0;
  const Line line = line_of(__reduce_add_sync(0xffffffffu, of_narrow), __reduce_add_sync(0xffffffffu, of_wide),
                               __reduce_max_sync(0xffffffffu, one ? sums[24 + lane] : 0));
  int at = __reduce_add_sync(0xffffffffu, lane < warp ? (line.narrow ? of_narrow : of_wide) : 0) +
           (line.narrow ? narrow_incl - narrow : wide_incl - wide);
  for (int b = b0; b < b1; ++b) {
    const int cost = line.narrow ? prefix[b] : -prefix[b];
    prefix[b] = at;
    at += max(cost, 0);
  }
  if (threadIdx.x == kThreads - 1) prefix[B] = at;
  __syncthreads();
  return line;
}

// The sequence whose range of the line of all costs has `pos`.
__device__ __forceinline__ int seq_of(const int *prefix, int B, int pos) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= pos) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Cost per CTA of a launch of n_ctas.
__device__ __forceinline__ int cost_per_cta(int total, int n_ctas) { return total / n_ctas + (total % n_ctas != 0); }

// An item and the cost before a position within it, found by a warp.
struct Place {
  int b, h, rb, r;
};
__device__ __forceinline__ Place place_of(const PagedAttnParams &p, const int *prefix, int pos, Seq &s) {
  const int b = seq_of(prefix, p.cache.B, pos);
  s = sequence(p, b);
  const int per_head = max(1, (prefix[b + 1] - prefix[b]) / p.cache.Hkv);
  // (the bounds matter only if cu_seqlens decreases, when costs need not fit 32 bits)
  const int off = max(0, pos - prefix[b]), h = min(off / per_head, p.cache.Hkv - 1);
  int rest = off - h * per_head;
  const int rbs = row_blocks(p, s);
  if (rbs == 1) return {b, h, 0, rest};
  const int lane = threadIdx.x & 31;
  for (int rb = 0; rb < rbs; rb += 32) {
    const int n = rb + lane < rbs ? item_cost(item_tiles(p, s, rb + lane)) : 0;
    int incl = n;
#pragma unroll
    for (int step = 1; step < 32; step <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, step);
      if (lane >= step) incl += y;
    }
    const unsigned behind = __ballot_sync(0xffffffffu, rest < incl);
    if (behind != 0) {
      const int at = __ffs(behind) - 1;
      return {b, h, rb + at, rest - __shfl_sync(0xffffffffu, incl - n, at)};
    }
    rest -= __shfl_sync(0xffffffffu, incl, 31);
  }
  return {b, h, rbs, rest};
}

// A CTA's part of one work item: key tiles [j0, j1) of row block rb. The first
// kItemCost units of an item's stretch of the line stand for no tile.
struct Segment {
  Seq s;
  int b, rbs, h, rb, j0, j1;  // rbs: row blocks of the sequence
  int slot;  // partial written, -1: the whole item, written directly
  int next;  // position of the line behind the segment
  int ring;  // the first K tile's place in the order of all tiles of the CTA
};
static_assert(sizeof(Segment) == 48, "its place in shared memory");
__device__ __forceinline__ const int *page_row(const PagedAttnParams &p, const Segment &g) {
  return p.cache.page_table + g.b * p.cache.table_stride;
}

// Walks the segments of a CTA's range of the line in order: the producer does,
// from the first one on (g, when next is called first), and hands them on.
struct Walk {
  int pos, end, per;
  int first_cta, last_cta;  // of the line
  bool fresh, narrow;
  __device__ __forceinline__ explicit Walk(const Line &line) : fresh(true), narrow(line.narrow) {
    per = cost_per_cta(line.total, line.n_ctas);
    first_cta = line.first_cta;
    last_cta = line.first_cta + line.n_ctas - 1;
    const long long total = line.total;
    pos = static_cast<int>(min(static_cast<long long>(per) * (static_cast<int>(blockIdx.x) - first_cta), total));
    end = static_cast<int>(min(static_cast<long long>(pos) + per, total));
  }
  // The segment of row block rb at cost `within` of it, which is position `pos`
  // (j0 == j1 if the range ends before its first tile).
  __device__ __forceinline__ void make(const PagedAttnParams &p, int rb, int within, Segment &g) const {
    const int n = item_tiles(p, g.s, rb), stop = min(n + kItemCost, within + (end - pos));
    g.rb = rb;
    g.j0 = max(0, within - kItemCost);
    g.j1 = max(g.j0, stop - kItemCost);
    g.slot = g.j0 == 0 && g.j1 == n ? -1 : 2 * static_cast<int>(blockIdx.x) + (g.j0 == 0 ? 1 : 0);
    g.next = pos + (stop - within);
  }
  __device__ __forceinline__ bool next(const PagedAttnParams &p, Segment &g) {
    if (pos >= end) return false;
    if (fresh) {
      fresh = false;
      pos = g.next;
      if (g.j1 > g.j0) return true;
    }
    return next_item(p, g);
  }
  __device__ __noinline__ bool next_item(const PagedAttnParams &p, Segment &g) {
    while (pos < end) {
      // the item after the last one, skipping those that see no key
      int rb = g.rb + 1;
      if (rb >= g.rbs) {
        rb = 0;
        if (++g.h >= p.cache.Hkv) {
          g.h = 0;
          do {
            if (++g.b >= p.cache.B) return false;
            g.s = sequence(p, g.b);
          } while (g.s.q_len == 0 || g.s.kv_len == 0 || is_narrow(p, g.s) != narrow);
          g.rbs = row_blocks(p, g.s);
        }
      }
      // (the bounds on b and rb only matter when the lengths change during the
      // call, which must not happen: then the walk ends instead of running on)
      while (rb < g.rbs && item_tiles(p, g.s, rb) == 0) ++rb;
      if (rb >= g.rbs) return false;
      make(p, rb, 0, g);
      pos = g.next;
      if (g.j1 > g.j0) return true;
    }
    return false;
  }
  // The last CTA of an item that this one begins with segment g.
  __device__ __forceinline__ int ends_in(const PagedAttnParams &p, const Segment &g) const {
    return min(first_cta + (g.next - (g.j1 + kItemCost) + item_tiles(p, g.s, g.rb) + kItemCost - 1) / per, last_cta);
  }
  // Key tiles of segment g that query tile t (of the wide form) goes through, counted from g.j0.
  static __device__ __forceinline__ int tiles(const PagedAttnParams &p, const Segment &g, int t) {
    const int first = (2 * g.rb + t) * p.tok;
    if (first >= g.s.q_len) return 0;
    return max(0, min(g.j1, tiles_seen(p, g.s, first + p.tok)) - g.j0);
  }
};

// The segments on their way from the producer to the other roles, in four places
// of shared memory, each with a barrier for "there" and one for "read by every
// warp". (When every role walked by itself that was 1,300 to 3,500 clocks of each
// item in each role.) A segment without tiles ends the CTA's range.
struct Items {
  Segment *places;
  uint32_t bar;  // four for "there", four for "read"
  int i;
  __device__ __forceinline__ Items(Segment *places_, uint32_t bar_) : places(places_), bar(bar_), i(0) {}
  __device__ __forceinline__ uint32_t there() const { return bar + 8u * static_cast<uint32_t>(i & 3); }
  // The next segment, by a whole warp of a role; false at the end and after a timeout.
  __device__ __forceinline__ bool wait(volatile int *abort_flag, int *err) const {
    return __all_sync(0xffffffffu, mbar_wait(there(), static_cast<uint32_t>(i >> 2) & 1u, abort_flag, err)) &&
           places[i & 3].j1 > places[i & 3].j0;
  }
  // The same for the four warps of a role that meet at named barrier `id`: all go on
  // or none does. (One alone may give up after an error elsewhere just before the
  // producer hands the segment on; the others must not take it and wait for that one.)
  __device__ __forceinline__ bool wait_together(int id, volatile int *abort_flag, int *err) const {
    return named_bar_and(id, 128, wait(abort_flag, err));
  }
  __device__ __forceinline__ const Segment &get() const { return places[i & 3]; }
  // This warp has read it.
  __device__ __forceinline__ void release() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(there() + 32u);
    ++i;
  }
  // The producer warp hands on g.
  __device__ __forceinline__ bool put(const Segment &g, volatile int *abort_flag, int *err) {
    if (i >= 4 && !__all_sync(0xffffffffu, mbar_wait(there() + 32u, static_cast<uint32_t>((i >> 2) - 1) & 1u, abort_flag, err)))
      return false;
    if ((threadIdx.x & 31) == 0) {
      places[i & 3] = g;
      mbar_arrive(there());
    }
    __syncwarp();
    ++i;
    return true;
  }
};

// Pages of a key tile: 128 / page_size, or one larger page.
__device__ __forceinline__ int pages_of_tile(const PagedAttnParams &p) {
  return p.page_log2 < 7 ? kRowsPerTile >> p.page_log2 : 1;
}
// Index in the table row of the first page of key tile j.
__device__ __forceinline__ int first_page(const PagedAttnParams &p, int j) { return (j * kRowsPerTile) >> p.page_log2; }
// A lane's entry of the 32 from index `from` on, -1 past the sequence's pages.
__device__ __forceinline__ int window_entry(const PagedAttnParams &p, const int *row, int kv_len, int from) {
  const int i = from + static_cast<int>(threadIdx.x & 31);
  return i <= (kv_len - 1) >> p.page_log2 ? row[i] : -1;
}

// The producer's view of a segment's pages: 32 entries of the table, one a lane,
// and the 32 after them on their way, so that no load's latency is between two
// tiles (it was: 1,300 clocks a tile with pages of 32 keys). The first 32 of
// those are asked for behind the first tile, which does not wait for them.
struct PageWindow {
  const int *row;
  int kv_len, from, now, ahead;
  __device__ __forceinline__ PageWindow(const PagedAttnParams &p, const Segment &g, bool have_first, int first)
      : row(page_row(p, g)), kv_len(g.s.kv_len), from(first_page(p, g.j0)) {
    now = have_first ? first : window_entry(p, row, kv_len, from);
    ahead = -1;
  }
  __device__ __forceinline__ void prefetch(const PagedAttnParams &p) { ahead = window_entry(p, row, kv_len, from + 32); }
  // This lane's page of key tile j (lanes below pages_of_tile): n_pages, which
  // reads as zeros, where there is none. Tiles in ascending order.
  __device__ __forceinline__ int page(const PagedAttnParams &p, int j) {
    const int boxes = pages_of_tile(p), lane = threadIdx.x & 31;
    int off = first_page(p, j) - from;
    if (off >= 32) {  // (a tile's pages are never in two windows)
      __syncwarp();   // a branch, not a choice between `now` and `ahead`: that one would wait for both
      from += 32;
      off -= 32;
      now = ahead;
      ahead = window_entry(p, row, kv_len, from + 32);
    }
    const int e = __shfl_sync(0xffffffffu, now, off + (lane < boxes ? lane : 0));
    return e >= 0 && e < p.cache.n_pages ? e : p.cache.n_pages;
  }
};

// The boxes of a key tile, lane i's page the i-th: issued by one lane, in code that
// is uniform for the warp. (One lane a page took about 110 clocks a box: the
// lanes follow each other, each with its operands on the way to uniform
// registers.)
template <int D, int kBoxes>
__device__ __forceinline__ void load_boxes(uint32_t dst, const CUtensorMap *map, uint32_t bar, int in_page, int head,
                                           int first, int page, uint32_t box_bytes, bool leader, uint64_t pol) {
  int pg[kBoxes];
  dst += first * box_bytes;
#pragma unroll
  for (int i = 0; i < kBoxes; ++i) pg[i] = uniform(__shfl_sync(0xffffffffu, page, first + i));
  if (leader) {
#pragma unroll
    for (int i = 0; i < kBoxes; ++i)
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb)
        tma_load_4d_hint(dst + cb * kColBlockBytes + i * box_bytes, map, bar, cb * 64, in_page, head, pg[i], pol);
  }
  __syncwarp();
}
template <int D>
__device__ __forceinline__ void load_pages(uint32_t dst, const CUtensorMap *map, uint32_t bar, int in_page, int head,
                                           int page, int boxes, uint32_t box_bytes, bool leader, uint64_t pol) {
  if (boxes == 1) {
    load_boxes<D, 1>(dst, map, bar, in_page, head, 0, page, box_bytes, leader, pol);
  } else if (boxes == 2) {
    load_boxes<D, 2>(dst, map, bar, in_page, head, 0, page, box_bytes, leader, pol);
  } else {
#pragma unroll 1
    for (int i = 0; i < boxes; i += 4) load_boxes<D, 4>(dst, map, bar, in_page, head, i, page, box_bytes, leader, pol);
  }
}

// Whether a page of a segment's key tiles is missing, found by a warp at the
// segment's start, so that the tiles of a whole sequence look nothing up.
__device__ __forceinline__ bool pages_missing(const PagedAttnParams &p, const Segment &g) {
  const int lane = threadIdx.x & 31;
  const int first = (g.j0 * kRowsPerTile) >> p.page_log2;
  const int end = (min(g.j1 * kRowsPerTile, g.s.kv_len) + (1 << p.page_log2) - 1) >> p.page_log2;
  const int *row = page_row(p, g);
  bool missing = false;
#pragma unroll 8
  for (int i = first + lane; i < end; i += 32)
    missing |= static_cast<unsigned>(row[i]) >= static_cast<unsigned>(p.cache.n_pages);
  return __any_sync(0xffffffffu, missing);
}
// The pages of key tile j that are there, one bit each (set past them).
__device__ __forceinline__ unsigned pages_there(const PagedAttnParams &p, const int *row, int kv_len, int j) {
  const int lane = threadIdx.x & 31;
  const bool small = p.page_log2 < 7;
  const int i = small ? j * (kRowsPerTile >> p.page_log2) + lane : (j * kRowsPerTile) >> p.page_log2;
  bool there = true;
  if (lane < (small ? kRowsPerTile >> p.page_log2 : 1) && (i << p.page_log2) < kv_len)
    there = static_cast<unsigned>(row[i]) < static_cast<unsigned>(p.cache.n_pages);
  return __ballot_sync(0xffffffffu, there);
}

// V slots past kv_len may hold anything, NaN too, and 0 * NaN would reach O:
// they are zeroed in shared memory, by the 128 threads of a warpgroup, before
// the product reads them. The tile (at shared address v, its barrier and phase
// given) stays until the products that use it are done.
template <int D>
__device__ __forceinline__ bool clear_tail(int valid_keys, uint32_t v, uint32_t bar_full, uint32_t phase,
                                           volatile int *abort_flag, int *err) {
  if (!__all_sync(0xffffffffu, mbar_wait(bar_full, phase, abort_flag, err))) return false;
  const int pieces = (kRowsPerTile - valid_keys) * 8;  // 16-byte pieces of a 128-byte column block
  for (int i = threadIdx.x & 127; i < pieces * (D / 64); i += 128)
    st_shared_v4(v + (i / pieces) * kColBlockBytes + valid_keys * 128 + (i % pieces) * 16, 0u, 0u, 0u, 0u);
  fence_proxy_async_shared();
  return true;
}

// O rows of TMEM by alpha (this thread's row; its warp all together).
template <int D>
__device__ __forceinline__ void scale_o(uint32_t o_addr, float alpha) {
#pragma unroll 1
  for (int cb = 0; cb < D / 32; ++cb) {
    uint32_t v[32];
    tmem_ld32(o_addr + 32 * cb, v);
    tmem_ld_wait(v);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
    tmem_st32(o_addr + 32 * cb, v);
  }
  tmem_st_wait();
}

// Rows of the items that see no key at all (every row, if `all`): O = 0, lse = -inf.
template <int D>
__device__ __noinline__ void write_unseen(const PagedAttnParams &p, bool all, int tid, int nthreads) {
  for (int b = blockIdx.x; b < p.cache.B; b += gridDim.x) {
    const Seq s = sequence(p, b);
    const int rbs = row_blocks(p, s);
    int rb = 0;
    while (rb < rbs && item_tiles(p, s, rb) == 0) ++rb;
    const int toks = all ? s.q_len : min(s.q_len, rb * 2 * p.tok);
    for (long long i = tid; i < static_cast<long long>(toks) * p.Hq * (D / 8); i += nthreads) {
      const int c = static_cast<int>(i % (D / 8));
      const int head = static_cast<int>(i / (D / 8) % p.Hq), row = s.q0 + static_cast<int>(i / (D / 8) / p.Hq);
      *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + head * p.o_h + row * p.o_s + 8 * c) =
          make_uint4(0u, 0u, 0u, 0u);
      if (c == 0 && p.lse) p.lse[static_cast<size_t>(head) * p.total_q + row] = -INFINITY;
    }
  }
}

// ---------------------------------------------------------------- the wide form's roles
template <int D>
struct WideBars {
  static constexpr int kStages = Cfg<D>::kStages;
  static constexpr int kQFull = 0, kQEmpty = 1, kFull = 2, kEmpty = 2 + kStages, kSFull = 2 + 2 * kStages,
                       kPFull = kSFull + 2, kOFull = kPFull + 2, kMmaDone = kOFull + 2;
};
// TMEM columns of S_t / P_t and of O_t
__device__ __forceinline__ uint32_t s_column(uint32_t tmem, int t) { return tmem + 128u * static_cast<uint32_t>(t); }
__device__ __forceinline__ uint32_t o_column(uint32_t tmem, int t) { return tmem + 256u + 128u * static_cast<uint32_t>(t); }

// Producer: the whole warp. sQ [tile][col block][128 rows][128 B], sRing
// [slot][col block][128 rows][128 B].
template <int D>
__device__ __forceinline__ void wide_producer(const PagedAttnParams &p, Walk walk, Segment g, Items items,
                                           const CUtensorMap *tm_q,
                                           const CUtensorMap *tm_k, const CUtensorMap *tm_v, uint32_t bar0, uint32_t sQ,
                                           uint32_t sRing, int first_entry, volatile int *abort_flag, int *err) {
  using C = Cfg<D>;
  using W = WideBars<D>;
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  // K and V are read again by the other row blocks of their sequence, Q is not
  const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
  const int page_size = 1 << p.page_log2;
  const bool small = page_size < kRowsPerTile;
  const int boxes = uniform(pages_of_tile(p));
  const uint32_t box_bytes = uniform((small ? page_size : kRowsPerTile) * 128u);
  const bool leader = elect_one();
  auto wait = [&](int i, uint32_t phase) {
    return __all_sync(0xffffffffu, mbar_wait(bar(i), phase, abort_flag, err));
  };
  int c = 0, nq = 0;
  bool ok = true;
  // the item that this CTA begins and another one ends, for the merge
  int4 cut = make_int4(0, 0, 0, 0);
  while (ok && walk.next(p, g)) {
    g.ring = c;
    if (!items.put(g, abort_flag, err)) break;
    if (g.j0 == 0 && g.slot >= 0)
      cut = make_int4(g.s.q0 + g.rb * 2 * p.tok, min(2 * p.tok, g.s.q_len - g.rb * 2 * p.tok) * p.G, g.h, walk.ends_in(p, g));
    const int n_max = uniform(max(Walk::tiles(p, g, 0), Walk::tiles(p, g, 1)));
    const int j0 = uniform(g.j0), head = uniform(g.h);
    const bool two = Walk::tiles(p, g, 1) > 0;
    PageWindow pages(p, g, nq == 0, first_entry);
    ok = nq == 0 || wait(W::kQEmpty, (nq - 1) & 1);
    if (!ok) break;
    if (leader) {
      const uint32_t q_bytes = static_cast<uint32_t>(p.tok * p.G) * 128u * C::kColBlocks;
      mbar_arrive_expect_tx(bar(W::kQFull), two ? 2 * q_bytes : q_bytes);
      for (int t = 0; t < (two ? 2 : 1); ++t)
        for (int cb = 0; cb < C::kColBlocks; ++cb)
          tma_load_4d_hint(sQ + (t * C::kColBlocks + cb) * kColBlockBytes, tm_q, bar(W::kQFull), cb * 64, 0,
                           g.s.q0 + (2 * g.rb + t) * p.tok, head, pol_q);
    }
    __syncwarp();
    ++nq;
    for (int j = 0; j < n_max && ok; ++j) {
      const int page = pages.page(p, j0 + j);
      const int in_page = small ? 0 : ((j0 + j) * kRowsPerTile) & (page_size - 1);
      for (int which = 0; which < 2; ++which, ++c) {
        const int slot = c % C::kStages;
        ok = c < C::kStages || wait(W::kEmpty + slot, ((c / C::kStages) - 1) & 1);
        if (!ok) break;
        if (leader) mbar_arrive_expect_tx(bar(W::kFull + slot), C::kTileBytes);
        load_pages<D>(sRing + slot * C::kTileBytes, which ? tm_v : tm_k, bar(W::kFull + slot), in_page, head, page, boxes,
                      box_bytes, leader, pol_kv);
        if (j == 0 && which == 1) pages.prefetch(p);
      }
    }
  }
  g.j0 = g.j1 = 0;
  items.put(g, abort_flag, err);
  if (lane == 0) p.cuts[blockIdx.x] = cut;
  if (lane == 0) {  // every copy must have landed before the CTA may exit
    if (nq > 0) mbar_drain(bar(W::kQFull), (nq - 1) & 1, err);
    for (int i = max(0, c - C::kStages); i < c; ++i)
      mbar_drain(bar(W::kFull + i % C::kStages), (i / C::kStages) & 1, err);
  }
  __syncwarp();
}

// MMA issuer of query tile t (the dense forward's scheme): the whole warp, its
// code uniform, one lane for the products. (As the code of a single thread it
// took about 95 clocks an MMA to bring the operands into uniform registers,
// longer than the MMA itself; both issuers take turns, so that was the time of a
// key tile.)
template <int D>
__device__ __forceinline__ void wide_issuer(const PagedAttnParams &p, Items items, int t_in, uint32_t bar0, uint32_t sQ,
                                            uint32_t sRing, uint32_t tmem_in, volatile int *turn,
                                            volatile int *abort_flag, int *err) {
  using C = Cfg<D>;
  using W = WideBars<D>;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  auto wait = [&](int i, uint32_t phase) {
    return __all_sync(0xffffffffu, mbar_wait(bar(i), phase, abort_flag, err));
  };
  const bool leader = elect_one();
  const int t = uniform(t_in);
  const uint32_t tmem = uniform(tmem_in);
  constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false), idesc_o = idesc_bf16_f32(128, D, true);
  const uint64_t qd = sw128_desc(sQ + t * C::kTileBytes, 16, 1024);
  const uint32_t s_col = s_column(tmem, t), o_col = o_column(tmem, t);
  uint32_t nq = 0, steps = 0;
  int base = 0;
  bool ok = true;
  while (ok && items.wait(abort_flag, err)) {
    const int n0 = uniform(Walk::tiles(p, items.get(), 0)), n1 = uniform(Walk::tiles(p, items.get(), 1));
    const uint32_t c = uniform(items.get().ring);
    items.release();
    const int nt = t == 0 ? n0 : n1, n_max = max(n0, n1);
    // tile 1 has nothing to do: its issuer only gives Q back, and tile 0's
    // goes on without taking turns and releases each slot for both
    const bool single = n1 == 0;
    if (!wait(W::kQFull, nq & 1)) break;
    ++nq;
    if (nt == 0 && leader) mma_commit(bar(W::kQEmpty));
    __syncwarp();
    if (single && t == 1) continue;
    for (int j = 0; ok && j <= n_max; ++j) {
      const uint32_t cK = c + 2 * j, cV = c + 2 * j - 1;  // ring positions of K_j and V_{j-1}
      const uint32_t sK = cK % C::kStages, sV = cV % C::kStages;
      const uint32_t cV2 = cK + 1, sV2 = cV2 % C::kStages;
      const uint64_t kd = sw128_desc(sRing + sK * C::kTileBytes, 16, 1024);
      const uint64_t vd = sw128_desc(sRing + sV * C::kTileBytes, kColBlockBytes, 1024);
      const bool has_pv = j >= 1 && j - 1 < nt, has_s = j < nt, unused = !has_s && j < n_max;
      if ((has_s || unused) && !wait(W::kFull + sK, (cK / C::kStages) & 1)) {
        ok = false;
        break;
      }
      if (unused && !wait(W::kFull + sV2, (cV2 / C::kStages) & 1)) {
        ok = false;
        break;
      }
      if (has_pv && (!wait(W::kFull + sV, (cV / C::kStages) & 1) || !wait(W::kPFull + t, (steps + j - 1) & 1))) {
        ok = false;
        break;
      }
      const int turn_at = base + 2 * j + t;
      if (!single && !__all_sync(0xffffffffu, wait_turn(turn, turn_at, abort_flag, err))) {
        ok = false;
        break;
      }
      if (has_pv) {
        tc_fence_after();
        const uint32_t add = j > 1 ? 1u : 0u;
        if (leader) {
          mma_ts(o_col, s_col, vd, idesc_o, add);
#pragma unroll
          for (int kk = 1; kk < kRowsPerTile / 16; ++kk)
            mma_ts(o_col, s_col + kk * 8, vd + static_cast<uint64_t>(kk * 128), idesc_o, 1u);
        }
        __syncwarp();
      }
      if (has_s) {
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = static_cast<uint64_t>(((kk / 4) * kColBlockBytes + (kk % 4) * 32) >> 4);
            mma_ss(s_col, qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
          }
        }
        __syncwarp();
      }
      if (leader) {
        if (!single) *turn = turn_at + 1;
        if (has_s) mma_commit(bar(W::kSFull + t));
        if (has_pv) {
          if (j - 1 == nt - 1) mma_commit(bar(W::kOFull + t));
          mma_commit(bar(W::kEmpty + sV));
          if (single) mma_commit(bar(W::kEmpty + sV));
        }
        if (has_s) {
          mma_commit(bar(W::kEmpty + sK));
          if (single) mma_commit(bar(W::kEmpty + sK));
          if (j == nt - 1) mma_commit(bar(W::kQEmpty));
        }
        if (unused) {
          mma_commit(bar(W::kEmpty + sK));
          mma_commit(bar(W::kEmpty + sV2));
        }
      }
      __syncwarp();
    }
    steps += nt;
    if (!single) base += 2 * (n_max + 1);
  }
  if (leader) {
    mma_commit(bar(W::kMmaDone));
    mbar_drain(bar(W::kMmaDone), 0, err);
  }
  __syncwarp();
}

constexpr int kStageBytes = 2560;  // of a softmax warp's epilogue: 32 rows, 80 bytes apart

// x, in a way that nothing computed from it moves ahead of this place: what the
// ends of a segment need must not sit in registers through its main loop.
__device__ __forceinline__ int hidden(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

// Softmax warpgroup of query tile t: a thread has one row (TMEM lane = tile row),
// the dense forward's scheme. It reads its segment where the producer put it (with
// it in registers the main loop spilled, 15 % of the time of a long causal
// prompt). stage_in: this warp's kStageBytes of shared memory.
template <int D>
__device__ __forceinline__ void wide_softmax(const PagedAttnParams &p, Items items, int t, uint32_t bar0,
                                             uint32_t sRing, uint32_t tmem, uint32_t stage_in, volatile int *abort_flag,
                                             int *err) {
  using C = Cfg<D>;
  using W = WideBars<D>;
  const int lane = threadIdx.x & 31;
  const int r = threadIdx.x & 127;
  const uint32_t bar_t = bar0 + 8u * t;
  const uint32_t lane_off = static_cast<uint32_t>(r & ~31) << 16;
  const uint32_t s_addr = s_column(tmem, t) + lane_off, o_addr = o_column(tmem, t) + lane_off;
  uint32_t steps = 0;  // key tiles of this query tile so far
  uint32_t u = 0;      // segments in which it had any
  while (items.wait(abort_flag, err)) {
    const Segment &seg = items.get();
    const int n = Walk::tiles(p, seg, t);
    int first_key, row_rel, cut_from, tail_from;
    bool row_valid, holes;
    {
      const int first = (2 * seg.rb + t) * p.tok;  // the tile's first token within the sequence
      const int tok = hidden(r) / p.G, kv_len = seg.s.kv_len;
      row_valid = r < p.tok * p.G && first + tok < seg.s.q_len;
      // last key of the tile's first token, and of this row (rows of no token --
      // zeros, or other sequences' rows -- see every key: nothing of them is written)
      const int tile_last = p.causal ? kv_len - seg.s.q_len + first : kv_len - 1;
      const int row_last = row_valid && p.causal ? min(tile_last + tok, kv_len - 1) : kv_len - 1;
      first_key = seg.j0 * kRowsPerTile;
      row_rel = row_last - first_key;
      cut_from = (tile_last + 1 - first_key) >> 7;   // the first tile of which some row does not see all keys
      tail_from = (kv_len - first_key) >> 7;         // the tile that the sequence ends in
      holes = n > 0 && pages_missing(p, seg);     // pages have to be looked up tile by tile
    }
    const bool warp_valid = __any_sync(0xffffffffu, row_valid);
    const float c2 = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const unsigned there =
          holes ? pages_there(p, page_row(p, seg), seg.s.kv_len, seg.j0 + j) : 0xffffffffu;
      ok = __all_sync(0xffffffffu, mbar_wait(bar_t + 8u * W::kSFull, (steps + j) & 1u, abort_flag, err));
      if (!ok) break;
      tc_fence_after();
      if (warp_valid) {
        const bool cut = j >= cut_from;
        const int last = row_rel - j * kRowsPerTile;  // the last key of the tile that this row sees
        auto mask_scores = [&](uint32_t *x, int c0, int cols) {
          if (cut) {
#pragma unroll
            for (int c = 0; c < cols; ++c)
              if (c0 + c > last) x[c] = __float_as_uint(-INFINITY);
          }
          if (there != 0xffffffffu) {
            const int shift = p.page_log2 < 7 ? p.page_log2 : 31;  // a larger page: bit 0
#pragma unroll
            for (int c = 0; c < cols; ++c)
              if (!((there >> ((c0 + c) >> shift)) & 1u)) x[c] = __float_as_uint(-INFINITY);
          }
        };
        auto load_scores = [&](uint32_t(&sr)[128]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(s_addr + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * i]));
          tmem_ld_wait(sr);
          mask_scores(sr, 0, 128);
        };
        uint32_t pk[64];
        uint32_t sr[128];
        load_scores(sr);
        float rowsum;
        // A row that has seen no key yet takes this tile's maximum as its reference:
        // in the first tile, and behind tiles whose pages are all missing. (2^s of
        // scores left without a reference is 0 below -126 and would lose their
        // keys.) O is 0 or not yet written then, and needs no factor.
        if (m == -INFINITY) m = row_max(reinterpret_cast<const float *>(sr)) * c2;
        rowsum = exp_row<false, 0>(reinterpret_cast<const float *>(sr), c2, (m == -INFINITY) ? 0.f : m, pk);
        if (j > 0) {
          // as in the dense forward: the reference moves, and O with it, only
          // when the tile's P would sum to more than 2^8
          const bool big = row_valid && !(rowsum <= kRescaleSum);
          if (__any_sync(0xffffffffu, big)) {
            float mx = -INFINITY;  // 32 columns at a time: few live registers
#pragma unroll 1
            for (int cb = 0; cb < 4; ++cb) {
              uint32_t x[32];
              tmem_ld32(s_addr + 32 * cb, x);
              tmem_ld_wait(x);
              mask_scores(x, 32 * cb, 32);
#pragma unroll
              for (int c = 0; c < 32; ++c) mx = fmaxf(mx, __uint_as_float(x[c]));
            }
            const float m_new = fmaxf(m, mx * c2);
            const float alpha = (m_new == -INFINITY) ? 1.f : ex2_approx(m - m_new);
            m = m_new;
            l *= alpha;
            scale_o<D>(o_addr, alpha);
            load_scores(sr);
            rowsum = exp_row<false, 0>(reinterpret_cast<const float *>(sr), c2, (m == -INFINITY) ? 0.f : m, pk);
          }
        }
        l += rowsum;
        tmem_st32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
        tmem_st32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
        tmem_st_wait();
      }
      if (j >= tail_from) {
        const int cv = seg.ring + 2 * j + 1, slot = cv % C::kStages;  // ring position of the V tile
        ok = clear_tail<D>(seg.s.kv_len - first_key - j * kRowsPerTile, sRing + slot * C::kTileBytes,
                           bar0 + 8u * (W::kFull + slot), (cv / C::kStages) & 1, abort_flag, err);
        if (!ok) break;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_t + 8u * W::kPFull);  // one arrival per warp
    }
    // what the epilogue needs of the segment
    const int slot = seg.slot, h = seg.h, q0 = seg.s.q0 + (2 * seg.rb + t) * p.tok;
    steps += n;
    items.release();
    bool have_o = false;
    if (ok && n > 0) {
      have_o = __all_sync(0xffffffffu, mbar_wait(bar_t + 8u * W::kOFull, u & 1u, abort_flag, err));
      tc_fence_after();
      ++u;
    }
    if (!ok || (n > 0 && !have_o)) return;  // (a warp that gives up makes the others give up too)
    if (!warp_valid) continue;
    // (not l > 0: the NaN of a row with a NaN score must not look like a row without keys)
    const float inv_l = l != 0.f ? 1.f / l : 0.f;
    const float lse = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    const unsigned valid = __ballot_sync(0xffffffffu, row_valid);
    // Rows leave through shared memory, 64 bytes of each at a time, so that a
    // store instruction writes 64 bytes of eight rows (each lane its own row, 16
    // bytes at a time, cost twice the sectors and 10,000 clocks a segment; this
    // 4,500 to 7,500). `stage`: 32 rows of this warp, 80 bytes apart.
    const int ln = hidden(lane), rr = hidden(r);
    const uint32_t stage = stage_in, mine = stage + ln * 80u;
    const int sub = ln >> 2, quad = ln & 3;
    long long off;  // this lane's row in the output, elements
    if (slot >= 0) {
      const size_t at = static_cast<size_t>(slot) * p.part_rows + t * p.tok * p.G + rr;
      if (row_valid) p.part_lse[at] = lse;
      if (!have_o) continue;  // no key seen: the merge does not read O
      off = static_cast<long long>(at) * D;
      uint32_t v[16];
      tmem_ld16(o_addr, v);
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 16) {
        tmem_ld_wait(v);
        __syncwarp();  // the stage has been read
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st_shared_v4(mine + 16 * i, __float_as_uint(__uint_as_float(v[4 * i]) * inv_l),
                       __float_as_uint(__uint_as_float(v[4 * i + 1]) * inv_l),
                       __float_as_uint(__uint_as_float(v[4 * i + 2]) * inv_l),
                       __float_as_uint(__uint_as_float(v[4 * i + 3]) * inv_l));
        if (c0 + 16 < D) tmem_ld16(o_addr + c0 + 16, v);  // the next columns meanwhile
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 8 * i + sub;
          const long long to = __shfl_sync(0xffffffffu, off, row);
          const uint4 x = ld_shared_v4(stage + row * 80u + quad * 16u);
          if ((valid >> row) & 1u) *reinterpret_cast<uint4 *>(p.part_o + to + c0 + 4 * quad) = x;
        }
      }
      tmem_ld_wait(v);
      __syncwarp();
      continue;
    }
    const int head = h * p.G + rr % p.G, row_at = q0 + rr / p.G;
    if (row_valid && p.lse) p.lse[static_cast<size_t>(head) * p.total_q + row_at] = lse;
    off = head * p.o_h + row_at * p.o_s;
    uint32_t v[32];
    if (have_o) {
      tmem_ld32(o_addr, v);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0u;
    }
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
      tmem_ld_wait(v);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // the one rounding of O to its own type
          __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(v[8 * i + 2 * k]) * inv_l,
                                                   __uint_as_float(v[8 * i + 2 * k + 1]) * inv_l);
          w[k] = *reinterpret_cast<uint32_t *>(&x);
        }
        st_shared_v4(mine + 16 * i, w[0], w[1], w[2], w[3]);
      }
      if (have_o && c0 + 32 < D) tmem_ld32(o_addr + c0 + 32, v);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + sub;
        const long long to = __shfl_sync(0xffffffffu, off, row);
        const uint4 x = ld_shared_v4(stage + row * 80u + quad * 16u);
        if ((valid >> row) & 1u)
          *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + to + c0 + 8 * quad) = x;
      }
    }
    tmem_ld_wait(v);
    __syncwarp();
  }
}

}  // namespace paged
}  // namespace seqattn

#include "attn_paged_narrow.cuh"

namespace seqattn {
namespace paged {

// Query maps by the tokens of their box: a wide tile's, and 16, 32, 64 rows'.
struct QueryMaps {
  CUtensorMap wide, narrow[3];
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_paged_kernel(const __grid_constant__ QueryMaps tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedAttnParams p) {
  using C = Cfg<D>;
  using L = Narrow<D>;
  using W = WideBars<D>;
  static_assert(L::kAreaBytes <= C::kAreaBytes && L::kNumBarriers <= C::kItemBarrier && W::kMmaDone < C::kItemBarrier,
                "shared memory layout");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem =
      reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kAreaBytes);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::kMaxBarriers);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *turn = reinterpret_cast<volatile int *>(tmem_slot + 2);  // next MMA burst slot (wide)
  Segment *places = reinterpret_cast<Segment *>(tmem_slot + 4);
  float *red = reinterpret_cast<float *>(places + 4);
  int *warp_sums = reinterpret_cast<int *>(red);
  int *prefix = reinterpret_cast<int *>(smem + C::kPrefixAt);
  const uint32_t bar0 = smem_addr(bars), base = smem_addr(smem);
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int *err = &g_device_error;

  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  if (threadIdx.x == kTmaWarp * 32) {
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
  }
  wait_prerequisites();  // nothing of the tensors or the workspace is touched before
  // an earlier timeout, not yet cleared by the host: this CTA skips its work
  // and its rows come out as O = 0, lse = -inf
  const bool failed = warp == kMmaWarp1 && *reinterpret_cast<volatile int *>(err) != kErrNone;
  const Line line = prefix_costs(p, prefix, warp_sums);
  const bool narrow = line.narrow;
  const L sh(line.rows, p.G);
  const Walk walk(line);
  const Items items(places, bar(C::kItemBarrier));
  Segment first = {};    // the producer's
  int first_entry = -1;  // the producer's lanes: the first pages
  if (warp == kTmaWarp && walk.pos < walk.end) {
    const Place at = place_of(p, prefix, walk.pos, first.s);
    first.b = at.b;
    first.h = at.h;
    first.rbs = row_blocks(p, first.s);
    walk.make(p, at.rb, at.r, first);
    first_entry = window_entry(p, page_row(p, first), first.s.kv_len, first_page(p, first.j0));
  }
  if (warp == kMmaWarp1) {
    // a barrier a lane (one thread for all of them: 1,400 clocks)
    for (int i = lane; i < (narrow ? L::kNumBarriers : C::kNumBarriers); i += 32) {
      int arrivals = 1;
      if (narrow) {
        if (i == L::kPFull || i == L::kPFull + 1) arrivals = 4 * sh.groups;
      } else {
        if (i == W::kQEmpty || i == W::kMmaDone || (i >= W::kEmpty && i < W::kEmpty + C::kStages)) arrivals = 2;
        if (i == W::kPFull || i == W::kPFull + 1) arrivals = 4;
      }
      mbar_init(bar(i), arrivals);
    }
    // read by the issuer(s) and the softmax warps
    if (lane < 8) mbar_init(bar(C::kItemBarrier + lane), lane < 4 ? 1 : (narrow ? 1 + 4 * sh.groups : 10));
    if (lane == 0) {
      *abort_flag = failed;
      *turn = 0;
    }
    fence_barrier_init();
  }
  if (warp != kTmaWarp) {
    // rows of Q that no token fills: zeros, not whatever was there
    const uint32_t at = base + (narrow ? sh.q_at() : 0);
    const int pieces = (narrow ? sh.q_bufs * sh.q_bytes() : 2 * C::kTileBytes) / 16;
    for (int i = warp < kTmaWarp ? threadIdx.x : threadIdx.x - 32; i < pieces; i += kThreads - 32)
      st_shared_v4(at + 16 * i, 0u, 0u, 0u, 0u);
  }
  fence_proxy_async_shared();  // these and the prefix sums before the copies that follow
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  launch_dependents();  // the merge: its CTAs wait for this kernel before they read
  const uint32_t tmem = *tmem_slot;
  const bool skip = *abort_flag != 0;
  if (skip && threadIdx.x == 0) p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (warp < 8) write_unseen<D>(p, skip, threadIdx.x, 256);

  if (skip) {
    // nothing
  } else if (narrow) {
    if (warp == kTmaWarp) {
      narrow_producer<D>(p, sh, walk, first, items, &tm_q.narrow[sh.N == 16 ? 0 : (sh.N == 32 ? 1 : 2)], &tm_k, &tm_v, bar0, base,
                         first_entry, abort_flag, err);
    } else if (warp == kMmaWarp) {
      narrow_issuer<D>(p, sh, items, bar0, base, tmem, abort_flag, err);
    } else if (warp < 4 * sh.groups) {
      if (sh.N == 64)
        narrow_softmax<D, 32>(p, sh, items, warp >> 2, bar0, base, tmem, red + (warp >> 2) * 6 * 32, abort_flag, err);
      else
        narrow_softmax<D, 16>(p, sh, items, warp >> 2, bar0, base, tmem, red + (warp >> 2) * 6 * 32, abort_flag, err);
    }
  } else {
    const uint32_t sQ = base, sRing = base + 2 * C::kTileBytes;
    if (warp == kTmaWarp) {
      wide_producer<D>(p, walk, first, items, &tm_q.wide, &tm_k, &tm_v, bar0, sQ, sRing, first_entry, abort_flag, err);
    } else if (warp == kMmaWarp || warp == kMmaWarp1) {
      wide_issuer<D>(p, items, warp == kMmaWarp ? 0 : 1, bar0, sQ, sRing, tmem, turn, abort_flag, err);
    } else {
      wide_softmax<D>(p, items, warp >> 2, bar0, sRing, tmem, sRing + C::kStages * C::kTileBytes + warp * kStageBytes, abort_flag,
                      err);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// A lane's columns of row `row` of the partial that CTA c left of the item begun by CTA c0.
template <int D>
struct Partials {
  static constexpr int kCols = D / 32;  // columns of a lane
  const float *o, *lse;
  int rows, c0;
  __device__ __forceinline__ Partials(const PagedAttnParams &p)
      : o(p.part_o + (threadIdx.x & 31) * kCols), lse(p.part_lse), rows(p.part_rows), c0(blockIdx.x) {}
  __device__ __forceinline__ size_t at(int c, int row) const {
    return static_cast<size_t>(2 * c + (c == c0 ? 1 : 0)) * rows + row;
  }
  __device__ __forceinline__ void load(int c, int row, float (&v)[kCols]) const {
    const float *x = o + at(c, row) * D;
    if constexpr (kCols == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(x);
    else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(x);
  }
};

// One merged row of a cut item to O and lse: acc / sum, m + ln sum.
template <int D>
__device__ __forceinline__ void merged_row(const PagedAttnParams &p, const int4 &cut, int r, const float (&acc)[D / 32],
                                           float m, float sum) {
  constexpr int kCols = D / 32;
  const int lane = threadIdx.x & 31;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  const int head = cut.z * p.G + r % p.G, row = cut.x + r / p.G;
  __nv_bfloat162 *dst = reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p.o) + head * p.o_h + row * p.o_s +
                                                           lane * kCols);
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) dst[i] = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
  if (lane == 0 && p.lse)
    p.lse[static_cast<size_t>(head) * p.total_q + row] = sum != 0.f ? m + logf(sum) : -INFINITY;
}

// Rows of a cut item with at most kParts partials: a warp takes kRows of them and
// loads lse and O of all at once.
template <int D, int kParts, int kRows>
__device__ __forceinline__ void merge_few(const PagedAttnParams &p, const int4 &cut, int n, bool failed, int warp,
                                          int warps) {
  const Partials<D> parts(p);
  constexpr int kCols = D / 32;
  for (int r0 = warp * kRows; r0 < cut.y; r0 += warps * kRows) {
    float v[kParts][kRows][kCols], w[kParts][kRows];
#pragma unroll
    for (int k = 0; k < kParts; ++k)
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        w[k][u] = -INFINITY;
        if (k < n && r0 + u < cut.y && !failed) {
          w[k][u] = parts.lse[parts.at(blockIdx.x + k, r0 + u)];
          parts.load(blockIdx.x + k, r0 + u, v[k][u]);
        }
      }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (r0 + u >= cut.y) break;
      float m = w[0][u], acc[kCols] = {}, sum = 0.f;
#pragma unroll
      for (int k = 1; k < kParts; ++k) m = fmaxf(m, w[k][u]);
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        if (w[k][u] == -INFINITY) continue;  // a partial that saw no key has no O
        const float wk = expf(w[k][u] - m);
        sum += wk;
#pragma unroll
        for (int i = 0; i < kCols; ++i) acc[i] = fmaf(wk, v[k][u][i], acc[i]);
      }
      merged_row<D>(p, cut, r0 + u, acc, m, sum);
    }
  }
}

// The rows of the items that were cut: CTA blockIdx.x of the attention began such
// an item and described it (first token, rows, KV head, last CTA). Per row the
// weights exp(lse_i - max) of its partials and their weighted sum in the order of
// the keys. Bound by latency, so the loads are made to overlap: with two (four)
// partials a warp takes four (two) rows at once; with more, one row, eight
// partials at a time. (Loads that wait for the weights, two partials at a time:
// 17 us behind the attention of a batch of drafts, this: 8. Half the CTAs with
// twice the rows: 2.7 us more behind a small cross attention.)
constexpr int kMergeThreads = 256;
template <int D>
__global__ void __launch_bounds__(kMergeThreads, 4) merge_kernel(const __grid_constant__ PagedAttnParams p) {
  // (no launch_dependents here: the next attention's CTAs, let in early, cost a
  // small cross attention 36.5 -> 38.6 us)
  wait_prerequisites();
  const int4 cut = p.cuts[blockIdx.x];
  const int lane = threadIdx.x & 31;
  const int warp = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5), warps = gridDim.y * (kMergeThreads / 32);
  const int c0 = blockIdx.x, n = cut.w - c0 + 1;
  // a timeout somewhere: the partials may be missing, the rows come out empty
  const bool failed = *reinterpret_cast<volatile int *>(&g_device_error) != kErrNone;
  if (n <= 2) return merge_few<D, 2, 4>(p, cut, n, failed, warp, warps);
  if (n <= 4) return merge_few<D, 4, 2>(p, cut, n, failed, warp, warps);
  const Partials<D> parts(p);
  constexpr int kCols = D / 32;
  for (int r = warp; r < cut.y; r += warps) {
    float m = -INFINITY, sum = 0.f, acc[kCols] = {};
    if (!failed) {
      for (int k = lane; k < n; k += 32) m = fmaxf(m, parts.lse[parts.at(c0 + k, r)]);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      for (int k0 = 0; k0 < n; k0 += 8) {
        float v[8][kCols], w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          w[k] = -INFINITY;
          if (k0 + k < n) {
            w[k] = parts.lse[parts.at(c0 + k0 + k, r)];
            parts.load(c0 + k0 + k, r, v[k]);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (w[k] == -INFINITY) continue;
          const float wk = expf(w[k] - m);
          sum += wk;
#pragma unroll
          for (int i = 0; i < kCols; ++i) acc[i] = fmaf(wk, v[k][i], acc[i]);
        }
      }
    }
    merged_row<D>(p, cut, r, acc, m, sum);
  }
}

template <int D>
cudaError_t launch_typed(const QueryMaps &tq, const CUtensorMap &tk, const CUtensorMap &tv, const PagedAttnParams &p,
                         cudaStream_t stream) {
  auto kernel = attn_paged_kernel<D>;
  constexpr int kSmem = Cfg<D>::kSmemBytes;
  // once per device (the attribute holds for the kernel on the current device)
  static std::atomic<bool> prepared[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !prepared[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) prepared[dev].store(true, std::memory_order_release);
  }
  const int n_ctas = sm_count() < kPagedMaxCtas ? sm_count() : kPagedMaxCtas;
  e = launch_dependent(kernel, dim3(n_ctas), dim3(kThreads), kSmem, stream, tq, tk, tv, p);
  if (e != cudaSuccess || n_ctas == 1) return e;
  // the merge starts while the attention still runs and waits for its end inside
  constexpr int kRows = kMergeThreads / 32 * 4;
  return launch_dependent(merge_kernel<D>, dim3(n_ctas - 1, (p.part_rows + kRows - 1) / kRows), dim3(kMergeThreads), 0, stream,
                          p);
}

}  // namespace paged

cudaError_t launch_attn_paged(int D, const CUtensorMap &tq, const CUtensorMap (&tqn)[3], const CUtensorMap &tk,
                              const CUtensorMap &tv, const PagedAttnParams &p, cudaStream_t stream) {
  const paged::QueryMaps maps{tq, {tqn[0], tqn[1], tqn[2]}};
  return D == 64 ? paged::launch_typed<64>(maps, tk, tv, p, stream) : paged::launch_typed<128>(maps, tk, tv, p, stream);
}

}  // namespace seqattn
