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
// of 128-key tiles its last token sees. The key tiles of all items, put end
// to end, are cut into equal ranges, one per CTA, whatever the lengths: every
// CTA has the same work to within one tile. An item inside one range is
// written directly; an item that ranges cut leaves one fp32 partial per range
// (normalised, with its log-sum-exp) in the workspace, at most two per CTA,
// and a second kernel merges them in the order of the keys. The cuts follow
// from the lengths alone, so results do not depend on timing. Each CTA finds
// its range from prefix sums over the sequences that it forms itself: no
// planning launch, and a captured graph follows the lengths it finds.
//
// Inside a CTA the roles are those of the dense forward: a TMA producer warp,
// an MMA issuer per query tile taking turns, a softmax warpgroup per query
// tile. The producer reads the page table, one lane per page of a key tile
// (128 / page_size boxes, or one box inside a larger page).
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
  static constexpr int kSmemBytes = 1024 + 2 * kTileBytes + kStages * kTileBytes + 8 * kNumBarriers + 16 +
                                    8 * 12 + 8 * (kPagedMaxSeqs + 1);
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

// sum_{i=0}^{n-1} floor((a i + b) / m), a, b >= 0 (the lattice points under a
// line, by the Euclidean algorithm on a and m).
__device__ __forceinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
  long long sum = 0;
  while (n > 0) {
    sum += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const long long top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const long long t = m;
    m = a;
    a = t;
  }
  return sum;
}

// Key tiles of the items before row block `rb` of one KV head of a sequence.
__device__ __forceinline__ long long tiles_before(const PagedAttnParams &p, const Seq &s, int rb) {
  if (rb <= 0 || s.kv_len <= 0) return 0;
  const int rbs = row_blocks(p, s);
  if (!p.causal) return static_cast<long long>(min(rb, rbs)) * tiles_seen(p, s, s.q_len);
  // row block i < rbs - 1 sees ceil((c + i w) / 128) tiles, w = 2 tok rows, where c + i w > 0
  const int w = 2 * p.tok, n = min(rb, rbs - 1);
  const long long c = static_cast<long long>(s.kv_len) - s.q_len + w;
  long long sum = 0;
  const long long first = c > 0 ? 0 : (-c) / w + 1;  // first block that sees a key
  if (first < n) sum = floor_sum(n - first, kRowsPerTile, w, c + first * w + kRowsPerTile - 1);
  if (rb >= rbs) sum += tiles_seen(p, s, s.q_len);
  return sum;
}

// prefix[0 .. B]: key tiles of all KV heads of the sequences before each, by
// every thread of the CTA; warp_sums has 12 entries.
__device__ __forceinline__ void prefix_tiles(const PagedAttnParams &p, long long *prefix, long long *warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int B = p.cache.B, per = (B + blockDim.x - 1) / blockDim.x;
  const int b0 = min(B, static_cast<int>(threadIdx.x) * per), b1 = min(B, b0 + per);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = sequence(p, b);
    const long long t = s.q_len > 0 ? tiles_before(p, s, row_blocks(p, s)) * p.cache.Hkv : 0;
    prefix[b] = sum;
    sum += t;
  }
  long long incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  long long base = incl - sum;
  for (int i = 0; i < warp; ++i) base += warp_sums[i];
  for (int b = b0; b < b1; ++b) prefix[b] += base;
  if (threadIdx.x == blockDim.x - 1) prefix[B] = base + sum;
  __syncthreads();
}

// The sequence whose range of tiles has `pos`.
__device__ __forceinline__ int seq_of(const long long *prefix, int B, long long pos) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= pos) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Key tiles per CTA of a launch of n_ctas.
__device__ __forceinline__ long long tiles_per_cta(long long total, int n_ctas) {
  return (total + n_ctas - 1) / n_ctas;
}

// A CTA's part of one work item: key tiles [j0, j1) of row block rb.
struct Segment {
  Seq s;
  int b, h, rb, j0, j1;
  int slot;  // partial written, -1: the whole item, written directly
};

__device__ __forceinline__ const int *page_row(const PagedAttnParams &p, const Segment &g) {
  return p.cache.page_table + g.b * p.cache.table_stride;
}

// Walks the segments of tile range [pos, end) in order; every role walks its own.
struct Walk {
  long long pos, end, begin;
  int b, h, rb, r;  // r: first tile of the next segment within its item
  bool fresh;
  __device__ __forceinline__ Walk(const long long *prefix, int B, int n_ctas)
      : b(0), h(0), rb(0), r(0), fresh(true) {
    const long long per = tiles_per_cta(prefix[B], n_ctas);
    begin = pos = min(per * blockIdx.x, prefix[B]);
    end = min(pos + per, prefix[B]);
  }
  __device__ __forceinline__ bool next(const PagedAttnParams &p, const long long *prefix, Segment &g) {
    if (pos >= end) return false;
    if (fresh) {
      b = seq_of(prefix, p.cache.B, pos);
      g.s = sequence(p, b);
      const long long per_head = (prefix[b + 1] - prefix[b]) / p.cache.Hkv;
      const long long off = pos - prefix[b];
      h = static_cast<int>(off / per_head);
      long long rest = off - h * per_head;
      const int rbs = row_blocks(p, g.s);
      for (rb = 0; rb < rbs; ++rb) {
        const int n = item_tiles(p, g.s, rb);
        if (rest < n) break;
        rest -= n;
      }
      r = static_cast<int>(rest);
      fresh = false;
    } else {
      // the item after the last one, skipping those that see no key
      if (++rb >= row_blocks(p, g.s)) {
        rb = 0;
        if (++h >= p.cache.Hkv) {
          h = 0;
          do ++b;
          while (b < p.cache.B && prefix[b + 1] == prefix[b]);
          if (b >= p.cache.B) return false;
          g.s = sequence(p, b);
        }
      }
      const int rbs = row_blocks(p, g.s);
      while (rb < rbs && item_tiles(p, g.s, rb) == 0) ++rb;
      r = 0;
    }
    // (the bounds on b and rb only matter when the lengths change during the
    // call, which must not happen: then the walk ends instead of running on)
    const int n = rb < row_blocks(p, g.s) ? item_tiles(p, g.s, rb) : 0;
    if (n <= r) return false;
    g.b = b;
    g.h = h;
    g.rb = rb;
    g.j0 = r;
    g.j1 = static_cast<int>(min(static_cast<long long>(n), r + (end - pos)));
    g.slot = g.j0 == 0 && g.j1 == n ? -1 : 2 * static_cast<int>(blockIdx.x) + (g.j0 == 0 ? 1 : 0);
    pos += g.j1 - g.j0;
    return true;
  }
  // Key tiles of segment g that query tile t goes through, counted from g.j0.
  static __device__ __forceinline__ int tiles(const PagedAttnParams &p, const Segment &g, int t) {
    const int first = (2 * g.rb + t) * p.tok;
    if (first >= g.s.q_len) return 0;
    return max(0, min(g.j1, tiles_seen(p, g.s, first + p.tok)) - g.j0);
  }
};

// Softmax and epilogue of one row of query tile t over a segment (one thread a
// row, TMEM lane = tile row; the dense forward's scheme). `ring` is the ring
// position of the segment's first K tile.
template <int D>
__device__ __forceinline__ bool softmax_segment(const PagedAttnParams &p, const Segment &g, int t, int n, int r,
                                                uint32_t s_addr, uint32_t o_addr, uint32_t bar_sfull,
                                                uint32_t bar_pfull, uint32_t bar_ofull, uint32_t bar_full0,
                                                uint32_t ring_base, int ring, int step_base, uint32_t ofull_parity,
                                                volatile int *abort_flag, int *err) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  const int tok = (2 * g.rb + t) * p.tok + r / p.G;  // within the sequence
  const bool row_valid = r < p.tok * p.G && tok < g.s.q_len;
  const bool warp_valid = __any_sync(0xffffffffu, row_valid);
  const int row_last = !row_valid ? -1 : (p.causal ? g.s.kv_len - g.s.q_len + tok : g.s.kv_len - 1);
  const float c2 = p.scale_log2;
  const int page_size = 1 << p.page_log2;
  const int per_tile = page_size < kRowsPerTile ? kRowsPerTile >> p.page_log2 : 1;  // pages of a key tile
  // which pages of key tile j are there, one bit each (each lane looks one up)
  auto pages_there = [&](int j) -> unsigned {
    int e = 0;
    if (lane < per_tile) {
      const int i = page_size < kRowsPerTile ? j * per_tile + lane : (j * kRowsPerTile) >> p.page_log2;
      e = (i << p.page_log2) < g.s.kv_len ? page_row(p, g)[i] : 0;
    }
    return __ballot_sync(0xffffffffu, lane >= per_tile || (e >= 0 && e < p.cache.n_pages));
  };
  float m = -INFINITY, l = 0.f;
  bool ok = true;
  unsigned there = warp_valid ? pages_there(g.j0) : 0xffffffffu;

  for (int j = 0; j < n; ++j) {
    const unsigned now = there;
    if (warp_valid && j + 1 < n) there = pages_there(g.j0 + j + 1);
    ok = __all_sync(0xffffffffu, mbar_wait(bar_sfull, static_cast<uint32_t>(step_base + j) & 1u, abort_flag, err));
    if (!ok) break;
    tc_fence_after();
    const int kv0 = (g.j0 + j) * kRowsPerTile;
    if (warp_valid) {
      const int last = max(-1, min(row_last - kv0, kRowsPerTile - 1));
      const bool cut = __any_sync(0xffffffffu, last < kRowsPerTile - 1);
      const bool holes = now != 0xffffffffu;
      auto mask_scores = [&](uint32_t *x, int c0, int cols) {
        if (cut) {
#pragma unroll
          for (int c = 0; c < cols; ++c)
            if (c0 + c > last) x[c] = __float_as_uint(-INFINITY);
        }
        if (holes) {
#pragma unroll
          for (int c = 0; c < cols; ++c)
            if (!((now >> (per_tile == 1 ? 0 : (c0 + c) >> p.page_log2)) & 1u)) x[c] = __float_as_uint(-INFINITY);
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
      if (j == 0) m = row_max(reinterpret_cast<const float *>(sr)) * c2;
      rowsum = exp_row<false, 0>(reinterpret_cast<const float *>(sr), c2, (m == -INFINITY) ? 0.f : m, pk);
      if (j > 0) {
        // as in the dense forward: the reference moves, and O with it, only
        // when the tile's P would sum to more than 2^8 or there is none yet
        const bool big = !(rowsum <= kRescaleSum) || (m == -INFINITY && rowsum > 0.f);
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
#pragma unroll 1
          for (int cb = 0; cb < D / 32; ++cb) {
            uint32_t orr[32];
            tmem_ld32(o_addr + 32 * cb, orr);
            tmem_ld_wait(orr);
#pragma unroll
            for (int i = 0; i < 32; ++i) orr[i] = __float_as_uint(__uint_as_float(orr[i]) * alpha);
            tmem_st32(o_addr + 32 * cb, orr);
          }
          tmem_st_wait();
          load_scores(sr);
          rowsum = exp_row<false, 0>(reinterpret_cast<const float *>(sr), c2, (m == -INFINITY) ? 0.f : m, pk);
        }
      }
      l += rowsum;
      tmem_st32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
      tmem_st32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
      tmem_st_wait();
    }
    // V slots past kv_len may hold anything, NaN too, and 0 * NaN would reach
    // O: they are zeroed in shared memory before the product reads them. The
    // slot stays this tile's until both issuers have used it.
    const int valid_keys = g.s.kv_len - kv0;
    if (valid_keys < kRowsPerTile) {
      const int cv = ring + 2 * j + 1, slot = cv % C::kStages;
      ok = __all_sync(0xffffffffu, mbar_wait(bar_full0 + 8u * slot, (cv / C::kStages) & 1, abort_flag, err));
      if (!ok) break;
      const int pieces = (kRowsPerTile - valid_keys) * 8;  // 16-byte pieces of a 128-byte column block
      for (int i = threadIdx.x & 127; i < pieces * C::kColBlocks; i += 128)
        st_shared_v4(ring_base + slot * C::kTileBytes + (i / pieces) * kColBlockBytes + valid_keys * 128 +
                         (i % pieces) * 16,
                     0u, 0u, 0u, 0u);
      fence_proxy_async_shared();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_pfull);  // one arrival per warp
  }

  bool have_o = false;
  if (ok && n > 0) {
    have_o = __all_sync(0xffffffffu, mbar_wait(bar_ofull, ofull_parity, abort_flag, err));
    tc_fence_after();
  }
  const bool done = named_bar_and(1 + t, 128, ok && (n == 0 || have_o));
  if (!warp_valid) return done;
  const int head = g.h * p.G + r % p.G;
  const int row = g.s.q0 + tok;
  const float inv_l = l > 0.f ? 1.f / l : 0.f;
  const float lse = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
  if (g.slot >= 0) {
    const size_t at = static_cast<size_t>(g.slot) * p.part_rows + t * p.tok * p.G + r;
    if (row_valid) p.part_lse[at] = lse;
    if (have_o) {
#pragma unroll 1
      for (int cb = 0; cb < D / 32; ++cb) {
        uint32_t v[32];
        tmem_ld32(o_addr + 32 * cb, v);
        tmem_ld_wait(v);
        if (row_valid) {
          float4 *dst = reinterpret_cast<float4 *>(p.part_o + at * D + cb * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(v[4 * i]) * inv_l, __uint_as_float(v[4 * i + 1]) * inv_l,
                                 __uint_as_float(v[4 * i + 2]) * inv_l, __uint_as_float(v[4 * i + 3]) * inv_l);
        }
        __syncwarp();
      }
    }
    return done;
  }
  if (row_valid && p.lse) p.lse[static_cast<size_t>(head) * p.total_q + row] = lse;
#pragma unroll 1
  for (int cb = 0; cb < D / 32; ++cb) {
    uint32_t v[32];
    if (have_o) {
      tmem_ld32(o_addr + 32 * cb, v);
      tmem_ld_wait(v);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0u;
    }
    if (row_valid) {
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + head * p.o_h + row * p.o_s + cb * 32);
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
        dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncwarp();
  }
  return done;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedAttnParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem =
      reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sQ = smem;                          // [tile][col block][128 rows][128 B]
  uint8_t *sRing = smem + 2 * C::kTileBytes;   // [slot][col block][128 rows][128 B]
  uint64_t *bars = reinterpret_cast<uint64_t *>(sRing + C::kStages * C::kTileBytes);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::kNumBarriers);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *turn = reinterpret_cast<volatile int *>(tmem_slot + 2);
  long long *warp_sums = reinterpret_cast<long long *>(tmem_slot + 4);
  long long *prefix = warp_sums + 12;

  const uint32_t bar0 = smem_addr(bars);
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  const int kBarQFull = 0, kBarQEmpty = 1, kBarFull = 2, kBarEmpty = 2 + C::kStages, kBarSFull = 2 + 2 * C::kStages,
            kBarPFull = kBarSFull + 2, kBarOFull = kBarPFull + 2, kBarMmaDone = kBarOFull + 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int *err = &g_device_error;

  if (threadIdx.x == 0) {
    mbar_init(bar(kBarQFull), 1);
    mbar_init(bar(kBarQEmpty), 2);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(kBarFull + s), 1);
      mbar_init(bar(kBarEmpty + s), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kBarSFull + t), 1);
      mbar_init(bar(kBarPFull + t), 4);
      mbar_init(bar(kBarOFull + t), 1);
    }
    mbar_init(bar(kBarMmaDone), 2);
    // an earlier timeout, not yet cleared by the host: this CTA skips its work
    // and the merge writes O = 0, lse = -inf
    *abort_flag = *reinterpret_cast<volatile int *>(err) != kErrNone;
    *turn = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  prefix_tiles(p, prefix, warp_sums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool skip = *abort_flag != 0;
  auto tS = [&](int t) -> uint32_t { return tmem + 128u * static_cast<uint32_t>(t); };
  auto tO = [&](int t) -> uint32_t { return tmem + 256u + 128u * static_cast<uint32_t>(t); };
  Walk walk(prefix, p.cache.B, gridDim.x);
  Segment g;

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ producer (the whole warp)
    if (!skip) {
      if (lane == 0) {
        tma_prefetch_map(&tm_q);
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
      }
      const uint64_t pol_q = l2_policy_evict_last(), pol_kv = l2_policy_evict_first();
      const int page_size = 1 << p.page_log2;
      const bool small = page_size < kRowsPerTile;
      const int boxes = small ? kRowsPerTile >> p.page_log2 : 1;  // pages of a key tile
      const uint32_t box_bytes = (small ? page_size : kRowsPerTile) * 128u;
      const uint32_t q_bytes = static_cast<uint32_t>(p.tok * p.G) * 128u * C::kColBlocks;
      int c = 0, nq = 0;
      bool ok = true;
      while (ok && walk.next(p, prefix, g)) {
        const int n_max = max(Walk::tiles(p, g, 0), Walk::tiles(p, g, 1));
        const bool two = Walk::tiles(p, g, 1) > 0;
        const int *row = page_row(p, g);
        // the page of this lane for key tile j: n_pages (read as zeros) where there is none
        auto page_of = [&](int j) -> int {
          if (lane >= boxes) return 0;
          const int i = small ? j * boxes + lane : (j * kRowsPerTile) >> p.page_log2;
          int e = -1;
          if ((i << p.page_log2) < g.s.kv_len) e = row[i];
          return e >= 0 && e < p.cache.n_pages ? e : p.cache.n_pages;
        };
        int page = page_of(g.j0);
        if (lane == 0) {
          ok = nq == 0 || mbar_wait(bar(kBarQEmpty), (nq - 1) & 1, abort_flag, err);
          if (ok) {
            mbar_arrive_expect_tx(bar(kBarQFull), two ? 2 * q_bytes : q_bytes);
            for (int t = 0; t < (two ? 2 : 1); ++t)
              for (int cb = 0; cb < C::kColBlocks; ++cb)
                tma_load_4d_hint(smem_addr(sQ + (t * C::kColBlocks + cb) * kColBlockBytes), &tm_q, bar(kBarQFull),
                                 cb * 64, 0, g.s.q0 + (2 * g.rb + t) * p.tok, g.h, pol_q);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        ++nq;
        for (int j = 0; j < n_max && ok; ++j) {
          const int now = page;
          if (j + 1 < n_max) page = page_of(g.j0 + j + 1);
          const int in_page = small ? 0 : ((g.j0 + j) * kRowsPerTile) & (page_size - 1);
          for (int which = 0; which < 2; ++which, ++c) {
            const int slot = c % C::kStages;
            if (lane == 0) {
              ok = c < C::kStages || mbar_wait(bar(kBarEmpty + slot), ((c / C::kStages) - 1) & 1, abort_flag, err);
              if (ok) mbar_arrive_expect_tx(bar(kBarFull + slot), C::kTileBytes);
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
            if (lane < boxes) {
              const CUtensorMap *map = which ? &tm_v : &tm_k;
#pragma unroll
              for (int cb = 0; cb < C::kColBlocks; ++cb)
                tma_load_4d_hint(smem_addr(sRing + (slot * C::kColBlocks + cb) * kColBlockBytes) + lane * box_bytes, map,
                                 bar(kBarFull + slot), cb * 64, in_page, g.h, now, pol_kv);
            }
            __syncwarp();
          }
        }
      }
      if (lane == 0) {  // every copy must have landed before the CTA may exit
        if (nq > 0) mbar_drain(bar(kBarQFull), (nq - 1) & 1, err);
        for (int i = max(0, c - C::kStages); i < c; ++i)
          mbar_drain(bar(kBarFull + i % C::kStages), (i / C::kStages) & 1, err);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp || warp == kMmaWarp1) {
    // ------------------------------------------------------------ MMA issuers (the dense forward's scheme)
    const int t = (warp == kMmaWarp) ? 0 : 1;
    if (lane == 0 && !skip) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false), idesc_o = idesc_bf16_f32(128, D, true);
      constexpr int kKSteps = D / 16;
      const uint32_t qt = smem_addr(sQ) + t * C::kTileBytes, ring_base = smem_addr(sRing);
      const uint32_t s_col = tS(t), o_col = tO(t);
      int c = 0, nq = 0, steps = 0, base = 0;
      bool ok = true;
      while (ok && walk.next(p, prefix, g)) {
        const int nt = Walk::tiles(p, g, t);
        const int n_max = max(Walk::tiles(p, g, 0), Walk::tiles(p, g, 1));
        if (!mbar_wait(bar(kBarQFull), nq & 1, abort_flag, err)) break;
        ++nq;
        if (nt == 0) mma_commit(bar(kBarQEmpty));
        for (int j = 0; ok && j <= n_max; ++j) {
          const int cK = c + 2 * j, cV = c + 2 * j - 1;
          const int sK = cK % C::kStages, sV = (cV + C::kStages) % C::kStages;
          const int cV2 = cK + 1, sV2 = cV2 % C::kStages;
          const uint32_t k_base = ring_base + sK * C::kTileBytes, v_base = ring_base + sV * C::kTileBytes;
          const bool has_pv = j >= 1 && j - 1 < nt, has_s = j < nt, unused = !has_s && j < n_max;
          if ((has_s || unused) && !mbar_wait(bar(kBarFull + sK), (cK / C::kStages) & 1, abort_flag, err)) {
            ok = false;
            break;
          }
          if (unused && !mbar_wait(bar(kBarFull + sV2), (cV2 / C::kStages) & 1, abort_flag, err)) {
            ok = false;
            break;
          }
          if (has_pv && (!mbar_wait(bar(kBarFull + sV), (cV / C::kStages) & 1, abort_flag, err) ||
                         !mbar_wait(bar(kBarPFull + t), (steps + j - 1) & 1, abort_flag, err))) {
            ok = false;
            break;
          }
          const int turn_at = base + 2 * j + t;
          if (!wait_turn(turn, turn_at, abort_flag, err)) {
            ok = false;
            break;
          }
          if (has_pv) {
            tc_fence_after();
            const uint64_t vd = sw128_desc(v_base, kColBlockBytes, 1024);
#pragma unroll
            for (int kk = 0; kk < kRowsPerTile / 16; ++kk)
              mma_ts(o_col, s_col + kk * 8, vd + static_cast<uint64_t>(kk * 128), idesc_o, (j > 1 || kk > 0) ? 1u : 0u);
          }
          if (has_s) {
            const uint64_t qd = sw128_desc(qt, 16, 1024), kd = sw128_desc(k_base, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < kKSteps; ++kk) {
              const uint64_t off = static_cast<uint64_t>(((kk / 4) * kColBlockBytes + (kk % 4) * 32) >> 4);
              mma_ss(s_col, qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
            }
          }
          *turn = turn_at + 1;
          if (has_s) mma_commit(bar(kBarSFull + t));
          if (has_pv) {
            if (j - 1 == nt - 1) mma_commit(bar(kBarOFull + t));
            mma_commit(bar(kBarEmpty + sV));
          }
          if (has_s) {
            mma_commit(bar(kBarEmpty + sK));
            if (j == nt - 1) mma_commit(bar(kBarQEmpty));
          }
          if (unused) {
            mma_commit(bar(kBarEmpty + sK));
            mma_commit(bar(kBarEmpty + sV2));
          }
        }
        c += 2 * n_max;
        steps += nt;
        base += 2 * (n_max + 1);
      }
      mma_commit(bar(kBarMmaDone));
      mbar_drain(bar(kBarMmaDone), 0, err);
    }
    __syncwarp();
  } else if (warp < 8 && !skip) {
    // ------------------------------------------------------------ softmax + epilogue
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int steps = 0, ring = 0;
    uint32_t u = 0;
    while (walk.next(p, prefix, g)) {
      const int n = Walk::tiles(p, g, t), n_max = max(Walk::tiles(p, g, 0), Walk::tiles(p, g, 1));
      if (!softmax_segment<D>(p, g, t, n, r, tS(t) + lane_off, tO(t) + lane_off, bar(kBarSFull + t),
                              bar(kBarPFull + t), bar(kBarOFull + t), bar(kBarFull), smem_addr(sRing), ring, steps,
                              u & 1u, abort_flag, err))
        break;
      ring += 2 * n_max;
      steps += n;
      if (n > 0) ++u;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The rows that the ranges cut, and the rows of items that see no key. Grid:
// (row blocks, KV heads, sequences); a warp takes a row: the weights
// exp(lse_i - max) of its partials, then their weighted sum in the order of
// the keys, four (D = 128) or two columns a lane.
constexpr int kMergeThreads = 256;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ PagedAttnParams p, int n_ctas) {
  extern __shared__ long long prefix[];  // [B + 1], then 12 sums
  const bool failed = *reinterpret_cast<volatile int *>(&g_device_error) != kErrNone;
  prefix_tiles(p, prefix, prefix + p.cache.B + 1);
  const long long per = tiles_per_cta(prefix[p.cache.B], n_ctas);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kCols = D / 32;
  for (int b = blockIdx.z; b < p.cache.B; b += gridDim.z) {
    const Seq s = sequence(p, b);
    const int rbs = row_blocks(p, s);
    for (int rb = blockIdx.x; rb < rbs; rb += gridDim.x) {
      const int h = blockIdx.y;
      const int n = failed ? 0 : item_tiles(p, s, rb);
      long long t0 = 0;
      int c0 = 0, c1 = 0;
      if (n > 0) {
        const long long per_head = (prefix[b + 1] - prefix[b]) / p.cache.Hkv;
        t0 = prefix[b] + h * per_head + tiles_before(p, s, rb);
        c0 = static_cast<int>(t0 / per);
        c1 = static_cast<int>((t0 + n - 1) / per);
        if (c0 == c1) continue;
      }
      const int rows = min(2 * p.tok, s.q_len - rb * 2 * p.tok) * p.G;
      for (int r = warp; r < rows; r += kMergeThreads / 32) {
        float acc[kCols] = {};
        float m = -INFINITY, sum = 0.f;
        auto at = [&](int c) -> size_t {
          return static_cast<size_t>(2 * c + (c == c0 ? 1 : 0)) * p.part_rows + r;
        };
        if (n > 0) {
          for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, p.part_lse[at(c)]);
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        }
        if (m != -INFINITY) {
          for (int cb = c0; cb <= c1; cb += 32) {
            const float w = cb + lane <= c1 ? expf(p.part_lse[at(cb + lane)] - m) : 0.f;
            sum += w;
            const int k_end = min(32, c1 - cb + 1);
#pragma unroll 4
            for (int k = 0; k < k_end; ++k) {
              const float wk = __shfl_sync(0xffffffffu, w, k);
              if (wk == 0.f) continue;  // a partial that saw no key has no O
              const float *x = p.part_o + at(cb + k) * D + lane * kCols;
              if constexpr (kCols == 4) {
                const float4 v = *reinterpret_cast<const float4 *>(x);
                acc[0] = fmaf(wk, v.x, acc[0]);
                acc[1] = fmaf(wk, v.y, acc[1]);
                acc[2] = fmaf(wk, v.z, acc[2]);
                acc[3] = fmaf(wk, v.w, acc[3]);
              } else {
                const float2 v = *reinterpret_cast<const float2 *>(x);
                acc[0] = fmaf(wk, v.x, acc[0]);
                acc[1] = fmaf(wk, v.y, acc[1]);
              }
            }
          }
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const int head = h * p.G + r % p.G, row = s.q0 + rb * 2 * p.tok + r / p.G;
        __nv_bfloat162 *dst = reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p.o) + head * p.o_h +
                                                                 row * p.o_s + lane * kCols);
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) dst[i] = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
        if (lane == 0 && p.lse)
          p.lse[static_cast<size_t>(head) * p.total_q + row] = sum > 0.f ? m + logf(sum) : -INFINITY;
      }
    }
  }
}

template <int D>
cudaError_t launch_typed(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                         const PagedAttnParams &p, cudaStream_t stream) {
  auto kernel = attn_paged_kernel<D>;
  constexpr int kSmem = Cfg<D>::kSmemBytes;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int n_ctas = sm_count() < kPagedMaxCtas ? sm_count() : kPagedMaxCtas;
  kernel<<<n_ctas, kThreads, kSmem, stream>>>(tq, tk, tv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // row blocks of the longest chunk there can be, bounded: the kernel strides
  const long long rbs = (static_cast<long long>(p.total_q) + 2 * p.tok - 1) / (2 * p.tok);
  const unsigned gx = static_cast<unsigned>(rbs < 64 ? rbs : 64);
  const unsigned gz = static_cast<unsigned>(p.cache.B < 1024 ? p.cache.B : 1024);
  const size_t smem = sizeof(long long) * (static_cast<size_t>(p.cache.B) + 1 + 12);
  merge_kernel<D><<<dim3(gx, p.cache.Hkv, gz), kMergeThreads, smem, stream>>>(p, n_ctas);
  return cudaGetLastError();
}

}  // namespace paged

cudaError_t launch_attn_paged(int D, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                              const PagedAttnParams &p, cudaStream_t stream) {
  return D == 64 ? paged::launch_typed<64>(tq, tk, tv, p, stream) : paged::launch_typed<128>(tq, tk, tv, p, stream);
}

}  // namespace seqattn
