// The narrow form of the paged attention (included by attn_paged.cuh): sequences
// of at most 64 rows per KV head (single tokens, drafts).
//
// The cost is reading K and V, and what bounds that is bytes in flight: with
// 96, 128 KB of tiles per SM a batch of 64 sequences (8 KV heads of 128, 2.1 GB
// of cache) took 490, 389 us. So shared memory goes to the ring (192 KB, 160 KB
// beyond 32 rows: 310 us = 6.8 TB/s, what a copy reaches; 5.9 TB/s with heads of
// 64), and the products are turned over, keys on the 128 rows of
// the tensor tile: S^T = K Q^T (128 keys x N rows, N = 16, 32 or 64) and
// O^T += V^T P (D x N). Q and P are small then, no tensor row is wasted on
// queries that do not exist, and a thread has one key: N exponentials instead
// of 128. A softmax over keys runs across threads; per tile it needs no
// reduction, as each thread keeps its own part of the sums l until the end and
// the reference m moves only when some score passes it by more than 2^8 (one
// vote per tile; the maximum over the 128 keys is taken only then).
//
// Roles: warps 0-3 (and 4-7 for N > 16, with the upper half of the columns)
// softmax, warp 8 MMA issuer, warp 9 producer. TMEM columns: S^T in two
// buffers [0, N), [N, 2 N), O^T [2 N, 3 N). P goes through shared memory as
// [key][row], 128 bytes a key, 128-byte swizzle, in two buffers too (rows 0 and
// N of the 64 that a key has room for, or two tiles when N = 64): with one, a
// tile's P waited for the product of the tile before, 2,170 clocks a tile at
// N = 16 (measured), above D = 64's share of the DRAM rate.
#pragma once

namespace seqattn {
namespace paged {

// Sizes of the narrow form for N rows.
template <int D>
struct Narrow {
  static constexpr int kColBlocks = D / 64;
  static constexpr int kTileBytes = kRowsPerTile * D * 2;
  static constexpr int kPBytes = kRowsPerTile * 128;
  static constexpr int kMaxStages = 196608 / kTileBytes;
  int N, tok, stages, q_bufs, groups;  // groups: softmax warpgroups
  __device__ __forceinline__ Narrow(int rows, int G) {
    N = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
    tok = max(1, N / G);
    stages = (N == 64 ? 163840 : 196608) / kTileBytes;
    q_bufs = N == 64 ? 1 : 2;
    groups = N == 16 ? 1 : 2;
  }
  // shared memory behind the 1024-byte aligned start: ring, P, Q
  __device__ __forceinline__ int p_at() const { return stages * kTileBytes; }
  __device__ __forceinline__ int q_at() const { return p_at() + (N == 64 ? 2 : 1) * kPBytes; }
  __device__ __forceinline__ int q_bytes() const { return N * D * 2; }
  static constexpr int kAreaBytes = 196608 + kPBytes + 2 * 32 * D * 2;
  static_assert(163840 + 2 * kPBytes + 64 * D * 2 <= kAreaBytes, "narrow layouts");
  // barriers
  static constexpr int kFull = 0, kEmpty = kMaxStages, kQFull = 2 * kMaxStages, kQEmpty = kQFull + 2,
                       kSFull = kQEmpty + 2, kPFull = kSFull + 2, kPvDone = kPFull + 2, kMmaDone = kPvDone + 2,
                       kNumBarriers = kMmaDone + 1;
};

// A position of the ring and the parity of its current phase.
struct RingPos {
  int slot;
  uint32_t phase;
  __device__ __forceinline__ RingPos next(int stages) const {
    return slot + 1 == stages ? RingPos{0, phase ^ 1u} : RingPos{slot + 1, phase};
  }
};

// S^T instruction: K (K-major) x Q (K-major); O^T: V^T (M-major) x P (N-major).
__device__ __forceinline__ uint32_t idesc_narrow(int N, bool pv) {
  return idesc_bf16_f32(128, 0, pv) | (pv ? 1u << 15 : 0u) | (static_cast<uint32_t>(N >> 3) << 17);
}

// Producer: the whole warp.
template <int D>
__device__ __forceinline__ void narrow_producer(const PagedAttnParams &p, const Narrow<D> &sh, Walk walk, Segment g, Items items,
                                             const CUtensorMap *tm_q, const CUtensorMap *tm_k, const CUtensorMap *tm_v,
                                             uint32_t bar0, uint32_t smem, int first_entry, volatile int *abort_flag,
                                             int *err) {
  using C = Narrow<D>;
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  const uint64_t pol_q = l2_policy_evict_last(), pol_kv = l2_policy_evict_first();
  const int page_size = 1 << p.page_log2;
  const bool small = page_size < kRowsPerTile;
  const int boxes = uniform(pages_of_tile(p)), stages = uniform(sh.stages);
  const uint32_t box_bytes = uniform((small ? page_size : kRowsPerTile) * 128u);
  const uint32_t q_bytes = static_cast<uint32_t>(sh.tok * p.G) * 128u * C::kColBlocks;
  const bool leader = elect_one();
  auto wait = [&](int i, uint32_t phase) {
    return __all_sync(0xffffffffu, mbar_wait(bar(i), phase, abort_flag, err));
  };
  RingPos at{0, 0};
  long long fills = 0;
  int nq = 0, q_loads = 0;
  bool ok = true;
  int4 cut = make_int4(0, 0, 0, 0);
  while (ok && walk.next(p, g)) {
    g.ring = static_cast<int>(fills);
    if (!items.put(g, abort_flag, err)) break;
    if (g.j0 == 0 && g.slot >= 0) cut = make_int4(g.s.q0, min(g.s.q_len * p.G, kNarrowRows), g.h, walk.ends_in(p, g));
    const int j0 = uniform(g.j0), n = uniform(g.j1) - j0, head = uniform(g.h);
    PageWindow pages(p, g, nq == 0, first_entry);
    const int qb = nq % sh.q_bufs, use = nq / sh.q_bufs;
    bool q_due = true;  // this segment's Q is still to be loaded
    int page = 0;
    for (int f = 0; f < 2 * n && ok; ++f, ++fills) {
      // Q as soon as its buffer is free, but K and V go ahead of it meanwhile:
      // the slots of the first fills are given back by earlier segments
      if (q_due && (use == 0 || f >= stages / 2 || f == 2 * n - 1 ||
                    __all_sync(0xffffffffu, mbar_test(bar(C::kQEmpty + qb), (use - 1) & 1)))) {
        ok = use == 0 || wait(C::kQEmpty + qb, (use - 1) & 1);
        if (!ok) break;
        ++q_loads;
        q_due = false;
        if (leader) {
          mbar_arrive_expect_tx(bar(C::kQFull + qb), q_bytes);
          for (int cb = 0; cb < C::kColBlocks; ++cb)
            tma_load_4d_hint(smem + sh.q_at() + qb * sh.q_bytes() + cb * sh.N * 128, tm_q, bar(C::kQFull + qb), cb * 64, 0,
                             g.s.q0, head, pol_q);
        }
        __syncwarp();
      }
      const int j = j0 + (f >> 1), which = f & 1;
      if (!which) page = pages.page(p, j);
      ok = fills < stages || wait(C::kEmpty + at.slot, at.phase ^ 1u);
      if (!ok) break;
      if (leader) mbar_arrive_expect_tx(bar(C::kFull + at.slot), C::kTileBytes);
      const CUtensorMap *map = which ? tm_v : tm_k;
      const int in_page = small ? 0 : (j * kRowsPerTile) & (page_size - 1);
      load_pages<D>(smem + at.slot * C::kTileBytes, map, bar(C::kFull + at.slot), in_page, head, page, boxes, box_bytes,
                    leader, pol_kv);
      if (f == 1) pages.prefetch(p);
      at = at.next(stages);
    }
    ++nq;
  }
  g.j0 = g.j1 = 0;
  items.put(g, abort_flag, err);
  if (lane == 0) {
    p.cuts[blockIdx.x] = cut;
    // every copy must have landed before the CTA may exit
    for (int i = max(0, q_loads - sh.q_bufs); i < q_loads; ++i)
      mbar_drain(bar(C::kQFull + i % sh.q_bufs), (i / sh.q_bufs) & 1, err);
    for (long long i = max(0ll, fills - stages); i < fills; ++i)
      mbar_drain(bar(C::kFull + static_cast<int>(i % stages)), static_cast<uint32_t>(i / stages) & 1u, err);
  }
  __syncwarp();
}

// MMA issuer: the whole warp, its code uniform, one lane for the products. (As the
// code of a single thread it took about 95 clocks an MMA to bring the operands
// into uniform registers, 1,520 to 1,800 a tile: more than the MMAs.)
template <int D>
__device__ __forceinline__ void narrow_issuer(const PagedAttnParams &p, const Narrow<D> &sh, Items items, uint32_t bar0,
                                              uint32_t smem, uint32_t tmem_in, volatile int *abort_flag, int *err) {
  using C = Narrow<D>;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  auto wait = [&](int i, uint32_t phase) {
    return __all_sync(0xffffffffu, mbar_wait(bar(i), phase, abort_flag, err));
  };
  const bool leader = elect_one();
  const uint32_t tmem = uniform(tmem_in), N = uniform(static_cast<uint32_t>(sh.N));
  const int stages = uniform(sh.stages), q_bufs = N == 64 ? 1 : 2;
  const uint32_t p_at = smem + stages * C::kTileBytes, p_step = N == 64 ? static_cast<uint32_t>(C::kPBytes) : 2 * N;
  const uint32_t q_at = p_at + (N == 64 ? 2 : 1) * C::kPBytes, q_bytes = N * D * 2;
  const uint32_t idesc_s = idesc_narrow(N, false), idesc_o = idesc_narrow(N, true);
  const uint32_t o_col = tmem + 2 * N;
  RingPos k{0, 0};
  uint32_t step = 0;  // key tiles so far
  int nq = 0;
  bool ok = true;
  while (ok && items.wait(abort_flag, err)) {
    const int n = uniform(items.get().j1 - items.get().j0);
    items.release();
    const int qb = nq & (q_bufs - 1);
    if (!wait(C::kQFull + qb, (q_bufs == 2 ? nq >> 1 : nq) & 1)) break;
    ++nq;
    const uint64_t qd = sw128_desc(q_at + qb * q_bytes, 16, 1024);
    const uint64_t q_block = static_cast<uint64_t>((N * 128) >> 4);  // from one 64-column block to the next
    auto scores = [&](const RingPos &at, uint32_t to, bool last) {
      const uint64_t kd = sw128_desc(smem + at.slot * C::kTileBytes, 16, 1024);
      const uint32_t s_col = tmem + (to & 1u) * N;
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(s_col, kd + static_cast<uint64_t>(((kk / 4) * kColBlockBytes + (kk % 4) * 32) >> 4),
                 qd + (kk / 4) * q_block + static_cast<uint64_t>((kk % 4) * 2), idesc_s, kk > 0 ? 1u : 0u);
        mma_commit(bar(C::kSFull + (to & 1u)));
        mma_commit(bar(C::kEmpty + at.slot));
        if (last) mma_commit(bar(C::kQEmpty + qb));
      }
      __syncwarp();
    };
    if (!wait(C::kFull + k.slot, k.phase)) break;
    scores(k, step, n == 1);
    for (int j = 0; j < n; ++j, ++step) {
      const RingPos v = k.next(stages), k1 = v.next(stages);
      // the next scores ahead of this product if their keys are there; their
      // buffer was read before P of the tile before this one was signalled
      const bool early = j + 1 < n && __all_sync(0xffffffffu, mbar_test(bar(C::kFull + k1.slot), k1.phase));
      if (early) scores(k1, step + 1, j + 2 == n);
      if (!wait(C::kPFull + (step & 1u), (step >> 1) & 1u) || !wait(C::kFull + v.slot, v.phase)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // V as stored, [key][column], is the M-major A operand; for D = 64 the
      // upper 64 rows of the product read the bytes behind the tile and are
      // never looked at (rows of a product do not mix)
      const uint64_t vd = sw128_desc(smem + v.slot * C::kTileBytes, kColBlockBytes, 1024);
      const uint64_t pd = sw128_desc(p_at + (step & 1u) * p_step, kColBlockBytes, 1024);
      const uint32_t add = j > 0 ? 1u : 0u;
      if (leader) {
        mma_ss(o_col, vd, pd, idesc_o, add);
#pragma unroll
        for (int kk = 1; kk < kRowsPerTile / 16; ++kk)
          mma_ss(o_col, vd + static_cast<uint64_t>(kk * 128), pd + static_cast<uint64_t>(kk * 128), idesc_o, 1u);
        mma_commit(bar(C::kEmpty + v.slot));
        mma_commit(bar(C::kPvDone + (step & 1u)));
      }
      __syncwarp();
      if (j + 1 < n && !early) {
        if (!wait(C::kFull + k1.slot, k1.phase)) {
          ok = false;
          break;
        }
        scores(k1, step + 1, j + 2 == n);
      }
      k = k1;
    }
  }
  if (leader) {
    mma_commit(bar(C::kMmaDone));
    mbar_drain(bar(C::kMmaDone), 0, err);
  }
  __syncwarp();
}

// Reduces 16 values over the 32 lanes of a warp at once, halving the values with
// every step: lane i returns the result of value i / 2.
template <typename Op>
__device__ __forceinline__ float reduce16(float (&v)[16], Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int half = 8; half > 0; half >>= 1) {
    const bool upper = lane & (2 * half);
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = upper ? v[i + half] : v[i], give = upper ? v[i] : v[i + half];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, 2 * half));
    }
  }
  return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

// The reference of a column that has seen no key, the lowest finite number: any
// score passes it, and 2^(-inf - it) is still 0.
constexpr float kNoReference = -3.402823466e38f;

// Softmax and epilogue of columns [col0, col0 + C) of S^T: one thread per key
// (and, in the epilogue, per column of O). `red` is this warpgroup's 6 x C
// floats of shared memory, `gi` its number. Every warp goes through the same
// barriers whatever fails: a wait that runs out is carried to the next vote, the
// wait for an item included.
template <int D, int C>
__device__ __forceinline__ void narrow_softmax(const PagedAttnParams &p, const Narrow<D> &sh, Items items,
                                            int gi, uint32_t bar0, uint32_t smem, uint32_t tmem, float *red,
                                            volatile int *abort_flag, int *err) {
  using L = Narrow<D>;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  const int key = threadIdx.x & 127, lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
  const int col0 = gi * C, id = 1 + gi;
  const uint32_t lane_off = static_cast<uint32_t>(32 * w) << 16;
  const uint32_t o_addr = tmem + lane_off + 2 * sh.N + col0;
  // until the product of key tile s (and so all before it) is done
  auto product_done = [&](uint32_t s) {
    return __all_sync(0xffffffffu, mbar_wait(bar(L::kPvDone + (s & 1u)), (s >> 1) & 1u, abort_flag, err));
  };
  const float c2 = p.scale_log2;
  auto larger = [](float a, float b) { return fmaxf(a, b); };
  auto sum_of = [](float a, float b) { return a + b; };
  float *ref = red + 4 * C, *factor = red + 5 * C;  // references of the columns; a factor for each
  RingPos k{0, 0};
  uint32_t step = 0;
  while (items.wait_together(id, abort_flag, err)) {
    const Segment g = items.get();
    items.release();
    const int n = g.j1 - g.j0, rows = g.s.q_len * p.G;
    const int first_last = p.causal ? g.s.kv_len - g.s.q_len : g.s.kv_len - 1;  // last key of the first token
    const int *table = page_row(p, g);
    auto entry_of = [&](int j) -> int {
      const int pos = j * kRowsPerTile + key;
      return pos < g.s.kv_len ? table[pos >> p.page_log2] : -1;
    };
    float m[C], l[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      m[c] = kNoReference;
      l[c] = 0.f;
    }
    if (key < C) ref[key] = kNoReference;
    int entry = entry_of(g.j0);
    bool ok = true;
    for (int j = 0; j < n; ++j, ++step) {
      const bool there = entry >= 0 && entry < p.cache.n_pages;
      if (j + 1 < n) entry = entry_of(g.j0 + j + 1);
      const int kv0 = (g.j0 + j) * kRowsPerTile;
      ok = ok && __all_sync(0xffffffffu,
                            mbar_wait(bar(L::kSFull + (step & 1u)), (step >> 1) & 1u, abort_flag, err));
      tc_fence_after();
      const bool partly = kv0 + kRowsPerTile - 1 > first_last;  // some row does not see all keys of the tile
      const bool holes = __any_sync(0xffffffffu, !there);
      // 16 columns from h on of this key's scores times scale log2(e), masked,
      // less the columns' references
      auto load_scores = [&](int h, const float *less, float *x) {
        uint32_t raw[16];
        tmem_ld16(tmem + lane_off + (step & 1u) * sh.N + col0 + h, raw);
        tmem_ld_wait(raw);
#pragma unroll
        for (int c = 0; c < 16; ++c) x[c] = fmaf(__uint_as_float(raw[c]), c2, less ? -less[c] : 0.f);
        if (holes) {
#pragma unroll
          for (int c = 0; c < 16; ++c) x[c] = there ? x[c] : -INFINITY;
        }
        if (partly) {
          int tok = (col0 + h) / p.G, head = col0 + h - tok * p.G;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int last = p.causal ? min(first_last + tok, g.s.kv_len - 1) : first_last;
            if (kv0 + key > last) x[c] = -INFINITY;
            if (++head == p.G) {
              head = 0;
              ++tok;
            }
          }
        }
      };
      float x[C];
      float top = -INFINITY;
      if (j > 0) {
#pragma unroll
        for (int h = 0; h < C; h += 16) {
          load_scores(h, m + h, x + h);
#pragma unroll
          for (int c = 0; c < 16; c += 2) top = fmax3(top, x[h + c], x[h + c + 1]);
        }
      }
      // the first tile of a segment has no reference yet
      if (j == 0 || !named_bar_and(id, 128, ok && !(top > 8.f))) {
        // maxima of the tile's 128 keys, then O and l onto the new reference
#pragma unroll
        for (int h = 0; h < C; h += 16) {
          float y[16];
          load_scores(h, nullptr, y);
          const float most = reduce16(y, larger);
          if (!(lane & 1)) red[w * C + h + (lane >> 1)] = most;
        }
        named_bar_sync(id, 128);
        if (key < C) {
          const float most = fmaxf(fmaxf(red[key], red[C + key]), fmaxf(red[2 * C + key], red[3 * C + key]));
          const float old_ref = ref[key], new_ref = fmaxf(old_ref, most);
          ref[key] = new_ref;
          factor[key] = ex2_approx(old_ref - new_ref);
        }
        ok = named_bar_and(id, 128, ok);
        if (ok && j > 0)
          ok = product_done(step - 1);
        tc_fence_after();
        const bool old = ok && j > 0;  // O holds the sum of the tiles before
#pragma unroll
        for (int h = 0; h < C; h += 16) {
          uint32_t v[16] = {};
          if (old) {
            tmem_ld16(o_addr + h, v);
            tmem_ld_wait(v);
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float alpha = factor[h + c];
            m[h + c] = ref[h + c];
            l[h + c] *= alpha;
            v[c] = __float_as_uint(__uint_as_float(v[c]) * alpha);
          }
          if (old) tmem_st16(o_addr + h, v);
          load_scores(h, m + h, x + h);
        }
        if (old) tmem_st_wait();
      }
      uint32_t pk[C / 2];
#pragma unroll
      for (int i = 0; i < C; i += 2) {
        const float a = ex2_approx(x[i]), b = ex2_approx(x[i + 1]);
        l[i] += a;
        l[i + 1] += b;
        // P enters the tensor cores in bf16, as in the dense forward; l is summed before the rounding
        __nv_bfloat162 pair = __floats2bfloat162_rn(a, b);
        pk[i / 2] = *reinterpret_cast<uint32_t *>(&pair);
      }
      // the product of the tile before the last has read its P
      if (step >= 2) ok = ok && product_done(step - 2);
      if (ok) {
        // 16-byte pieces of this key's rows, at the swizzled places
        const uint32_t p_key = smem + sh.p_at() + (sh.N == 64 ? (step & 1u) * L::kPBytes : 0u) + key * 128;
        const int piece = (col0 + (sh.N == 64 ? 0 : static_cast<int>(step & 1u) * sh.N)) / 8;
#pragma unroll
        for (int i = 0; i < C / 8; ++i)
          st_shared_v4(p_key + (static_cast<uint32_t>((piece + i) ^ (key & 7)) << 4), pk[4 * i], pk[4 * i + 1],
                       pk[4 * i + 2], pk[4 * i + 3]);
        const RingPos v = k.next(sh.stages);
        if (gi == 0 && g.s.kv_len - kv0 < kRowsPerTile)
          ok = clear_tail<D>(g.s.kv_len - kv0, smem + v.slot * L::kTileBytes, bar(L::kFull + v.slot), v.phase, abort_flag,
                             err);
        fence_proxy_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kPFull + (step & 1u)));  // one arrival per warp
      }
      k = k.next(sh.stages).next(sh.stages);
    }
    ok = ok && product_done(step - 1);
    tc_fence_after();
    // l over the keys, and from it each row's factor and lse
#pragma unroll
    for (int h = 0; h < C; h += 16) {
      float y[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) y[c] = l[h + c];
      const float s = reduce16(y, sum_of);
      if (!(lane & 1)) red[w * C + h + (lane >> 1)] = s;
    }
    if (!named_bar_and(id, 128, ok)) return;
    const size_t part = static_cast<size_t>(max(g.slot, 0)) * p.part_rows + col0;
    if (key < C) {
      const float sum = (red[key] + red[C + key]) + (red[2 * C + key] + red[3 * C + key]);
      factor[key] = sum != 0.f ? 1.f / sum : 0.f;
      if (col0 + key < rows) {
        const float lse = sum != 0.f ? (ref[key] + log2f(sum)) * kLn2 : -INFINITY;
        const int tok = (col0 + key) / p.G, head = g.h * p.G + (col0 + key) - tok * p.G;
        if (g.slot >= 0) p.part_lse[part + key] = lse;
        else if (p.lse) p.lse[static_cast<size_t>(head) * p.total_q + g.s.q0 + tok] = lse;
      }
    }
    named_bar_sync(id, 128);
    // a thread has column `key` of O, one row after the other
    const int n_rows = min(C, rows - col0);
    int tok = col0 / p.G, head = col0 - tok * p.G;
    float *to_part = p.part_o + part * D + key;
    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(p.o) + (g.h * p.G + head) * p.o_h + (g.s.q0 + tok) * p.o_s + key;
#pragma unroll 1
    for (int h = 0; h < n_rows; h += 8) {
      uint32_t v[8];
      tmem_ld8(o_addr + h, v);
      tmem_ld_wait(v);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (h + c < n_rows && key < D) {
          const float o = __uint_as_float(v[c]) * factor[h + c];
          if (g.slot >= 0) to_part[(h + c) * D] = o;
          else *to = __float2bfloat16_rn(o);
        }
        to += p.o_h;
        if (++head == p.G) {
          head = 0;
          to += p.o_s - p.G * p.o_h;
        }
      }
      __syncwarp();
    }
  }
}

}  // namespace paged
}  // namespace seqattn
