// The narrow form of the paged attention (included by attn_paged.cuh): every
// sequence of the call has at most 64 rows per KV head (single tokens, drafts).
//
// The cost is reading K and V, and what bounds that is bytes in flight: with
// 96, 128 KB of tiles per SM the 64-sequence batch of the benchmark (2.1 GB of
// cache) took 490, 389 us. So shared memory goes to the ring (192 KB, 160 KB
// beyond 32 rows), and the products are turned over, keys on the 128 rows of
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
// [key][row], 128 bytes a key, 128-byte swizzle.
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
    q_bufs = N == 16 ? 2 : 1;
    groups = N == 16 ? 1 : 2;
  }
  // shared memory behind the 1024-byte aligned start: ring, P, Q
  __device__ __forceinline__ int p_at() const { return stages * kTileBytes; }
  __device__ __forceinline__ int q_at() const { return p_at() + kPBytes; }
  __device__ __forceinline__ int q_bytes() const { return N * D * 2; }
  static constexpr int kAreaBytes = 196608 + kPBytes + 2 * 16 * D * 2;  // N = 16 or 32; N = 64 needs less
  static_assert(163840 + kPBytes + 64 * D * 2 <= kAreaBytes, "narrow layouts");
  // barriers
  static constexpr int kFull = 0, kEmpty = kMaxStages, kQFull = 2 * kMaxStages, kQEmpty = kQFull + 2,
                       kSFull = kQEmpty + 2, kPFull = kSFull + 2, kPvDone = kPFull + 1, kMmaDone = kPvDone + 1,
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
__device__ __noinline__ void narrow_producer(const PagedAttnParams &p, const Narrow<D> &sh, Walk walk, const int *prefix,
                                             const CUtensorMap *tm_q, const CUtensorMap *tm_k, const CUtensorMap *tm_v,
                                             uint32_t bar0, uint32_t smem, volatile int *abort_flag, int *err) {
  using C = Narrow<D>;
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  const uint64_t pol_q = l2_policy_evict_last(), pol_kv = l2_policy_evict_first();
  const int page_size = 1 << p.page_log2;
  const bool small = page_size < kRowsPerTile;
  const int boxes = small ? kRowsPerTile >> p.page_log2 : 1;
  const uint32_t box_bytes = (small ? page_size : kRowsPerTile) * 128u;
  const uint32_t q_bytes = static_cast<uint32_t>(sh.tok * p.G) * 128u * C::kColBlocks;
  RingPos at{0, 0};
  long long fills = 0;
  int nq = 0, q_loads = 0;
  bool ok = true;
  Segment g;
  int4 cut = make_int4(0, 0, 0, 0);
  while (ok && walk.next(p, prefix, g)) {
    if (g.j0 == 0 && g.slot >= 0) cut = make_int4(g.s.q0, g.s.q_len * p.G, g.h, g.last_cta);
    const int n = g.j1 - g.j0;
    const int *row = page_row(p, g);
    auto page_of = [&](int j) -> int {  // n_pages (read as zeros) where there is none
      if (lane >= boxes) return 0;
      const int i = small ? j * boxes + lane : (j * kRowsPerTile) >> p.page_log2;
      int e = -1;
      if ((i << p.page_log2) < g.s.kv_len) e = row[i];
      return e >= 0 && e < p.cache.n_pages ? e : p.cache.n_pages;
    };
    const int qb = nq % sh.q_bufs, use = nq / sh.q_bufs;
    bool q_due = true;  // this segment's Q is still to be loaded
    int page = page_of(g.j0);
    for (int f = 0; f < 2 * n && ok; ++f, ++fills) {
      // Q as soon as its buffer is free, but K and V go ahead of it meanwhile:
      // the slots of the first fills are given back by earlier segments
      if (lane == 0 && q_due &&
          (use == 0 || f >= sh.stages / 2 || f == 2 * n - 1 || mbar_test(bar(C::kQEmpty + qb), (use - 1) & 1))) {
        ok = use == 0 || mbar_wait(bar(C::kQEmpty + qb), (use - 1) & 1, abort_flag, err);
        if (ok) {
          ++q_loads;
          mbar_arrive_expect_tx(bar(C::kQFull + qb), q_bytes);
          for (int cb = 0; cb < C::kColBlocks; ++cb)
            tma_load_4d_hint(smem + sh.q_at() + qb * sh.q_bytes() + cb * sh.N * 128, tm_q, bar(C::kQFull + qb), cb * 64, 0,
                             g.s.q0, g.h, pol_q);
        }
        q_due = false;
      }
      const int j = g.j0 + (f >> 1), which = f & 1;
      const int now = page;
      if (lane == 0 && ok) {
        ok = fills < sh.stages || mbar_wait(bar(C::kEmpty + at.slot), at.phase ^ 1u, abort_flag, err);
        if (ok) mbar_arrive_expect_tx(bar(C::kFull + at.slot), C::kTileBytes);
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      if (lane < boxes) {
        const CUtensorMap *map = which ? tm_v : tm_k;
        const int in_page = small ? 0 : (j * kRowsPerTile) & (page_size - 1);
#pragma unroll
        for (int cb = 0; cb < C::kColBlocks; ++cb)
          tma_load_4d_hint(smem + at.slot * C::kTileBytes + cb * kColBlockBytes + lane * box_bytes, map,
                           bar(C::kFull + at.slot), cb * 64, in_page, g.h, now, pol_kv);
      }
      if (which && f + 1 < 2 * n) page = page_of(j + 1);
      at = at.next(sh.stages);
    }
    ++nq;
  }
  if (lane == 0) {
    p.cuts[blockIdx.x] = cut;
    // every copy must have landed before the CTA may exit
    for (int i = max(0, q_loads - sh.q_bufs); i < q_loads; ++i)
      mbar_drain(bar(C::kQFull + i % sh.q_bufs), (i / sh.q_bufs) & 1, err);
    for (long long i = max(0ll, fills - sh.stages); i < fills; ++i)
      mbar_drain(bar(C::kFull + static_cast<int>(i % sh.stages)), static_cast<uint32_t>(i / sh.stages) & 1u, err);
  }
  __syncwarp();
}

// MMA issuer: one thread.
template <int D>
__device__ __noinline__ void narrow_issuer(const PagedAttnParams &p, const Narrow<D> &sh, Walk walk, const int *prefix,
                                           uint32_t bar0, uint32_t smem, uint32_t tmem, volatile int *abort_flag,
                                           int *err) {
  using C = Narrow<D>;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  const uint32_t idesc_s = idesc_narrow(sh.N, false), idesc_o = idesc_narrow(sh.N, true);
  const uint32_t o_col = tmem + 2 * sh.N;
  const uint64_t pd = sw128_desc(smem + sh.p_at(), kColBlockBytes, 1024);
  RingPos k{0, 0};
  uint32_t step = 0;  // key tiles so far
  int nq = 0;
  bool ok = true;
  Segment g;
  while (ok && walk.next(p, prefix, g)) {
    const int n = g.j1 - g.j0;
    const int qb = nq % sh.q_bufs;
    if (!mbar_wait(bar(C::kQFull + qb), (nq / sh.q_bufs) & 1, abort_flag, err)) break;
    ++nq;
    const uint64_t qd = sw128_desc(smem + sh.q_at() + qb * sh.q_bytes(), 16, 1024);
    const uint64_t q_block = static_cast<uint64_t>((sh.N * 128) >> 4);  // from one 64-column block to the next
    auto scores = [&](const RingPos &at, uint32_t to, bool last) {
      const uint64_t kd = sw128_desc(smem + at.slot * C::kTileBytes, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss(tmem + (to & 1u) * sh.N, kd + static_cast<uint64_t>(((kk / 4) * kColBlockBytes + (kk % 4) * 32) >> 4),
               qd + (kk / 4) * q_block + static_cast<uint64_t>((kk % 4) * 2), idesc_s, kk > 0 ? 1u : 0u);
      mma_commit(bar(C::kSFull + (to & 1u)));
      mma_commit(bar(C::kEmpty + at.slot));
      if (last) mma_commit(bar(C::kQEmpty + qb));
    };
    if (!mbar_wait(bar(C::kFull + k.slot), k.phase, abort_flag, err)) break;
    scores(k, step, n == 1);
    for (int j = 0; j < n; ++j, ++step) {
      const RingPos v = k.next(sh.stages), k1 = v.next(sh.stages);
      // the next scores ahead of this product if their keys are there; their
      // buffer was read before P of the tile before this one was signalled
      const bool early = j + 1 < n && mbar_test(bar(C::kFull + k1.slot), k1.phase);
      if (early) scores(k1, step + 1, j + 2 == n);
      if (!mbar_wait(bar(C::kPFull), step & 1u, abort_flag, err) ||
          !mbar_wait(bar(C::kFull + v.slot), v.phase, abort_flag, err)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // V as stored, [key][column], is the M-major A operand; for D = 64 the
      // upper 64 rows of the product read the bytes behind the tile and are
      // never looked at (rows of a product do not mix)
      const uint64_t vd = sw128_desc(smem + v.slot * C::kTileBytes, kColBlockBytes, 1024);
#pragma unroll
      for (int kk = 0; kk < kRowsPerTile / 16; ++kk)
        mma_ss(o_col, vd + static_cast<uint64_t>(kk * 128), pd + static_cast<uint64_t>(kk * 128), idesc_o,
               (j > 0 || kk > 0) ? 1u : 0u);
      mma_commit(bar(C::kEmpty + v.slot));
      mma_commit(bar(C::kPvDone));
      if (j + 1 < n && !early) {
        if (!mbar_wait(bar(C::kFull + k1.slot), k1.phase, abort_flag, err)) {
          ok = false;
          break;
        }
        scores(k1, step + 1, j + 2 == n);
      }
      k = k1;
    }
  }
  mma_commit(bar(C::kMmaDone));
  mbar_drain(bar(C::kMmaDone), 0, err);
}

// Floats as ints of the same order (finite values and infinities), and back.
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// Softmax and epilogue of columns [col0, col0 + C) of S^T: one thread per key
// (and, in the epilogue, per column of O). `red` is this warpgroup's 4 x C
// floats of shared memory, `gi` its number. Every warp goes through the same
// barriers whatever fails: a wait that runs out is carried to the next vote.
template <int D, int C>
__device__ __noinline__ void narrow_softmax(const PagedAttnParams &p, const Narrow<D> &sh, Walk walk, const int *prefix,
                                            int gi, uint32_t bar0, uint32_t smem, uint32_t tmem, float *red,
                                            volatile int *abort_flag, int *err) {
  using L = Narrow<D>;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  const int key = threadIdx.x & 127, lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
  const int col0 = gi * C, id = 1 + gi;
  const uint32_t lane_off = static_cast<uint32_t>(32 * w) << 16;
  const uint32_t o_addr = tmem + lane_off + 2 * sh.N + col0;
  const uint32_t p_row = smem + sh.p_at() + key * 128;
  const float c2 = p.scale_log2;
  RingPos k{0, 0};
  uint32_t step = 0;
  Segment g;
  while (walk.next(p, prefix, g)) {
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
      m[c] = -INFINITY;
      l[c] = 0.f;
    }
    int entry = entry_of(g.j0);
    bool ok = true;
    for (int j = 0; j < n; ++j, ++step) {
      const bool there = entry >= 0 && entry < p.cache.n_pages;
      if (j + 1 < n) entry = entry_of(g.j0 + j + 1);
      const int kv0 = (g.j0 + j) * kRowsPerTile;
      ok = ok && __all_sync(0xffffffffu,
                            mbar_wait(bar(L::kSFull + (step & 1u)), (step >> 1) & 1u, abort_flag, err));
      tc_fence_after();
      float x[C];
      {
        uint32_t raw[C];
        if constexpr (C == 16) tmem_ld16(tmem + lane_off + (step & 1u) * sh.N + col0, raw);
        else tmem_ld32(tmem + lane_off + (step & 1u) * sh.N + col0, raw);
        tmem_ld_wait(raw);
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = there ? __uint_as_float(raw[c]) * c2 : -INFINITY;
      }
      if (kv0 + kRowsPerTile - 1 > first_last) {  // some row does not see all keys of the tile
        int tok = col0 / p.G, head = col0 - tok * p.G;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int last = p.causal ? min(first_last + tok, g.s.kv_len - 1) : first_last;
          if (kv0 + key > last) x[c] = -INFINITY;
          if (++head == p.G) {
            head = 0;
            ++tok;
          }
        }
      }
      bool move = false;
#pragma unroll
      for (int c = 0; c < C; ++c) move = move || x[c] > m[c] + 8.f;
      if (!named_bar_and(id, 128, ok && !move)) {
        // maxima of the tile's 128 keys, then O and l onto the new reference
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float top = from_ordered(__reduce_max_sync(0xffffffffu, ordered(x[c])));
          if (lane == 0) red[w * C + c] = top;
        }
        ok = named_bar_and(id, 128, ok);
        if (ok && j > 0)
          ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kPvDone), (step - 1) & 1u, abort_flag, err));
        tc_fence_after();
        const bool old = ok && j > 0;  // O holds the sum of the tiles before
        uint32_t v[C] = {};
        if (old) {
          if constexpr (C == 16) tmem_ld16(o_addr, v);
          else tmem_ld32(o_addr, v);
          tmem_ld_wait(v);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float top = fmaxf(fmaxf(red[c], red[C + c]), fmaxf(red[2 * C + c], red[3 * C + c]));
          const float m_new = fmaxf(m[c], top);
          const float alpha = m_new == -INFINITY ? 1.f : ex2_approx(m[c] - m_new);
          m[c] = m_new;
          l[c] *= alpha;
          v[c] = __float_as_uint(__uint_as_float(v[c]) * alpha);
        }
        if (old) {
          if constexpr (C == 16) tmem_st16(o_addr, v);
          else tmem_st32(o_addr, v);
          tmem_st_wait();
        }
      }
      uint32_t pk[C / 2];
#pragma unroll
      for (int c = 0; c < C; c += 2) {
        const float a = ex2_approx(x[c] - (m[c] == -INFINITY ? 0.f : m[c]));
        const float b = ex2_approx(x[c + 1] - (m[c + 1] == -INFINITY ? 0.f : m[c + 1]));
        l[c] += a;
        l[c + 1] += b;
        // P enters the tensor cores in bf16, as in the dense forward; l is summed before the rounding
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        pk[c / 2] = *reinterpret_cast<uint32_t *>(&h);
      }
      // the product of the tile before has read P
      if (j > 0)
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(L::kPvDone), (step - 1) & 1u, abort_flag, err));
      if (ok) {
#pragma unroll
        for (int i = 0; i < C / 8; ++i)
          st_shared_v4(p_row + (static_cast<uint32_t>((col0 / 8 + i) ^ (key & 7)) << 4), pk[4 * i], pk[4 * i + 1],
                       pk[4 * i + 2], pk[4 * i + 3]);
        const RingPos v = k.next(sh.stages);
        if (gi == 0 && g.s.kv_len - kv0 < kRowsPerTile)
          ok = clear_tail<D>(g.s.kv_len - kv0, smem + v.slot * L::kTileBytes, bar(L::kFull + v.slot), v.phase, abort_flag,
                             err);
        fence_proxy_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kPFull));  // one arrival per warp
      }
      k = k.next(sh.stages).next(sh.stages);
    }
    ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(L::kPvDone), (step - 1) & 1u, abort_flag, err));
    tc_fence_after();
    // l over the keys: the warps' sums through shared memory
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float s = l[c];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      l[c] = s;
    }
    named_bar_sync(id, 128);  // red has been read
    if (lane == 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) red[w * C + c] = l[c];
    }
    if (!named_bar_and(id, 128, ok)) return;
#pragma unroll
    for (int c = 0; c < C; ++c) l[c] = (red[c] + red[C + c]) + (red[2 * C + c] + red[3 * C + c]);
    uint32_t v[C];
    if constexpr (C == 16) tmem_ld16(o_addr, v);
    else tmem_ld32(o_addr, v);
    tmem_ld_wait(v);
    const size_t part = static_cast<size_t>(max(g.slot, 0)) * p.part_rows;
    int tok = col0 / p.G, head = col0 - tok * p.G;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (col0 + c < rows) {
        const float inv = l[c] > 0.f ? 1.f / l[c] : 0.f;
        const float o = __uint_as_float(v[c]) * inv;
        const float lse = l[c] > 0.f ? (m[c] + log2f(l[c])) * kLn2 : -INFINITY;
        if (g.slot >= 0) {
          if (key < D) p.part_o[(part + col0 + c) * D + key] = o;
          if (key == c) p.part_lse[part + col0 + c] = lse;
        } else {
          const int h = g.h * p.G + head, row = g.s.q0 + tok;
          if (key < D) static_cast<__nv_bfloat16 *>(p.o)[h * p.o_h + row * p.o_s + key] = __float2bfloat16_rn(o);
          if (key == c && p.lse) p.lse[static_cast<size_t>(h) * p.total_q + row] = lse;
        }
      }
      if (++head == p.G) {
        head = 0;
        ++tok;
      }
    }
  }
}

}  // namespace paged
}  // namespace seqattn
