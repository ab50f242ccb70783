// Attention of new tokens over a paged K/V cache held in e4m3 (included by attn_kernel.cu).
//
// The same work, dealt out the same way, as over a bf16 cache (attn_paged.cuh): items,
// ranges of equal cost, the walk, the merge are shared, and the two forms. What
// differs is how tiles of 8-bit codes meet the tensor cores, whose 8-bit
// instructions want both operands in 8 bits and whose 16-bit ones both in 16.
//
// Narrow form (memory bound), in 8 bits:
//   S = Q K^T   on the codes as they lie in shared memory. A row of Q, after a power of
//     two that brings its largest element to [128, 256), is the sum of two e4m3 numbers
//     an element, the nearest one and the nearest of what that leaves: bf16 has 8
//     significant bits, e4m3 4, and the remainder needs no more than 4. The powers of
//     two and the keys' scales multiply the fp32 scores.
//   O = P V   wants every weight scaled by its value's scale (V is read by columns, its
//     scales belong to rows): w = 2^(s_j + e_j - E - m), E an exponent that the tiles of a
//     segment share. The column's reference m follows the largest s_j + e_j - E, what a
//     key brings to O, and not the largest s_j: a key of much weight and next to no value,
//     the first of many long contexts, takes no bits from the others, and neither does a
//     large value of no weight. Sums l are of 2^(s_j - m), in fp32. w 2^11, rounded to
//     fp16, is three e5m2 numbers (fp16's upper byte; that of the rest; the rest of that
//     to nearest, times 2^4), three bits each, in columns of their own, so that V is read
//     once for all: 2^-9 of a weight, as bf16 gives, down to 2^-23 of the column's largest,
//     and steps of 2^-31 of that below. (As two e4m3 numbers, steps of 2^-18: batch decoding
//     177 us, now 183 to 186, trees of up to 64 rows 143, now 148 to 157; but of the answer behind a
//     first key 12 nats above 8,191 others 3 to 5 % was lost, 14 above 16,383 half of it.)
// Wide form (compute bound), in fp16, which holds codes and ratios of scales: warps of their
// own turn K and V tiles, K to a unit of the tile's, V to one that fits many tiles
// (value_unit), on their way into the ring of the bf16 form; Q goes there after its rows'
// powers of two. The softmax has a factor more a tile and none an element, and references
// that fall as well as rise, as fp16's weights need (kLeastSum). (Scales applied to scores and weights by the softmax
// warps instead, read from shared memory: 6,700 clocks a pair of tiles, 1,554 us for
// 1,024 tokens behind 65,536 keys.)
//
// Measured (GB300): 64 sequences' next tokens over 300 to 16,000 keys (1.06 GB, 8 KV
// heads of 128) 185 us = 5.7 TB/s; 1,024 tokens behind 65,536 keys, 32 heads over 8 of
// 128, 874 us = 1,268 TFLOP/s.
#pragma once

namespace seqattn {
namespace paged8 {

using namespace detail;
using paged::codes::largest_of;
using paged::codes::row_scale;
using paged::codes::RowScale;
using paged::codes::two_to;
using paged::Items;
using paged::Line;
using paged::PageWindow;
using paged::Segment;
using paged::Seq;
using paged::Walk;

// Warps 0-7 softmax, 8 and 10 MMA issuers, 9 producer (narrow) or walk (wide), 12-15
// turners (wide). The softmax warps take registers over from the issuers' warpgroup.
constexpr int kThreads8 = 512;
constexpr int kMmaWarp = 8, kTmaWarp = 9, kMmaWarp1 = 10, kTurners = 12;
constexpr int kSoftmaxRegs = 184, kIssuerRegs = 56, kTurnerRegs = 88;
static_assert(2 * kSoftmaxRegs + kIssuerRegs + kTurnerRegs <= 4 * (65536 / kThreads8), "registers of the four warpgroups");
// Cost of a narrow tile in wide ones (as kNarrowUnit of the bf16 form), by its rows. At
// 0.29, 0.32, 0.34, 0.36, 0.40: 60 and 63 single tokens beside a piece of 512, and 20 pairs beside
// two pieces of 700, in all 584, 569, 555, 562, 609 us; 30 fours of 28 rows beside a piece of 512 at
// 0.36, 0.4, 0.45, 0.5: 105, 105, 97, 100; 20 drafts of 35 rows beside two pieces of 300, 40 of 32
// beside one of 700, 32 trees of 6 to 60 drafts, in all, at 0.65, 0.76, 0.8, 0.85: 593, 545, 557, 588.
__device__ __forceinline__ float narrow_unit8(int rows) { return rows <= 16 ? 0.34f : (rows <= 32 ? 0.45f : 0.77f); }

template <int D>
struct Cfg8 {
  using Wide = paged::Cfg<D>;
  static constexpr int kTileBytes = kRowsPerTile * D;       // of codes
  static constexpr int kMaxStages = 196608 / kTileBytes;    // narrow ring
  // narrow: ring, P, Q, reductions; wide: Q, ring, codes (the epilogue goes through the
  // place of Q, whose products are done then)
  static constexpr int kCodesAt = (2 + Wide::kStages) * Wide::kTileBytes, kCodesBytes = 64 * D;  // of a turner
  static constexpr int kRedAt = 196608 + 16384 + 8192, kRedBytes = 2 * 1024;
  static constexpr int kAreaBytes =
      kCodesAt + 4 * kCodesBytes > kRedAt + kRedBytes ? kCodesAt + 4 * kCodesBytes : kRedAt + kRedBytes;
  static_assert(4 * 2560 <= Wide::kTileBytes, "epilogue in the place of Q");
  static constexpr int kItemBarrier = 2 * kMaxStages + 10, kMaxBarriers = kItemBarrier + 8;
  static constexpr int kPrefixAt = Wide::kPrefixAt;         // inside the ring of either form
  static_assert(kPrefixAt + 4 * (kPagedMaxSeqs + 1) <= 131072, "prefix sums inside the narrow ring");
  // behind them: barriers, three words, segments, the wide form's exponents and factors (before: sums over warps)
  static constexpr int kSmallBytes = 4 * 32 + 4 * 256;
  static constexpr int kSmemBytes = 1024 + kAreaBytes + 8 * kMaxBarriers + 16 + 4 * 48 + kSmallBytes;
};
static_assert(Cfg8<128>::kSmemBytes <= 232448 && Cfg8<64>::kSmemBytes <= 232448, "shared memory per CTA");

// Descriptors of tiles whose rows are D bytes: atoms of eight rows, swizzled over
// the whole row. `next`: from one block of D columns to the next, of an operand
// stored by columns (M- or N-contiguous) that is wider than that.
template <int D>
__device__ __forceinline__ uint64_t code_desc(uint32_t at, uint32_t next) {
  return D == 128 ? sw128_desc(at, next, 1024) : sw64_desc(at, next, 512);
}
// Byte of 16-byte piece c of row r of such a tile.
template <int D>
__device__ __forceinline__ uint32_t piece_of(int r, int c) {
  return r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

// Eight elements (bf16 pairs) times `up`: eight codes each of the two numbers.
__device__ __forceinline__ void split_codes(const uint4 &x, float up, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[2], l[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t w = u[2 * i + k];
      // fp16 holds them: eight significant bits, sizes below 256 (and what it loses below 2^-17 e4m3 does not have)
      const uint32_t y = f16x2_of_floats(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
      h[k] = e4m3x2_of_f16x2(y);
      l[k] = e4m3x2_of_f16x2(sub_f16x2(y, f16x2_of_e4m3x2(h[k])));
    }
    hi[i] = h[0] | h[1] << 16;
    lo[i] = l[0] | l[1] << 16;
  }
}
constexpr int kNoExponent = -10000;  // of a key that is not there

// The table entry of a thread's key in tile j of a segment, -1 past the end.
__device__ __forceinline__ int entry_of(const PagedAttnParams &p, const int *table, int kv_len, int j, int key) {
  const int pos = j * kRowsPerTile + key;
  return pos < kv_len ? table[pos >> p.page_log2] : -1;
}
// The scales of this thread's key in every kStep-th tile of a segment, one of those
// tiles ahead, and the table entry that they need two ahead, so that neither load is
// waited for.
template <int kStep>
struct KeyScales {
  const PagedAttnParams &p;
  const int *table;
  int kv_len, key;
  const unsigned char *k_scales, *v_scales;  // of the KV head
  int entry;           // of the tile after the next
  bool there, next_there;
  unsigned kb, vb, next_kb, next_vb;
  // first: the entry of tile j
  __device__ __forceinline__ KeyScales(const PagedAttnParams &p_, const Segment &g, int key_, int j, int first)
      : p(p_), table(paged::page_row(p_, g)), kv_len(g.s.kv_len), key(key_),
        k_scales(p_.scales.k + (static_cast<long long>(g.h) << p_.page_log2)),
        v_scales(p_.scales.v + (static_cast<long long>(g.h) << p_.page_log2)), entry(first) {
    load(j);
    entry = entry_of(p, table, kv_len, j + kStep, key);
    there = false;
    kb = vb = 0;
  }
  __device__ __forceinline__ void load(int j) {
    next_there = entry >= 0 && entry < p.cache.n_pages;
    next_kb = next_vb = 127;
    if (next_there) {
      const long long from = entry * p.scales.page_stride + ((j * kRowsPerTile + key) & ((1 << p.page_log2) - 1));
      next_kb = k_scales[from];
      next_vb = v_scales[from];
    }
  }
  // On to tile j; the first one first.
  __device__ __forceinline__ void step(int j) {
    there = next_there;
    kb = next_kb;
    vb = next_vb;
    load(j + kStep);
    entry = entry_of(p, table, kv_len, j + 2 * kStep, key);
  }
  __device__ __forceinline__ int exponent() const { return there ? static_cast<int>(max(vb, 1u)) - 127 : kNoExponent; }
};

// K and V of a key tile to ring slots `k` and `v`, each when it is free: pages of whole
// rows of D bytes, their ids found once for both. (A part at a time, ids found for
// each, the producer took 850 clocks a part, 1,700 a tile: more than the bytes.)
// Returns how many of the two are on their way.
struct TileSlots {
  uint32_t k, v, k_full, v_full, k_empty, v_empty, k_phase, v_phase;
  bool k_used, v_used;  // the slot has been filled before
};
template <int D, int kBoxes>
__device__ __forceinline__ int load_tile8(const TileSlots &t, const CUtensorMap *tm_k, const CUtensorMap *tm_v, int in_page,
                                           int head, int page, uint32_t box_bytes, bool leader, uint64_t pol,
                                           volatile int *abort_flag, int *err) {
  int pg[kBoxes];
#pragma unroll
  for (int i = 0; i < kBoxes; ++i) pg[i] = uniform(__shfl_sync(0xffffffffu, page, i));
  if (t.k_used && !__all_sync(0xffffffffu, mbar_wait(t.k_empty, t.k_phase, abort_flag, err))) return 0;
  if (leader) {
    mbar_arrive_expect_tx(t.k_full, Cfg8<D>::kTileBytes);
#pragma unroll
    for (int i = 0; i < kBoxes; ++i) tma_load_4d_hint(t.k + i * box_bytes, tm_k, t.k_full, 0, in_page, head, pg[i], pol);
  }
  __syncwarp();
  if (t.v_used && !__all_sync(0xffffffffu, mbar_wait(t.v_empty, t.v_phase, abort_flag, err))) return 1;
  if (leader) {
    mbar_arrive_expect_tx(t.v_full, Cfg8<D>::kTileBytes);
#pragma unroll
    for (int i = 0; i < kBoxes; ++i) tma_load_4d_hint(t.v + i * box_bytes, tm_v, t.v_full, 0, in_page, head, pg[i], pol);
  }
  __syncwarp();
  return 2;
}

// Producer of the narrow form: the whole warp. K and V tiles in turn through a ring of
// `stages` slots, their barriers `full` and `empty` on.
template <int D>
__device__ __forceinline__ void narrow_producer8(const PagedAttnParams &p, Walk walk, Segment g, Items items,
                                                 const CUtensorMap *tm_k, const CUtensorMap *tm_v, uint32_t full,
                                                 uint32_t empty, uint32_t ring, int stages_in, int first_entry,
                                                 volatile int *abort_flag, int *err) {
  using C = Cfg8<D>;
  const int lane = threadIdx.x & 31;
  const uint64_t pol = l2_policy_evict_first();
  const int page_size = 1 << p.page_log2;
  const bool small = page_size < kRowsPerTile;
  const int boxes = uniform(paged::pages_of_tile(p)), stages = uniform(stages_in);
  const uint32_t box_bytes = uniform((small ? page_size : kRowsPerTile) * static_cast<uint32_t>(D));
  const bool leader = elect_one();
  paged::RingPos at{0, 0};
  int fills = 0;  // of the ring, as far as they count
  bool ok = true, first = true;
  int4 cut = make_int4(0, 0, 0, 0);  // the item that this CTA begins and another one ends, for the merge
  while (ok && walk.next(p, g)) {
    g.ring = 0;  // (of the wide form)
    if (!items.put(g, abort_flag, err)) break;
    if (g.j0 == 0 && g.slot >= 0)
      cut = make_int4(g.s.q0, min(g.s.q_len * p.G, paged::kNarrowRows), g.h, walk.ends_in(p, g));
    const int j0 = uniform(g.j0), n = uniform(g.j1 - g.j0), head = uniform(g.h);
    PageWindow pages(p, g, first, first_entry);
    first = false;
#pragma unroll 1
    for (int j = 0; j < n && ok; ++j) {
      const int page = pages.page(p, j0 + j);
      const int in_page = small ? 0 : ((j0 + j) * kRowsPerTile) & (page_size - 1);
      const paged::RingPos v = at.next(stages);
      const TileSlots t{ring + at.slot * C::kTileBytes, ring + v.slot * C::kTileBytes, full + 8u * at.slot, full + 8u * v.slot,
                        empty + 8u * at.slot, empty + 8u * v.slot, at.phase ^ 1u, v.phase ^ 1u,
                        fills >= stages, fills + 1 >= stages};
      int parts;
      if (boxes == 1) parts = load_tile8<D, 1>(t, tm_k, tm_v, in_page, head, page, box_bytes, leader, pol, abort_flag, err);
      else if (boxes == 2) parts = load_tile8<D, 2>(t, tm_k, tm_v, in_page, head, page, box_bytes, leader, pol, abort_flag, err);
      else if (boxes == 4) parts = load_tile8<D, 4>(t, tm_k, tm_v, in_page, head, page, box_bytes, leader, pol, abort_flag, err);
      else parts = load_tile8<D, 8>(t, tm_k, tm_v, in_page, head, page, box_bytes, leader, pol, abort_flag, err);
      if (j == 0) pages.prefetch(p);
      fills = min(fills + parts, 2 * stages);
      at = parts == 2 ? v.next(stages) : (parts == 1 ? v : at);
      ok = parts == 2;
    }
  }
  g.j0 = g.j1 = 0;
  items.put(g, abort_flag, err);
  if (lane == 0) {
    p.cuts[blockIdx.x] = cut;
    // every copy must have landed before the CTA may exit: the slots filled last, from the ring's position back
    paged::RingPos s = at;
    for (int i = 0; i < min(fills, stages); ++i) {
      s = s.slot == 0 ? paged::RingPos{stages - 1, s.phase ^ 1u} : paged::RingPos{s.slot - 1, s.phase};
      mbar_drain(full + 8u * s.slot, s.phase, err);
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------- the narrow form
template <int D>
struct Narrow8 {
  int N, stages;
  bool turns;  // they take tiles in turn, each with sums, reference and O of its own; else half the columns each
  __device__ __forceinline__ explicit Narrow8(int rows) {
    N = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
    stages = (N == 16 ? 196608 : (N == 32 ? 163840 : 131072)) / Cfg8<D>::kTileBytes;
    turns = N == 16;
  }
  // shared memory: ring, two buffers of P, Q (two parts). A key's 3 N codes of P lie in rows of 128 bytes: half a
  // row a buffer, a row, or two rows a block of 128 columns apart.
  static constexpr int kPBytes = kRowsPerTile * 128;
  __device__ __forceinline__ int p_at() const { return stages * Cfg8<D>::kTileBytes; }
  __device__ __forceinline__ int p_step() const { return N == 16 ? 64 : (N == 32 ? kPBytes : 2 * kPBytes); }
  __device__ __forceinline__ int q_at() const { return p_at() + (N == 16 ? 1 : (N == 32 ? 2 : 4)) * kPBytes; }
  static_assert(196608 + kPBytes + 2 * 16 * D <= Cfg8<D>::kRedAt && 163840 + 2 * kPBytes + 2 * 32 * D <= Cfg8<D>::kRedAt &&
                    131072 + 4 * kPBytes + 2 * 64 * D <= Cfg8<D>::kRedAt,
                "narrow layouts");
  // TMEM columns: two buffers of S, then O, 3 N columns, or with turns two of 48, 64 apart
  static constexpr int kOStep = 64;
  // barriers
  static constexpr int kFull = 0, kEmpty = Cfg8<D>::kMaxStages, kQFull = 2 * Cfg8<D>::kMaxStages, kSFull = kQFull + 1,
                       kPFull = kSFull + 2, kPvDone = kPFull + 2, kScoresDone = kPvDone + 2, kProductsDone = kScoresDone + 1,
                       kNumBarriers = kProductsDone + 1;
  static_assert(kNumBarriers <= Cfg8<D>::kItemBarrier, "barriers");
};

// MMA issuers: whole warps, their code uniform, one lane for the products. One has the
// scores, one the products with V. (One warp for both took 1,700 clocks a tile, most of it
// on its own way through issues and waits: 188 us for the batch that takes 156 to read.)
template <int D>
__device__ __forceinline__ void narrow_scores8(const Narrow8<D> &sh, Items items, uint32_t bar0, uint32_t smem,
                                               uint32_t tmem_in, volatile int *abort_flag, int *err) {
  using C = Cfg8<D>;
  using L = Narrow8<D>;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  auto wait = [&](int i, uint32_t phase) {
    return __all_sync(0xffffffffu, mbar_wait(bar(i), phase, abort_flag, err));
  };
  const bool leader = elect_one();
  const uint32_t tmem = uniform(tmem_in), N = uniform(static_cast<uint32_t>(sh.N));
  const int stages = uniform(sh.stages);
  const uint32_t q_at = smem + uniform(static_cast<uint32_t>(sh.q_at()));
  const uint32_t idesc_s = idesc_e4m3_f32(128, 0, false, false) | (N >> 3) << 17;
  const uint64_t qd = code_desc<D>(q_at, 16), q_lo = static_cast<uint64_t>((N * D) >> 4);
  paged::RingPos k{0, 0};
  uint32_t step = 0;  // key tiles so far
  uint32_t nq = 0;
  bool ok = true;
  while (ok && items.wait(abort_flag, err)) {
    const int n = uniform(items.get().j1 - items.get().j0);
    items.release();
    if (!wait(L::kQFull, nq & 1u)) break;
    ++nq;
    for (int j = 0; j < n; ++j, ++step) {
      // the scores' buffer was read before P of its last tile was signalled
      if (!wait(L::kFull + k.slot, k.phase) || (step >= 2 && !wait(L::kPFull + (step & 1u), ((step >> 1) - 1) & 1u))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint64_t kd = code_desc<D>(smem + k.slot * C::kTileBytes, 16);
      const uint32_t s_col = tmem + (step & 1u) * N;
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
          mma_ss_e4m3(s_col, kd + 2 * kk, qd + 2 * kk, idesc_s, kk > 0 ? 1u : 0u);
          mma_ss_e4m3(s_col, kd + 2 * kk, qd + q_lo + 2 * kk, idesc_s, 1u);
        }
        mma_commit(bar(L::kSFull + (step & 1u)));
        mma_commit(bar(L::kEmpty + k.slot));
      }
      __syncwarp();
      k = k.next(stages).next(stages);
    }
  }
  if (leader) {
    mma_commit(bar(L::kScoresDone));
    mbar_drain(bar(L::kScoresDone), 0, err);
  }
  __syncwarp();
}
template <int D>
__device__ __forceinline__ void narrow_products8(const Narrow8<D> &sh, Items items, uint32_t bar0, uint32_t smem,
                                                 uint32_t tmem_in, volatile int *abort_flag, int *err) {
  using C = Cfg8<D>;
  using L = Narrow8<D>;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  auto wait = [&](int i, uint32_t phase) {
    return __all_sync(0xffffffffu, mbar_wait(bar(i), phase, abort_flag, err));
  };
  const bool leader = elect_one();
  const uint32_t tmem = uniform(tmem_in), N = uniform(static_cast<uint32_t>(sh.N));
  const int stages = uniform(sh.stages);
  const uint32_t p_at = smem + stages * C::kTileBytes, p_step = uniform(static_cast<uint32_t>(sh.p_step()));
  const uint32_t idesc_o = idesc_e4m3_e5m2_f32(128, 0, true, true) | (3 * N >> 3) << 17;
  const bool turns = N == 16;
  paged::RingPos v{1, 0};
  uint32_t step = 0;  // key tiles so far
  bool ok = true;
  while (ok && items.wait(abort_flag, err)) {
    const int n = uniform(items.get().j1 - items.get().j0);
    items.release();
    for (int j = 0; j < n; ++j, ++step) {
      if (!wait(L::kFull + v.slot, v.phase) || !wait(L::kPFull + (step & 1u), (step >> 1) & 1u)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // V as stored, [key][column], is the M-major A operand; for D = 64 the upper 64
      // rows of the product read the tile behind it and are never looked at
      const uint64_t vd = code_desc<D>(smem + v.slot * C::kTileBytes, C::kTileBytes);
      const uint64_t pd = sw128_desc(p_at + (step & 1u) * p_step, L::kPBytes, 1024);
      const uint32_t add = j > (turns ? 1 : 0) ? 1u : 0u, o_col = tmem + 2 * N + (turns ? (step & 1u) * L::kOStep : 0u);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < kRowsPerTile / 32; ++kk)
          mma_ss_e4m3(o_col, vd + static_cast<uint64_t>(kk * 2 * D), pd + static_cast<uint64_t>(kk * 256), idesc_o,
                      kk > 0 ? 1u : add);
        mma_commit(bar(L::kEmpty + v.slot));
        mma_commit(bar(L::kPvDone + (step & 1u)));
      }
      __syncwarp();
      v = v.next(stages).next(stages);
    }
  }
  if (leader) {
    mma_commit(bar(L::kProductsDone));
    mbar_drain(bar(L::kProductsDone), 0, err);
  }
  __syncwarp();
}

// V slots past kv_len may hold any code, NaN too: zeroed before the product reads them.
template <int D>
__device__ __forceinline__ bool clear_tail8(int valid_keys, uint32_t v, uint32_t bar_full, uint32_t phase,
                                            volatile int *abort_flag, int *err) {
  if (!__all_sync(0xffffffffu, mbar_wait(bar_full, phase, abort_flag, err))) return false;
  for (int i = valid_keys * D + 16 * (threadIdx.x & 127); i < kRowsPerTile * D; i += 16 * 128)
    st_shared_v4(v + i, 0u, 0u, 0u, 0u);
  fence_proxy_async_shared();
  return true;
}

// Four weights to the codes of their three numbers (see the top of the file): the upper bytes of their fp16 forms,
// those of what these leave, and what both leave times 2^4, to the nearest code.
__device__ __forceinline__ void split_weights(const float (&a)[4], uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  const uint32_t w0 = f16x2_of_floats(a[0], a[1]), w1 = f16x2_of_floats(a[2], a[3]);
  auto upper = [](uint32_t x, uint32_t y) { return __byte_perm(x, y, 0x7531); };
  auto rest = [](uint32_t x) { return sub_f16x2(x, x & 0xff00ff00u); };  // exact
  hi = upper(w0, w1);
  const uint32_t r0 = rest(w0), r1 = rest(w1);
  mid = upper(r0, r1);
  lo = e5m2x2_of_f16x2(mul_f16x2(rest(r0), 0x4c004c00u)) | e5m2x2_of_f16x2(mul_f16x2(rest(r1), 0x4c004c00u)) << 16;  // 16, 16
}
constexpr float kLastPart = 0.0625f;  // the third number's unit
constexpr int kWeightUnit = 11;       // a weight of 1 as a code: 2^11

// This thread's share of a segment's rows of Q, eight threads a row, 16 rows from
// col0 + h on: asked for, and brought to shared memory as codes of two numbers.
template <int D>
struct RowsOfQ {
  static constexpr int kVecs = D / 64;  // 8 elements each
  uint4 x[kVecs];
  __device__ __forceinline__ void load(const PagedAttnParams &p, const Segment &g, int col, int key) {
    const int r = col + (key >> 3), sub = key & 7;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < g.s.q_len * p.G) {
      const int tok = r / p.G;
      const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + (g.h * p.G + r - tok * p.G) * p.q_h +
                               (g.s.q0 + tok) * p.q_s + sub * (D / 8);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) x[i] = reinterpret_cast<const uint4 *>(q)[i];
    }
  }
  // To row `col` + key / 8 of the tile at `to` (parts `part` bytes apart); the row's unit to back[key / 8].
  __device__ __forceinline__ void put(const PagedAttnParams &p, int col, int key, uint32_t to, uint32_t part, float *back) const {
    const int r = col + (key >> 3), sub = key & 7;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) top = fmaxf(top, largest_of(x[i]));
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const RowScale rs = row_scale(top, p.scale_log2);
    uint32_t hi[kVecs][2], lo[kVecs][2];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) split_codes(x[i], rs.up, hi[i], lo[i]);
    if constexpr (D == 128) {
      const uint32_t at = to + piece_of<D>(r, sub);
      st_shared_v4(at, hi[0][0], hi[0][1], hi[1][0], hi[1][1]);
      st_shared_v4(at + part, lo[0][0], lo[0][1], lo[1][0], lo[1][1]);
    } else {
      const uint32_t at = to + piece_of<D>(r, sub >> 1) + 8 * (sub & 1);
      st_shared_v2(at, hi[0][0], hi[0][1]);
      st_shared_v2(at + part, lo[0][0], lo[0][1]);
    }
    if (sub == 0) back[key >> 3] = rs.back;
  }
};

// What a warpgroup leaves in its 256 floats of shared memory, C columns.
template <int C>
struct Reductions {
  float *red, *ref, *factor, *back;  // of the warps (4 C); of the columns: reference, a factor, score unit
  int *tops;                         // of the warps: largest exponent of a tile's values
  __device__ __forceinline__ explicit Reductions(float *at)
      : red(at), ref(at + 4 * C), factor(at + 5 * C), back(at + 6 * C), tops(reinterpret_cast<int *>(at + 7 * C)) {}
};

// Softmax and epilogue, and rows of Q: the scheme of the bf16 narrow form (one thread
// per key, and in the epilogue per column of O). With kTurns a warpgroup has every
// second tile and all C = N columns: two tiles are under way at a time (one
// warpgroup's 1,900 clocks a tile were above the 1,465 that its bytes take), and the
// first warpgroup, which also brings Q, joins both's results in the epilogue. Else it
// has every tile and columns [gi C, gi C + C). `reds`: 256 floats for each warpgroup.
template <int D, int C, bool kTurns>
__device__ __forceinline__ void narrow_softmax8(const PagedAttnParams &p, const Narrow8<D> &sh, Items items, int gi,
                                                uint32_t bar0, uint32_t smem, uint32_t tmem, float *reds,
                                                volatile int *abort_flag, int *err) {
  using L = Narrow8<D>;
  constexpr int kStep = kTurns ? 2 : 1;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  const int key = threadIdx.x & 127, lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
  const int col0 = kTurns ? 0 : gi * C, id = 1 + gi;
  const bool brings_q = !kTurns || gi == 0;
  const uint32_t lane_off = static_cast<uint32_t>(32 * w) << 16;
  const uint32_t o_addr = tmem + lane_off + 2 * sh.N + col0 + (kTurns ? gi * L::kOStep : 0);
  auto product_done = [&](uint32_t s) {  // of key tile s, and so of all before it
    return __all_sync(0xffffffffu, mbar_wait(bar(L::kPvDone + (s & 1u)), (s >> 1) & 1u, abort_flag, err));
  };
  auto larger = [](float a, float b) { return fmaxf(a, b); };
  auto sum_of = [](float a, float b) { return a + b; };
  const Reductions<C> mine(reds + 256 * gi);
  const float *back = Reductions<C>(reds + (kTurns ? 0 : 256 * gi)).back;
  // In powers of two: how far w may pass 1 (fp16 ends at 2^5 of it); how far 2^(s - m) may, and so, with as much
  // room, a value's scale counts in the reference; and how far a reference may fall behind its highest, as it
  // does when E rises. Together they hold l, of up to 2^30 keys, below 2^126.
  constexpr float kMost = 4.f, kFar = 48.f;
  constexpr int kFall = 48;
  // scores from here on lie 4 apart and more: their references are scores, without a scale, which would be rounded to
  // as much (up to 2^kFar, and fp16 ends at 2^5)
  constexpr float kLarge = 0x1p25f;
  paged::RingPos k{0, 0};       // of the segment's first K tile
  uint32_t first_step = 0;      // key tiles of the segments before
  uint32_t nq = 0;
  RowsOfQ<D> q[C / 16];
  int next_entry = -1;
  bool asked = false;           // the next segment's rows of Q and first entry are on their way
  // the first of this warpgroup's tiles in a segment that begins at step s
  auto first_of = [&](uint32_t s) { return kTurns ? static_cast<int>((s ^ static_cast<uint32_t>(gi)) & 1u) : 0; };
  auto ask = [&](const Segment &g, uint32_t s) {
    next_entry = entry_of(p, paged::page_row(p, g), g.s.kv_len, g.j0 + first_of(s), key);
    if (brings_q) {
#pragma unroll
      for (int h = 0; h < C; h += 16) q[h / 16].load(p, g, col0 + h, key);
    }
  };
  // (in turns the warpgroups take an item together or leave together, and the second
  // waits here until the first has done with its results)
  while (kTurns ? named_bar_and(4, 256, items.wait(abort_flag, err)) : items.wait_together(id, abort_flag, err)) {
    if (kTurns) tc_fence_after();  // the first warpgroup's loads of the second's O, ahead of its next product
    const Segment g = items.get();
    items.release();
    const int n = g.j1 - g.j0, rows = g.s.q_len * p.G, j_first = first_of(first_step);
    if (!asked) ask(g, first_step);
    asked = false;
    KeyScales<kStep> scale(p, g, key, g.j0 + j_first, next_entry);
    // (every product that read the rows of Q before is done)
    if (brings_q) {
#pragma unroll
      for (int h = 0; h < C; h += 16)
        q[h / 16].put(p, col0 + h, key, smem + sh.q_at(), static_cast<uint32_t>(sh.N * D), mine.back + h);
      fence_proxy_async_shared();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kQFull));  // one arrival per warp
    }
    const bool tree = paged::is_tree(p, g.s);
    const int first_last = p.causal ? g.s.kv_len - g.s.q_len - (tree ? 1 : 0) : g.s.kv_len - 1;
    float l[C];
#pragma unroll
    for (int c = 0; c < C; ++c) l[c] = 0.f;
    if (key < C) mine.ref[key] = paged::kNoReference;
    int top_e = kNoExponent;  // E
    float highest = paged::kNoReference;  // of the reference of column `key`
    bool ok = true;
    // `back` is there
    if (kTurns && gi != 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kQFull), nq & 1u, abort_flag, err));
    ++nq;
    ok = named_bar_and(id, 128, ok);
    paged::RingPos at = k;
    if (j_first > 0) at = at.next(sh.stages).next(sh.stages);
    uint32_t step = first_step + j_first;
    for (int j = j_first; j < n; j += kStep, step += kStep) {
      scale.step(g.j0 + j);
      const bool there = scale.there;
      const int kv0 = (g.j0 + j) * kRowsPerTile, e = scale.exponent();
      const float kx = scale_value(scale.kb);
      ok = ok && __all_sync(0xffffffffu,
                            mbar_wait(bar(L::kSFull + (step & 1u)), (step >> 1) & 1u, abort_flag, err));
      tc_fence_after();
      const bool partly = kv0 + kRowsPerTile - 1 > first_last;
      const bool holes = __any_sync(0xffffffffu, !there);
      // 16 columns from h on of this key's scores in units of log2, masked, less the
      // columns' references (`less`)
      auto load_scores = [&](int h, bool less, float *x) {
        uint32_t raw[16];
        tmem_ld16(tmem + lane_off + (step & 1u) * sh.N + col0 + h, raw);
        tmem_ld_wait(raw);
        // (in this order: the second product is exact, so a score that is its column's
        // reference comes out as 0 however large it is)
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
          const float4 b = *reinterpret_cast<const float4 *>(back + h + c);
          float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
          if (less) m = *reinterpret_cast<const float4 *>(mine.ref + h + c);
          x[c] = fmaf(__uint_as_float(raw[c]) * b.x, kx, -m.x);
          x[c + 1] = fmaf(__uint_as_float(raw[c + 1]) * b.y, kx, -m.y);
          x[c + 2] = fmaf(__uint_as_float(raw[c + 2]) * b.z, kx, -m.z);
          x[c + 3] = fmaf(__uint_as_float(raw[c + 3]) * b.w, kx, -m.w);
        }
        if (holes) {
#pragma unroll
          for (int c = 0; c < 16; ++c) x[c] = there ? x[c] : -INFINITY;
        }
        if (partly) paged::mask_columns(p, g.s, tree, kv0 + key, first_last, col0 + h, x);
      };
      float x[C];
      float top = -INFINITY;
      const bool begun = j > j_first;  // O holds a sum of tiles before
#pragma unroll
      for (int h = 0; h < C; h += 16) {
        load_scores(h, true, x + h);
#pragma unroll
        for (int c = 0; c < 16; c += 2) top = fmax3(top, x[h + c], x[h + c + 1]);
      }
      const bool seen = top > -INFINITY;  // by a row of these
      const bool fits = !(top + static_cast<float>(e - top_e) > kMost || top > kFar || (seen && e - top_e > 100));
      // the first tile of a segment has no reference yet (its scores were only looked at for masks)
      if (!begun || !named_bar_and(id, 128, ok && fits)) {
        // the largest exponent of the values that a row sees, then the maxima of s + e - E over the tile's 128 keys, then
        // O and l onto the new references
        const int warp_e = __reduce_max_sync(0xffffffffu, seen ? e : kNoExponent);
        if (lane == 0) mine.tops[w] = warp_e;
        named_bar_sync(id, 128);
        const int new_e = max(top_e, max(max(mine.tops[0], mine.tops[1]), max(mine.tops[2], mine.tops[3])));
        const float less_e = fmaxf(static_cast<float>(e - new_e), kMost - kFar);
#pragma unroll
        for (int h = 0; h < C; h += 16) {
          float y[16];
          load_scores(h, false, y);
#pragma unroll
          for (int c = 0; c < 16; ++c) y[c] += fabsf(y[c]) < kLarge ? less_e : 0.f;
          const float most = paged::reduce16(y, larger);
          if (!(lane & 1)) mine.red[w * C + h + (lane >> 1)] = most;
        }
        named_bar_sync(id, 128);
        if (key < C) {
          const float most = fmaxf(fmaxf(mine.red[key], mine.red[C + key]), fmaxf(mine.red[2 * C + key], mine.red[3 * C + key]));
          const float old_ref = mine.ref[key];
          const float fall = fabsf(old_ref) < kLarge ? static_cast<float>(max(top_e - new_e, -kFall)) : 0.f;
          const float new_ref = fmaxf(fmaxf(most, highest - kFall), old_ref + fall);
          highest = fmaxf(highest, new_ref);
          mine.ref[key] = new_ref;
          mine.factor[key] = ex2_approx(old_ref - new_ref);
        }
        const float down = two_to(top_e - new_e);  // what a larger exponent takes from O
        top_e = new_e;
        ok = named_bar_and(id, 128, ok);
        if (ok && begun) ok = product_done(step - kStep);
        tc_fence_after();
        const bool old = ok && begun;
#pragma unroll
        for (int h = 0; h < C; h += 16) {
          float alpha[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            alpha[c] = mine.factor[h + c];
            l[h + c] *= alpha[c];
          }
          if (old) {
#pragma unroll
            for (int part = 0; part < 3; ++part) {
              uint32_t v[16];
              const uint32_t o = o_addr + part * sh.N + h;
              tmem_ld16(o, v);
              tmem_ld_wait(v);
#pragma unroll
              for (int c = 0; c < 16; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * (alpha[c] * down));
              tmem_st16(o, v);
            }
          }
          load_scores(h, true, x + h);
        }
        if (old) tmem_st_wait();
      }
      const float fw = seen ? two_to(e - top_e + kWeightUnit) : 0.f;
      const uint32_t p_key = smem + sh.p_at() + (sh.N == 16 ? 0u : (step & 1u) * sh.p_step()) + key * 128;
      const int first = sh.N == 16 ? static_cast<int>(step & 1u) * 64 : 0;
#pragma unroll
      for (int h = 0; h < C; h += 16) {
        uint32_t part[3][4];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          float a[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            a[c] = ex2_approx(x[h + i + c]);
            l[h + i + c] += a[c];
            a[c] *= fw;
          }
          split_weights(a, part[0][i / 4], part[1][i / 4], part[2][i / 4]);
        }
        // the product of the tile before the last has read its P
        if (h == 0 && step >= 2) ok = ok && product_done(step - 2);
#pragma unroll
        for (int n = 0; n < 3; ++n) {
          const int byte = first + n * sh.N + col0 + h;  // of the key's row, or past it of the next block's
          if (ok)
            st_shared_v4(p_key + (byte >> 7) * L::kPBytes + (static_cast<uint32_t>((byte >> 4 & 7) ^ (key & 7)) << 4), part[n][0],
                         part[n][1], part[n][2], part[n][3]);
        }
      }
      if (ok) {
        const paged::RingPos v = at.next(sh.stages);
        if ((kTurns || gi == 0) && g.s.kv_len - kv0 < kRowsPerTile)
          ok = clear_tail8<D>(g.s.kv_len - kv0, smem + v.slot * Cfg8<D>::kTileBytes, bar(L::kFull + v.slot), v.phase, abort_flag,
                              err);
        fence_proxy_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kPFull + (step & 1u)));  // one arrival per warp
      }
      at = at.next(sh.stages).next(sh.stages);
      if (kTurns) at = at.next(sh.stages).next(sh.stages);
    }
    const bool any = n > j_first;  // this warpgroup had a tile
    const int behind = k.slot + 2 * n, laps = behind / sh.stages;
    k = {behind - laps * sh.stages, k.phase ^ (static_cast<uint32_t>(laps) & 1u)};
    first_step += n;
    // the next segment, if it is known, is asked for ahead of the epilogue
    if (__all_sync(0xffffffffu, mbar_test(items.there(), static_cast<uint32_t>(items.i >> 2) & 1u))) {
      const Segment &next = items.get();
      if (next.j1 > next.j0) {
        ask(next, first_step);
        asked = true;
      }
    }
    if (any) ok = ok && product_done(step - kStep);
    tc_fence_after();
    // l over the keys
#pragma unroll
    for (int h = 0; h < C; h += 16) {
      float y[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) y[c] = l[h + c];
      const float s = paged::reduce16(y, sum_of);
      if (!(lane & 1)) mine.red[w * C + h + (lane >> 1)] = s;
    }
    auto sum_at = [&](const Reductions<C> &x, int c) { return (x.red[c] + x.red[C + c]) + (x.red[2 * C + c] + x.red[3 * C + c]); };
    if (kTurns) {
      if (gi != 0 && key == 0) mine.tops[0] = top_e;
      tc_fence_before();  // the second's products, which only it has waited for, ahead of the first's loads
      if (!named_bar_and(3, 256, ok)) return;
      tc_fence_after();
      if (gi != 0) continue;
    } else {
      if (!named_bar_and(id, 128, ok)) return;
    }
    // each row's factors (of the other warpgroup's O too) and lse
    const Reductions<C> other(reds + 256);
    const size_t part = static_cast<size_t>(max(g.slot, 0)) * p.part_rows + col0;
    if (key < C) {
      float sum = sum_at(mine, key), ref = mine.ref[key];
      float f0 = 1.f, f1 = 0.f;
      if (kTurns) {
        const float sum1 = sum_at(other, key), ref1 = other.ref[key], most = fmaxf(ref, ref1);
        f0 = ex2_approx(ref - most);
        f1 = ex2_approx(ref1 - most);
        sum = sum * f0 + sum1 * f1;
        ref = most;
      }
      const float inv = sum != 0.f ? 1.f / sum : 0.f;
      mine.factor[key] = f0 * inv;
      if (kTurns) other.factor[key] = f1 * inv;
      if (col0 + key < rows) {
        const float lse = sum != 0.f ? (ref + log2f(sum)) * kLn2 : -INFINITY;
        const int tok = (col0 + key) / p.G, head = g.h * p.G + (col0 + key) - tok * p.G;
        if (g.slot >= 0) p.part_lse[part + key] = lse;
        else if (p.lse) p.lse[static_cast<size_t>(head) * p.total_q + g.s.q0 + tok] = lse;
      }
    }
    named_bar_sync(id, 128);
    // O back from 2^(kWeightUnit - E), in two steps as that may leave the range of one number
    auto halves = [](int e, float &a, float &b) {
      const int unit = max(e, -200) - kWeightUnit;
      a = two_to(unit / 2);
      b = two_to(unit - unit / 2);
    };
    float up0, up1, other0 = 0.f, other1 = 0.f;
    halves(top_e, up0, up1);
    const bool both = kTurns && n > 1;  // (O of a warpgroup without a tile is not written)
    if (both || (kTurns && !any)) halves(other.tops[0], other0, other1);
    // a thread has column `key` of O, one row after the other
    const int n_rows = min(C, rows - col0);
    int tok = col0 / p.G, head = col0 - tok * p.G;
    float *to_part = p.part_o + part * D + key;
    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(p.o) + (g.h * p.G + head) * p.o_h + (g.s.q0 + tok) * p.o_s + key;
#pragma unroll 1
    for (int h = 0; h < n_rows; h += 8) {
      float o[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = 0.f;
      auto add = [&](uint32_t at, const float *factor, float a, float b) {
        uint32_t v[8], u[8], t[8];
        tmem_ld8(at + h, v);
        tmem_ld8(at + sh.N + h, u);
        tmem_ld8(at + 2 * sh.N + h, t);
        tmem_ld_wait(v);
        tmem_ld_wait(u);
        tmem_ld_wait(t);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          o[c] += fmaf(__uint_as_float(t[c]), kLastPart, __uint_as_float(v[c]) + __uint_as_float(u[c])) * factor[h + c] * a * b;
      };
      if (!kTurns || any) add(o_addr, mine.factor, up0, up1);
      if (kTurns && (both || !any)) add(o_addr + L::kOStep, other.factor, other0, other1);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (h + c < n_rows && key < D) {
          if (g.slot >= 0) to_part[(h + c) * D] = o[c];
          else *to = __float2bfloat16_rn(o[c]);
        }
        to += p.o_h;
        if (++head == p.G) {
          head = 0;
          to += p.o_s - p.G * p.o_h;
        }
      }
      __syncwarp();
    }
    if (kTurns) tc_fence_before();
  }
}

// ---------------------------------------------------------------- the wide form
// K and V tiles as fp16 in the ring that the bf16 form has, its issuers and its
// softmax (kCodes). Four warps turn the codes, each of K or V one half of every tile,
// through registers: as it turns one tile it asks for the next, so that neither the
// codes' way from memory nor a copy in shared memory is between a free slot of the ring
// and its tile.
// (What it took, in clocks of a pair of query tiles: one warp for all of K, one
// for V, 8,000 by bulk copies through shared memory, 500 to start one, 5,700 by
// asynchronous ones; code longer than the instruction caches hold, all of a tile
// unrolled in two roles, 24,000.)
template <int D>
struct Turner {
  static constexpr int kRows = 512 / D;  // rows of a warp's access: 512 bytes
  const PagedAttnParams &p;
  const unsigned char *pool, *scales;  // of K or V; from `head` on of the segment's KV head
  const unsigned char *head, *head_scales;
  uint32_t place, factors;             // shared memory: the half's codes, its keys' factors
  int lane, half;     // half: first row of this warp's half

  bool word;          // scales can be read four at a time
  uint32_t bytes;     // scale bytes of keys 4 lane .. 4 lane + 3 of the next tile, 0: not there
  int e, largest;     // the exponent of the tile's unit; V: the largest of the segment
  __device__ __forceinline__ Turner(const PagedAttnParams &p_, bool values, int half_, uint32_t place_, uint32_t factors_)
      : p(p_), pool(static_cast<const unsigned char *>(values ? p.cache.v_pages : p.cache.k_pages)),
        scales(values ? p.scales.v : p.scales.k), lane(threadIdx.x & 31), half(half_), place(place_), factors(factors_) {
    word = ((reinterpret_cast<uintptr_t>(scales) | static_cast<uintptr_t>(p.scales.page_stride)) & 3) == 0;
  }
  __device__ __forceinline__ void set_head(int h) {
    head = pool + (static_cast<long long>(h) << p.page_log2) * D;
    head_scales = scales + (static_cast<long long>(h) << p.page_log2);
  }
  // `page`: lane i's page of tile j the i-th, n_pages for none (PageWindow::page). Its
  // page of row r, and the slot there.
  __device__ __forceinline__ int page_at(int page, int r) const {
    return __shfl_sync(0xffffffffu, page, p.page_log2 < 7 ? r >> p.page_log2 : 0);
  }
  __device__ __forceinline__ int slot_at(int j, int r) const { return (j * kRowsPerTile + r) & ((1 << p.page_log2) - 1); }
  __device__ __forceinline__ void load_scales(int page, int j, int valid) {
    const int pg = page_at(page, 4 * lane);
    bytes = 0;
    if (pg < p.cache.n_pages && 4 * lane < valid) {
      const unsigned char *from = head_scales + pg * p.scales.page_stride + slot_at(j, 4 * lane);
      if (word) {
        bytes = *reinterpret_cast<const uint32_t *>(from);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) bytes |= static_cast<uint32_t>(from[i]) << (8 * i);
      }
    }
  }
  // The factors 2^(e_key - e) of the tile whose scales were loaded: for K e is 7 below the largest exponent, for V
  // value_unit makes it of that.
  __device__ __forceinline__ void take_scales(int valid, bool values, bool first) {
    int b[4], most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[i] = static_cast<int>(bytes >> (8 * i) & 255u);
      if (4 * lane + i < valid) most = max(most, b[i]);  // (those past the end may be anything)
    }
    most = __reduce_max_sync(0xffffffffu, most);
    const int top = max(most, 1) - 127;
    if (!values) {
      e = max(top - paged::codes::kAbove, -126);  // (what masks leave is -inf times it: no zero)
    } else if (first || most > 0) {  // (a tile without a key leaves the unit)
      e = paged::codes::value_unit(top, e, largest, first);
      largest = first ? e : max(largest, e);
    }
    uint32_t f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = fminf(two_to(max(b[i], 1) - 127 - e), static_cast<float>(1 << paged::codes::kAbove));
      f[i] = f16x2_of_floats(x, x);
    }
    if (4 * lane >= half && 4 * lane < half + 64) st_shared_v4(factors + 4 * (4 * lane - half), f[0], f[1], f[2], f[3]);
    __syncwarp();
  }
  // Codes of the half of tile j; keys that are not there (past the end, where codes may
  // be NaN, or on no page) as zeros.
  __device__ __forceinline__ void fetch(int page, int j, int valid) const {
    const int per = min(64, 1 << p.page_log2);  // rows that lie in one page
#pragma unroll 1
    for (int c = 0; c < 64; c += per) {
      const int r = half + c, pg = page_at(page, r);
      const bool there = pg < p.cache.n_pages;
      const unsigned char *from = head + ((there ? pg : 0) * p.cache.page_stride + static_cast<long long>(slot_at(j, r)) * D + 16 * lane);
      const int rows = there ? valid - r - lane / (D / 16) : 0;
      const uint32_t to = place + c * D + 16 * lane;
      if (per == 64) {
#pragma unroll
        for (int i = 0; i < 64 / kRows; ++i) copy_async16(to + 512 * i, from + 512 * i, rows > kRows * i);
      } else {
#pragma unroll
        for (int i = 0; i < 16 / kRows; ++i) copy_async16(to + 512 * i, from + 512 * i, rows > kRows * i);
        if (per == 32) {
#pragma unroll
          for (int i = 16 / kRows; i < 32 / kRows; ++i) copy_async16(to + 512 * i, from + 512 * i, rows > kRows * i);
        }
      }
    }
    copy_async_commit();
  }
  // What was fetched to fp16 at `tile`.
  __device__ __forceinline__ void turn(uint32_t tile) const {
    constexpr int kPieces = D / 16, kIter = 32 / kRows;  // pieces of a row; accesses of 32 rows
    const int c = lane % kPieces, r0 = lane / kPieces;
    // a thread's two pieces of a row in turn, those of the second column block in the
    // other order, so that no two lanes of a row are on one bank
    const bool swap = c / 4;
    const uint32_t first = (((c % 4) * 2 + (swap ? 1 : 0)) ^ (r0 & 7)) << 4;
    uint32_t from = place + 16 * lane, to = tile + (c / 4) * kColBlockBytes + (half + r0) * 128, factor = factors + 4 * r0;
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
      uint4 x[kIter];
      uint32_t f[kIter];
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        x[i] = ld_shared_v4(from + 512 * i);
        f[i] = ld_shared(factor + 4 * kRows * i);
      }
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const uint32_t lo0 = swap ? x[i].z : x[i].x, lo1 = swap ? x[i].w : x[i].y;  // the piece that goes first
        const uint32_t hi0 = swap ? x[i].x : x[i].z, hi1 = swap ? x[i].y : x[i].w;
        const uint32_t at = to + kRows * 128 * i, piece = first ^ (kRows * i % 8 << 4);
        auto wide = [&](uint32_t codes) { return mul_f16x2(f16x2_of_e4m3x2(codes), f[i]); };
        st_shared_v4(at + piece, wide(lo0), wide(lo0 >> 16), wide(lo1), wide(lo1 >> 16));
        st_shared_v4(at + (piece ^ 16u), wide(hi0), wide(hi0 >> 16), wide(hi1), wide(hi1 >> 16));
      }
      from += 32 * D;
      to += 32 * 128;
      factor += 128;
    }
  }
};

// Walks the line for the others: the whole warp.
__device__ __forceinline__ void wide_walker(const PagedAttnParams &p, Walk walk, Segment g, Items items,
                                            volatile int *abort_flag, int *err) {
  int4 cut = make_int4(0, 0, 0, 0);  // the item that this CTA begins and another one ends, for the merge
  int c = 0;
  while (walk.next(p, g)) {
    g.ring = c;
    if (!items.put(g, abort_flag, err)) break;
    if (g.j0 == 0 && g.slot >= 0)
      cut = make_int4(g.s.q0 + g.rb * 2 * p.tok, min(2 * p.tok, g.s.q_len - g.rb * 2 * p.tok) * p.G, g.h, walk.ends_in(p, g));
    c += 2 * max(Walk::tiles(p, g, 0), Walk::tiles(p, g, 1));
  }
  g.j0 = g.j1 = 0;
  items.put(g, abort_flag, err);
  if ((threadIdx.x & 31) == 0) p.cuts[blockIdx.x] = cut;
  __syncwarp();
}

// One half of the K or, with `values`, V tiles of the CTA's segments. `place`: shared
// memory for the codes, `factors` 256 bytes more. Called in one place, so that the four
// warps share its instructions.
template <int D>
__device__ __forceinline__ void wide_turner(bool values, int half, const PagedAttnParams &p, Items items, uint32_t bar0,
                                            uint32_t ring, uint32_t place, uint32_t factors, volatile int *exps,
                                            volatile int *abort_flag, int *err) {
  using C = paged::Cfg<D>;
  using W = paged::WideBars<D>;
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  Turner<D> t(p, values, half, place, factors);
  bool ok = true;
  while (ok && items.wait(abort_flag, err)) {
    const Segment g = items.get();
    items.release();
    const int j0 = uniform(g.j0), n = uniform(max(Walk::tiles(p, g, 0), Walk::tiles(p, g, 1)));
    if (n == 0) continue;
    t.set_head(uniform(g.h));
    const int kv_len = uniform(g.s.kv_len);
    int c = uniform(g.ring);  // of the tile's K
    PageWindow pages(p, g, false, 0);
    pages.prefetch(p);
    int page = pages.page(p, j0), valid = kv_len - j0 * kRowsPerTile;
    t.load_scales(page, j0, valid);
    t.fetch(page, j0, valid);
    // the factors of a tile, its exponent where the softmax finds it
    auto take = [&](int at, bool first) {
      t.take_scales(valid, values, first);
      if (lane == 0) exps[at % paged::codes::kExponents] = t.e;  // (both halves' warps the same)
    };
    take(values ? c + 1 : c, true);
#pragma unroll 1
    for (int j = 0; j < n; ++j, c += 2) {
      const int at = c + (values ? 1 : 0), slot = at % C::kStages;
      const bool more = j + 1 < n;
      if (more) {
        page = pages.page(p, j0 + j + 1);
        valid -= kRowsPerTile;
        t.load_scales(page, j0 + j + 1, valid);
      }
      copy_async_wait<0>();
      __syncwarp();  // every lane's copies
      ok = at < C::kStages || __all_sync(0xffffffffu, mbar_wait(bar(W::kEmpty + slot), ((at / C::kStages) - 1) & 1, abort_flag, err));
      if (!ok) break;
      t.turn(ring + slot * C::kTileBytes);
      fence_proxy_async_shared();
      __syncwarp();  // (the codes and factors have been read, too)
      // the next tile's exponent before this tile: the softmax needs that of V, whose slot
      // is free only behind the product before, ahead of the scores' way through it
      if (more) take(at + 2, false);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(W::kFull + slot));
      if (more) t.fetch(page, j0 + j + 1, valid);
    }
  }
  copy_async_wait<0>();
  __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(kThreads8, 1)
    attn_paged_e4m3_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ PagedAttnParams p) {
  using C = Cfg8<D>;
  using L = Narrow8<D>;
  using W = paged::WideBars<D>;
  using Wide = typename C::Wide;
  static_assert(Wide::kNumBarriers <= C::kItemBarrier, "barriers");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem =
      reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kAreaBytes);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::kMaxBarriers);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *turn = reinterpret_cast<volatile int *>(tmem_slot + 2);  // next MMA burst slot (wide)
  Segment *places = reinterpret_cast<Segment *>(tmem_slot + 4);
  float *red = reinterpret_cast<float *>(smem + C::kRedAt);
  int *small = reinterpret_cast<int *>(places + 4), *warp_sums = small;
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
  // an earlier timeout, not yet cleared by the host: this CTA skips its work and its rows come out as O = 0, lse = -inf
  const bool failed = warp == kMmaWarp1 && *reinterpret_cast<volatile int *>(err) != kErrNone;
  const Line line = paged::prefix_costs<kThreads8>(p, narrow_unit8, prefix, warp_sums);
  const bool narrow = line.narrow;
  const L sh(line.rows);
  const Walk walk(line);
  const Items items(places, bar(C::kItemBarrier));
  Segment first = {};    // the producer's
  int first_entry = -1;  // the producer's lanes: the first pages
  if (warp == kTmaWarp && walk.pos < walk.end) {
    const paged::Place at = paged::place_of(p, prefix, walk.pos, first.s);
    first.b = at.b;
    first.h = at.h;
    first.rbs = paged::row_blocks(p, first.s);
    walk.make(p, at.rb, at.r, first);
    first_entry = paged::window_entry(p, paged::page_row(p, first), first.s.kv_len, paged::first_page(p, first.j0));
  }
  if (warp == kMmaWarp1) {
    for (int i = lane; i < (narrow ? L::kNumBarriers : Wide::kNumBarriers); i += 32) {
      int arrivals = 1;
      if (narrow) {
        if (i == L::kQFull || i == L::kPFull || i == L::kPFull + 1) arrivals = sh.turns ? 4 : 8;
      } else {
        if (i == W::kMmaDone || (i >= W::kFull && i < W::kEmpty + W::kStages)) arrivals = 2;
        if (i == W::kQFull || i == W::kQEmpty || i == W::kPFull || i == W::kPFull + 1) arrivals = 4;
      }
      mbar_init(bar(i), arrivals);
    }
    // read by the issuer(s), the softmax warps and the turners
    if (lane < 8) mbar_init(bar(C::kItemBarrier + lane), lane < 4 ? 1 : (narrow ? 10 : 14));
    if (lane == 0) {
      *abort_flag = failed;
      *turn = 0;
    }
    fence_barrier_init();
  }
  fence_proxy_async_shared();  // the prefix sums before the copies that follow
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  launch_dependents();  // the merge: its CTAs wait for this kernel before they read
  const uint32_t tmem = *tmem_slot;
  const bool skip = *abort_flag != 0;
  if (skip && threadIdx.x == 0) p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
  const uint32_t sQ = base, sRing = base + 2 * Wide::kTileBytes;
  volatile int *exps = small;
  // (two branches to the kernel's end: behind a join no one would have the larger share)
  if (warp < 8) {
    set_max_registers<kSoftmaxRegs, true>();
    paged::write_unseen<D>(p, skip, threadIdx.x, 256);
    if (skip) {
      // nothing
    } else if (!narrow) {
      paged::wide_softmax<D, true>(p, items, warp >> 2, bar0, sQ, sRing, tmem,
                                   sQ + (warp >> 2) * Wide::kTileBytes + (warp & 3) * paged::kStageBytes, exps, abort_flag, err);
    } else {
      if (sh.turns) narrow_softmax8<D, 16, true>(p, sh, items, warp >> 2, bar0, base, tmem, red, abort_flag, err);
      else if (sh.N == 32) narrow_softmax8<D, 16, false>(p, sh, items, warp >> 2, bar0, base, tmem, red, abort_flag, err);
      else narrow_softmax8<D, 32, false>(p, sh, items, warp >> 2, bar0, base, tmem, red, abort_flag, err);
    }
  } else if (warp < kTurners) {
    set_max_registers<kIssuerRegs, false>();
    if (skip) {
      // nothing
    } else if (narrow) {
      if (warp == kTmaWarp)
        narrow_producer8<D>(p, walk, first, items, &tm_k, &tm_v, bar(L::kFull), bar(L::kEmpty), base, sh.stages, first_entry,
                            abort_flag, err);
      else if (warp == kMmaWarp)
        narrow_scores8<D>(sh, items, bar0, base, tmem, abort_flag, err);
      else if (warp == kMmaWarp1)
        narrow_products8<D>(sh, items, bar0, base, tmem, abort_flag, err);
    } else if (warp == kTmaWarp) {
      wide_walker(p, walk, first, items, abort_flag, err);
    } else if (warp == kMmaWarp || warp == kMmaWarp1) {
      paged::wide_issuer<D, true>(p, items, warp == kMmaWarp ? 0 : 1, bar0, sQ, sRing, tmem, turn, abort_flag, err);
    }
  } else {
    set_max_registers<kTurnerRegs, false>();
    if (!skip && !narrow) {
      const int i = warp - kTurners;
      wide_turner<D>(i >= 2, i % 2 * 64, p, items, bar0, sRing, base + C::kCodesAt + i * C::kCodesBytes,
                     smem_addr(small + 32) + 256 * i, exps, abort_flag, err);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_typed8(const CUtensorMap &tk, const CUtensorMap &tv, const PagedAttnParams &p, cudaStream_t stream) {
  return paged::launch_with_merge<D>(attn_paged_e4m3_kernel<D>, Cfg8<D>::kSmemBytes, kThreads8, p, stream, tk, tv, p);
}

}  // namespace paged8

cudaError_t launch_attn_paged_e4m3(int D, const CUtensorMap &tk, const CUtensorMap &tv, const PagedAttnParams &p,
                                   cudaStream_t stream) {
  return D == 64 ? paged8::launch_typed8<64>(tk, tv, p, stream) : paged8::launch_typed8<128>(tk, tv, p, stream);
}

}  // namespace seqattn
