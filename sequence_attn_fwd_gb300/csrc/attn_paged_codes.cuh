// Pieces of the paged attention over e4m3 codes that its wide form's softmax needs
// (included by attn_paged.cuh; see attn_paged_e4m3.cuh).
#pragma once

namespace seqattn {
namespace paged {
namespace codes {

// A row of q in few bits: the power of two that brings its largest
// size `top` to [128, 256) (less for rows below 2^-119), and what takes scores of it
// back to units of log2: c2 over that power. Rows with an infinity come out as NaN.
struct RowScale {
  float up, back;
};
__device__ __forceinline__ RowScale row_scale(float top, float c2) {
  const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -119), 127);
  const float up = __int_as_float((127 + 7 - e) << 23);
  const float down = __int_as_float(max(127 - 7 + e, 1) << 23);
  return {top > 0.f ? up : 1.f, top == INFINITY ? NAN : (top > 0.f ? c2 * down : c2)};
}
__device__ __forceinline__ float largest_of(const uint4 &x) {
  float top = 0.f;
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xffff0000u))));
  return top;
}

// 2^e for any e: 0 below the range of normal numbers.
__device__ __forceinline__ float two_to(int e) { return ex2_approx(static_cast<float>(e)); }

// What a tile's exponents make of it. K and V come in fp16, in units of powers of two:
// `key` that of K, the tile's own; that of V, O's unit too, changes where the tiles'
// largest scales leave its range (value_unit): `down` brings O along.
struct TileUnits {
  float key, down;
};
constexpr int kExponents = 32;   // places for the exponents of ring positions
__device__ __forceinline__ TileUnits tile_units(const volatile int *exps, int cv, bool first, int &e_ref) {
  const int ek = exps[(cv - 1) % kExponents], ev = exps[cv % kExponents];
  const float down = first ? 1.f : two_to(e_ref - ev);
  e_ref = ev;
  return {two_to(ek), down};
}
// The unit's exponent for a tile of V whose largest scale is 2^e, behind one of `unit`, the largest so far
// `most`: the same for a few sizes. Codes end at 2^9 and fp16 at 2^16, so scales may be up to 2^7
// in it, and are 2^2 or more, for what fp16 has below: factors end at 2^-24. (K's unit is
// 2^-7 of the tile's largest scale.) A unit 2^40 below the largest one at the least, as O
// holds that, too.
constexpr int kAbove = 7, kBelow = 2, kChosen = 5, kUnitFall = 40;
__device__ __forceinline__ int value_unit(int e, int unit, int most, bool first) {
  if (!first && e <= unit + kAbove && e >= unit + kBelow) return unit;
  return first ? e - kChosen : max(e - kChosen, most - kUnitFall);
}
// A row's weights are against a reference 2^kHeadroom below its largest score. Sums of a
// tile's weights up to kMostSum, 2^15 of fp16, are let by. Sums below kLeastSum bring the
// reference down, so that what the keys behind an attention sink bring, a little each, keeps
// its bits: fp16 ends in steps of 2^-24, so a weight is held to 2^-11 of itself or to 2^-18 of its
// tile's sum. References fall as far as l stays below 2^kMostL, and while it is below kFallL. A
// segment's first tile has kFirstHeadroom: the keys beside a sink at the start of a context
// have no other tile to be held in. (1,024 tokens behind 65,536 keys of sizes 2^-1.5 to 2^1.5, and a batch of prompt pieces with heads
// of 64: with both 7, 7, 6, 5, 3: 968, 898, 880, 869, 855 us and 236, 203, 192, 184, 183, the first with
// kLeastSum 2; 5 and 13: 868 and 201.)
constexpr float kHeadroom = 5.f, kFirstHeadroom = 13.f, kMostSum = 32768.f, kLeastSum = 0.0078125f, kMostL = 57.f,
                kFallL = 0x1p50f, kMostHeadroom = 15.f;
// O from units of 2^e: 1 / l times two factors, as 2^e may leave the range of one.
__device__ __forceinline__ void units_back(int e, float &inv_l, float &back) {
  const int half = e / 2;
  inv_l *= two_to(half);
  back = two_to(e - half);
}

// The weights of a row's 128 scores, packed as fp16 pairs; returns the fp32 sum of the
// weights. x = s unit key - ref, fused, or, kApart, with the second
// product exact and the first rounded as in the reference: then a score that is the
// reference comes out as 0 however large it is. (Scores past 2^24 have no more
// than whole powers of two between them; fused, the sum passes its bound there and the
// warp comes back for the other form. As a choice in front of both forms, in both
// places: 21 us of 306 for 1,024 tokens behind 16,384 keys.)
template <bool kApart>
__device__ __forceinline__ float weights_row(const float *s, float unit, float key, float ref, uint32_t *pk) {
  const uint64_t unit2 = kApart ? f2_pack(unit, unit) : f2_pack(unit * key, unit * key), key2 = f2_pack(key, key);
  const uint64_t neg_m2 = f2_pack(-ref, -ref);
  uint64_t sum_a = f2_pack(0.f, 0.f), sum_b = sum_a;
  auto exponent = [&](int i) {
    const uint64_t x = f2_pack(s[i], s[i + 1]);
    return kApart ? f2_fma(f2_mul(x, unit2), key2, neg_m2) : f2_fma(x, unit2, neg_m2);
  };
#pragma unroll
  for (int q = 0; q < 64; q += 2) {  // pairs q and q + 1: elements 2q .. 2q + 3
    const uint64_t pa = exp2_pair(exponent(2 * q), false), pb = exp2_pair(exponent(2 * q + 2), false);
    sum_a = f2_add(sum_a, pa);
    sum_b = f2_add(sum_b, pb);
    float p0, p1, p2, p3;
    f2_unpack(pa, p0, p1);
    f2_unpack(pb, p2, p3);
    // fp16: 2^-11 of a weight, or 2^-18 of their sum (kLeastSum)
    pk[q] = f16x2_of_floats(p0, p1);
    pk[q + 1] = f16x2_of_floats(p2, p3);
  }
  float a0, a1, b0, b1;
  f2_unpack(sum_a, a0, a1);
  f2_unpack(sum_b, b0, b1);
  return (a0 + a1) + (b0 + b1);
}
template <bool kApart>
__device__ __forceinline__ float weights(const float *s, float unit, const TileUnits &u, float ref, uint32_t (&pk)[64]) {
  return weights_row<kApart>(s, unit, u.key, ref, pk);
}

// This thread's row of a query tile (first: the tile's first token) to shared
// memory in fp16, [column block of 64][128 rows][128 bytes], swizzled, after its power
// of two; returns the unit of its scores.
template <int D>
__device__ __forceinline__ float put_query(const PagedAttnParams &p, const Segment &g, int first, bool row_valid,
                                           uint32_t tile) {
  const int r = threadIdx.x & 127, tok = r / p.G;
  uint4 x[D / 8] = {};
  if (row_valid) {
    const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) +
                                                     (g.h * p.G + r - tok * p.G) * p.q_h + (g.s.q0 + first + tok) * p.q_s);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) x[i] = q[i];
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) top = fmaxf(top, largest_of(x[i]));
  const RowScale rs = row_scale(top, p.scale_log2);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)  // exact, down to 2^-24 of the row's largest
      h[k] = f16x2_of_floats(__uint_as_float(u[k] << 16) * rs.up, __uint_as_float(u[k] & 0xffff0000u) * rs.up);
    st_shared_v4(tile + (i / 8) * kColBlockBytes + r * 128 + (((i % 8) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
  }
  fence_proxy_async_shared();
  return rs.back;
}

}  // namespace codes
}  // namespace paged
}  // namespace seqattn
