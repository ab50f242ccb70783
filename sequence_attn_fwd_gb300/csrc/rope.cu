// Rotary positions with several axes, alone and on the way into a paged cache.
//
// Pair i of a row is turned by positions[axis_i] * inv_freq_i. The angle is
// formed in turns, in 64-bit fixed point: f_i = inv_freq_i / 2 pi as a binary
// fraction of 64 bits (made on the host in double), position * f_i modulo 2^64
// by one integer product, so whole turns drop out exactly and a position of
// 10^6 costs no precision; the signed fraction, as a float, goes through
// sincospif.
//
// Memory-bound: every element is read and written once. A thread takes one
// slice of 16 elements -- eight pairs, two 16-byte pieces in bf16, four in fp32
// -- of one token, forms its eight sines and cosines once, in registers, and
// goes over heads with them, four rows in flight; D / 16 threads cover a row
// with whole 32-byte sectors in either pairing. (Sines in shared memory, shared
// by the CTA, cost more in reads than they save: 109 us instead of 89 for
// 32,768 tokens of 32 heads of 128 in bf16, 6.0 TB/s of the 6.8 that a copy
// reaches.) The heads of a token are dealt over the CTA and, with few tokens, over
// the grid.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kernels.h"
#include "ptx.cuh"

namespace seqattn {
namespace {

constexpr int kRopeThreads = 256;

// 16 elements of a row as fp32: the first members of eight pairs, then the second.
template <typename T>
struct Vec16;
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int kPieces = 2;  // 16-byte pieces
};
template <>
struct Vec16<float> {
  static constexpr int kPieces = 4;
};

__device__ __forceinline__ void unpack(const uint4 (&w)[2], float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[8 * i + 2 * k] = __uint_as_float(u[k] << 16);
      x[8 * i + 2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void pack(const float (&x)[16], uint4 (&w)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // one rounding, to nearest: the result leaves in the tensor's own type
      __nv_bfloat162 h = __floats2bfloat162_rn(x[8 * i + 2 * k], x[8 * i + 2 * k + 1]);
      u[k] = *reinterpret_cast<uint32_t *>(&h);
    }
    w[i] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}
__device__ __forceinline__ void unpack(const uint4 (&w)[4], float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[4 * i] = __uint_as_float(w[i].x);
    x[4 * i + 1] = __uint_as_float(w[i].y);
    x[4 * i + 2] = __uint_as_float(w[i].z);
    x[4 * i + 3] = __uint_as_float(w[i].w);
  }
}
__device__ __forceinline__ void pack(const float (&x)[16], uint4 (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                      __float_as_uint(x[4 * i + 3]));
}

// Puts the turned elements into w and leaves those of the pairs `still` (one bit
// each) as they are, a 32-bit word at a time.
template <typename T, bool kInterleaved>
__device__ __forceinline__ void keep_copied(unsigned still, const uint4 (&turned)[Vec16<T>::kPieces],
                                            uint4 (&w)[Vec16<T>::kPieces]) {
  constexpr int kPer = 4 / static_cast<int>(sizeof(T)), kWords = 16 / kPer;  // elements of a word, words
  uint32_t *to = reinterpret_cast<uint32_t *>(w);
  const uint32_t *from = reinterpret_cast<const uint32_t *>(turned);
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    // pairs of the word's first and last element
    const int a = kPer * i, b = a + kPer - 1, pa = kInterleaved ? a / 2 : a % 8, pb = kInterleaved ? b / 2 : b % 8;
    const uint32_t keep = (still >> pa & 1u ? (pa == pb ? 0xffffffffu : 0xffffu) : 0u) |
                          (pa != pb && (still >> pb & 1u) ? 0xffff0000u : 0u);
    to[i] = (to[i] & keep) | (from[i] & ~keep);
  }
}

// Element offset of piece i (16 bytes) of the 16 elements that slice `sl` of a
// row has: consecutive ones when pairs are neighbours, else eight at 8 sl and
// their partners D / 2 further on.
template <typename T, int D, bool kInterleaved>
__device__ __forceinline__ int piece_at(int sl, int i) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(T));  // elements per piece
  if (kInterleaved) return 16 * sl + kPer * i;
  constexpr int kHalf = Vec16<T>::kPieces / 2;
  return 8 * sl + (i / kHalf) * (D / 2) + kPer * (i % kHalf);
}

// The slot of token t of an append: its page and its place there (page -1: it has
// none); *live: whether the token belongs to a sequence. `one`: of the threads with
// this token, the one that writes for a guarded row.
struct Slot {
  int page, at;
};
__device__ __forceinline__ Slot slot_of(const PagedView &c, int *guard, long long t, long long n_tok, bool one, bool *live) {
  int lo = 0, hi = c.B;  // the first sequence that ends behind t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (c.cu_seqlens[mid + 1] <= t) lo = mid + 1;
    else hi = mid;
  }
  *live = lo < c.B && c.cu_seqlens[lo] <= t;
  if (!*live) return {-1, 0};
  const long long max_keys = static_cast<long long>(c.max_pages) * c.page_size;
  long long len = c.kv_lens[lo];
  len = len < 0 ? 0 : (len > max_keys ? max_keys : len);
  const long long end = c.cu_seqlens[lo + 1] < n_tok ? c.cu_seqlens[lo + 1] : n_tok;
  const long long slot = len - (end - t);
  if (guard != nullptr) {
    const RowGuard row(guard, c.B);
    const int q0 = max(c.cu_seqlens[lo], 0);
    const bool refused = row.refuses(lo, static_cast<int>(len), static_cast<int>(end) - q0);
    if (one && t == q0) {
      row.open[lo] = 0;
      row.lens[lo] = refused ? 0 : static_cast<int>(len);
    }
    if (refused) return {-1, 0};
  }
  if (slot < 0) return {-1, 0};
  const int page = c.page_table[lo * c.table_stride + slot / c.page_size];
  if (page < 0 || page >= c.n_pages) return {-1, 0};
  return {page, static_cast<int>(slot % c.page_size)};
}

// The exponent of the scale of a row of which kSlices neighbouring threads have 16
// elements each: the least e with max |y| <= 448 2^e (1.75 2^8 is the largest e4m3
// number), so the lowest one that loses nothing at the top; -126 at the least.
// A power of two costs no precision (e4m3 is a floating format) and makes every
// product with it exact. NaN elements do not count, and stay NaN. An infinity gives
// 2^120, and its code, 448, is past what fp32 and bf16 hold: it is read as one again.
template <int kSlices>
__device__ __forceinline__ int scale_of(const float (&y)[16]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(y[i]));
  // the threads of a row go the same way; others of the warp need not
  const unsigned lane = threadIdx.x & 31, mask = ((1u << kSlices) - 1u) << (lane & ~(kSlices - 1u));
#pragma unroll
  for (int off = kSlices / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, off));
  // m 2^E with 1 <= m < 2: E - 8, and one more if m > 1.75 (the sum carries)
  const int e = static_cast<int>((__float_as_uint(top) + 0x1fffffu) >> 23) - 127 - 8;
  return min(max(e, -126), 127);
}

// Sine and cosine of `turn` (a signed fraction of a turn, 64 bits) as sums of two
// floats, off by less than 2^-26 of the larger: Taylor's series on the nearest quarter's
// remainder r, |r| <= pi / 4, all but the leading terms in single floats. (Codes have
// few bits and no rounding behind them: a rotated key that one float's error takes
// past the middle of two codes is off by a whole one. The same appends with sincospif: 34 us,
// and more such keys than with sines rounded once.)
struct SineCosine {
  float s, s_lo, c, c_lo;
};
__device__ __forceinline__ SineCosine sine_cosine(long long turn) {
  const long long quarter = (turn >> 62) + (turn >> 61 & 1);  // to the nearest
  const long long rest = static_cast<long long>(static_cast<uint64_t>(turn) - (static_cast<uint64_t>(quarter) << 62));
  // r = rest 2 pi / 2^64; 2 pi as two floats
  const float a = static_cast<float>(rest), a_lo = static_cast<float>(rest - static_cast<long long>(a));
  constexpr float kHi = 6.283185307179586f, kLo = static_cast<float>(6.283185307179586476925 - static_cast<double>(kHi));
  constexpr float kUnit = 0x1p-64f;
  const float r = a * kUnit * kHi;
  const float r_lo = fmaf(a * kUnit, kHi, -r) + fmaf(a * kUnit, kLo, a_lo * kUnit * kHi);
  const float z = r * r, z_lo = fmaf(r, r, -z) + 2.f * r * r_lo;
  // sin r = r + r z (-1/3! + z/5! - ...)
  float p = fmaf(z, -1.f / 39916800.f, 1.f / 362880.f);
  p = fmaf(z, p, -1.f / 5040.f);
  p = fmaf(z, p, 1.f / 120.f);
  p = fmaf(z, p, -1.f / 6.f);
  const float t = r * z * p;
  const float s = r + t, s_lo = (r - s) + t + fmaf(r_lo * z, -0.5f, r_lo);
  // cos r = 1 - z/2 + z^2 (1/4! - z/6! + ...)
  float q = fmaf(z, 1.f / 479001600.f, -1.f / 3628800.f);
  q = fmaf(z, q, 1.f / 40320.f);
  q = fmaf(z, q, -1.f / 720.f);
  q = fmaf(z, q, 1.f / 24.f);
  const float w = fmaf(z, -0.5f, 1.f);
  const float u = fmaf(z * z, q, fmaf(z, -0.5f, 1.f - w) - 0.5f * z_lo);
  const float c = w + u, c_lo = (w - c) + u;
  SineCosine out = quarter & 1 ? SineCosine{c, c_lo, -s, -s_lo} : SineCosine{s, s_lo, c, c_lo};
  if (quarter & 2) out = {-out.s, -out.s_lo, -out.c, -out.c_lo};
  return out;
}
// x c - y s, c and s sums of two floats: two roundings of the result.
__device__ __forceinline__ float turned_pair(float x, float c, float c_lo, float y, float s, float s_lo) {
  const float p = y * s;
  return fmaf(x, c, -p) - (fmaf(y, s, -p) + fmaf(y, s_lo, -x * c_lo));
}

// blockIdx.x: tile of kTok tokens; blockIdx.y: share of the heads (those of q,
// then k, then, in an append, v). kStill: some pairs are copied, whatever they hold
// (turned by an angle of 0, an infinity would make its partner NaN). A variant of
// its own: tested in the one loop, it cost the others 17 %. Held to 64 registers,
// and to two rows in flight in fp32, it takes their time (32,768 tokens of 28 heads
// of 128, halves and neighbours as pairs: bf16 81 and 83 us, fp32 153 and 165; with
// 72 to 77 registers 94 and 96, 163 and 179; with four fp32 rows in flight 162 and 179).
// kAppend 0: rows turned; 1: appended to a bf16 cache; 2: to an e4m3 one, which is held
// to 64 registers too (prompt pieces of 10,500 tokens, 28 and 4 heads of 128: 37.4 us;
// with 98 registers 47; 64 single tokens 7.1).
template <typename T, int D, bool kInterleaved, int kAppend, int kTok, bool kStill>
__global__ void __launch_bounds__(kRopeThreads, kStill || kAppend == 2 ? 4 : 0)
    rope_kernel(const __grid_constant__ RopeParams p, const __grid_constant__ RopeTable tbl) {
  constexpr int kSlices = D / 16;                               // threads per row
  constexpr int kHeads = kRopeThreads / (kSlices * kTok);       // heads of a CTA at a time
  constexpr int kPieces = Vec16<T>::kPieces;
  launch_dependents();
  wait_prerequisites();
  const int sl = threadIdx.x % kSlices;
  const long long t = static_cast<long long>(blockIdx.x) * kTok + threadIdx.x / kSlices % kTok;
  const long long n_tok = static_cast<long long>(p.B) * p.S;
  if (t >= n_tok) return;
  const long long b = kAppend ? 0 : t / p.S, s = kAppend ? t : t - b * p.S;
  bool live = true;
  const bool one = blockIdx.y == 0 && sl == 0 && threadIdx.x < kSlices * kTok;
  const Slot slot = kAppend ? slot_of(p.cache, p.guard, t, n_tok, one, &live) : Slot{-1, 0};
  float cn[8], sn[8];
  __half2 low[kAppend == 2 ? 8 : 1];  // to codes: what the floats leave of cosine and sine, times 2^24 (at most 1/2)
  unsigned still = 0;  // pairs that are copied
  if (p.positions != nullptr) {
    const int *pos = p.positions + b * p.pos_b + s;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int axis = tbl.axis[8 * sl + k];
      if (kStill && axis < 0) still |= 1u << k;
      const long long at = axis < 0 ? 0 : pos[axis * p.pos_axis];
      // position times turns per position, whole turns dropped: [-1/2, 1/2) turns in 64 bits
      const long long turn = static_cast<long long>(static_cast<uint64_t>(at) * tbl.turns[8 * sl + k]);
      if constexpr (kAppend == 2) {
        const SineCosine a = sine_cosine(turn);
        sn[k] = a.s;
        cn[k] = a.c;
        low[k] = __floats2half2_rn(a.c_lo * 16777216.f, a.s_lo * 16777216.f);
      } else {
        sincospif(static_cast<float>(turn) * 0x1p-63f, &sn[k], &cn[k]);
        if (p.inverse) sn[k] = -sn[k];
      }
    }
  }
  constexpr int kRows = kStill && sizeof(T) == 4 ? 2 : 4;  // in flight
  const int heads = p.q.heads + p.k.heads + (kAppend ? p.v.heads : 0);
  const int h_per = (heads + gridDim.y - 1) / gridDim.y;
  const int h0 = blockIdx.y * h_per + threadIdx.x / (kSlices * kTok), h1 = min(heads, static_cast<int>(blockIdx.y + 1) * h_per);
  // this thread's heads among those of one tensor, which are first .. first + n - 1 of all
  auto rows = [&](int first, int n, const T *src, long long src_h, T *dst, long long dst_h, bool turned) {
    const int lo = h0 >= first ? h0 : first + (kHeads - (first - h0) % kHeads) % kHeads;
    const int hi = min(h1, first + n);
#pragma unroll kRows
    for (int h = lo; h < hi; h += kHeads) {
      const T *from = src + (h - first) * src_h;
      T *to = dst + (h - first) * dst_h;
      uint4 w[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        w[i] = __ldcs(reinterpret_cast<const uint4 *>(from + piece_at<T, D, kInterleaved>(sl, i)));
      if (turned) {
        float v[16], y[16];
        unpack(w, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int i1 = kInterleaved ? 2 * k : k, i2 = kInterleaved ? 2 * k + 1 : k + 8;
          y[i1] = fmaf(v[i1], cn[k], -v[i2] * sn[k]);
          y[i2] = fmaf(v[i1], sn[k], v[i2] * cn[k]);
        }
        if (kStill) {
          uint4 turned_w[kPieces];
          pack(y, turned_w);
          keep_copied<T, kInterleaved>(still, turned_w, w);
        } else {
          pack(y, w);
        }
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i)  // (streaming stores: 2 % of a long sequence's time)
        __stcs(reinterpret_cast<uint4 *>(to + piece_at<T, D, kInterleaved>(sl, i)), w[i]);
    }
  };
  auto in = [&](const RopeView &x) { return static_cast<const T *>(x.in) + (kAppend ? 0 : b * x.in_b) + s * x.in_s; };
  auto out = [&](const RopeView &x) { return static_cast<T *>(x.out) + (kAppend ? 0 : b * x.out_b) + s * x.out_s; };
  if (live) rows(0, p.q.heads, in(p.q), p.q.in_h, out(p.q), p.q.out_h, true);
  if (!kAppend) {
    rows(p.q.heads, p.k.heads, in(p.k), p.k.in_h, out(p.k), p.k.out_h, true);
  } else if (slot.page >= 0) {
    const long long page_h = static_cast<long long>(p.cache.page_size) * D;
    const long long to = static_cast<long long>(slot.page) * p.cache.page_stride + static_cast<long long>(slot.at) * D;
    if constexpr (kAppend == 1) {
      rows(p.q.heads, p.k.heads, in(p.k), p.k.in_h, static_cast<T *>(p.cache.k_pages) + to, page_h, p.positions != nullptr);
      rows(p.q.heads + p.k.heads, p.v.heads, in(p.v), p.v.in_h, static_cast<T *>(p.cache.v_pages) + to, page_h, false);
    } else if constexpr (kAppend == 2) {
      const long long scale_at = slot.page * p.scales.page_stride + slot.at;
      auto quantise = [&](int first, int n, const T *src, long long src_h, void *pool, unsigned char *scales, bool turned) {
        const int lo = h0 >= first ? h0 : first + (kHeads - (first - h0) % kHeads) % kHeads;
        const int hi = min(h1, first + n);
#pragma unroll 1  // (a row has arithmetic enough; two or four take registers that copies of q lack)
        for (int h = lo; h < hi; h += kHeads) {
          const T *from = src + (h - first) * src_h;
          uint4 w[kPieces];
#pragma unroll
          for (int i = 0; i < kPieces; ++i)
            w[i] = __ldcs(reinterpret_cast<const uint4 *>(from + piece_at<T, D, kInterleaved>(sl, i)));
          float v[16], y[16];
          unpack(w, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int i1 = kInterleaved ? 2 * k : k, i2 = kInterleaved ? 2 * k + 1 : k + 8;
            const bool as_is = !turned || (kStill && (still >> k & 1u));
            const float c_lo = __low2float(low[k]) * 0x1p-24f, s_lo = __high2float(low[k]) * 0x1p-24f;
            y[i1] = as_is ? v[i1] : turned_pair(v[i1], cn[k], c_lo, v[i2], sn[k], s_lo);
            y[i2] = as_is ? v[i2] : turned_pair(v[i1], sn[k], s_lo, -v[i2], cn[k], c_lo);
          }
          const int e = scale_of<kSlices>(y);
          const float by = __int_as_float((127 - e) << 23);  // 2^-e
          uint2 c[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float *z = y + 8 * i;
            c[i].x = pack_e4m3x2(z[0] * by, z[1] * by) | pack_e4m3x2(z[2] * by, z[3] * by) << 16;
            c[i].y = pack_e4m3x2(z[4] * by, z[5] * by) | pack_e4m3x2(z[6] * by, z[7] * by) << 16;
          }
          unsigned char *dst = static_cast<unsigned char *>(pool) + to + (h - first) * page_h;
          if (kInterleaved) {
            __stcs(reinterpret_cast<uint4 *>(dst + 16 * sl), make_uint4(c[0].x, c[0].y, c[1].x, c[1].y));
          } else {
            __stcs(reinterpret_cast<uint2 *>(dst + 8 * sl), c[0]);
            __stcs(reinterpret_cast<uint2 *>(dst + 8 * sl + D / 2), c[1]);
          }
          if (sl == 0) scales[scale_at + (h - first) * static_cast<long long>(p.cache.page_size)] = static_cast<unsigned char>(e + 127);
        }
      };
      quantise(p.q.heads, p.k.heads, in(p.k), p.k.in_h, p.cache.k_pages, p.scales.k, p.positions != nullptr);
      quantise(p.q.heads + p.k.heads, p.v.heads, in(p.v), p.v.in_h, p.cache.v_pages, p.scales.v, false);
    }
  }
}

template <typename T, int D, bool kInterleaved, int kAppend, int kTok, bool kStill>
cudaError_t launch_tile(const RopeParams &p, const RopeTable &tbl, cudaStream_t stream) {
  const long long n_tok = static_cast<long long>(p.B) * p.S;
  const long long tiles = (n_tok + kTok - 1) / kTok;
  const int heads = p.q.heads + p.k.heads + (kAppend ? p.v.heads : 0);
  constexpr int kHeads = kRopeThreads / (D / 16 * kTok);
  // few tiles: the heads are dealt over more CTAs, down to one row a thread
  long long want = static_cast<long long>(device_sm_count()) * 4 / tiles;
  const long long most = (heads + kHeads - 1) / kHeads;
  want = want < 1 ? 1 : (want > most ? most : want);
  if (tiles > 0x7fffffffll || want > 65535) return cudaErrorInvalidValue;
  return launch_dependent(rope_kernel<T, D, kInterleaved, kAppend, kTok, kStill>,
                          dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(want)), dim3(kRopeThreads), 0, stream, p,
                          tbl);
}

template <typename T, int D, int kAppend, bool kStill>
cudaError_t launch_variant(const RopeParams &p, const RopeTable &tbl, bool interleaved, cudaStream_t stream) {
  // Tiles of 32 tokens give a thread the most heads to its sines (32,768 tokens
  // of 32 heads in bf16: 89 us; tiles of 16 and 8: 4 us more); with fewer tokens than
  // one such tile an SM, tiles of 4 give more CTAs.
  const bool small = static_cast<long long>(p.B) * p.S < 32ll * device_sm_count();
  if (interleaved)
    return small ? launch_tile<T, D, true, kAppend, 4, kStill>(p, tbl, stream)
                 : launch_tile<T, D, true, kAppend, 32, kStill>(p, tbl, stream);
  return small ? launch_tile<T, D, false, kAppend, 4, kStill>(p, tbl, stream)
               : launch_tile<T, D, false, kAppend, 32, kStill>(p, tbl, stream);
}

template <typename T, int D, int kAppend>
cudaError_t launch_typed_rope(const RopeParams &p, const RopeTable &tbl, bool interleaved, cudaStream_t stream) {
  bool still = false;
  for (int i = 0; i < D / 2; ++i) still |= tbl.axis[i] < 0;
  return still ? launch_variant<T, D, kAppend, true>(p, tbl, interleaved, stream)
               : launch_variant<T, D, kAppend, false>(p, tbl, interleaved, stream);
}

// ---------------------------------------------------------------- reading back
// A CTA has kReadTok packed rows and a share of the heads: it finds the slot of
// each row once, then copies (or turns to bf16, exactly: four significant bits times
// a power of two) 16 elements a thread, K and V of a head after each other. Rows
// without a key come out as zeros. Bound by DRAM.
constexpr int kReadThreads = 256, kReadTok = 32;

// 16 e4m3 codes times 2^e as bf16.
__device__ __forceinline__ void widen(const uint4 &c, float scale, uint4 (&out)[2]) {
  const uint32_t u[4] = {c.x, c.y, c.z, c.w};
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(u[i / 2] >> (16 * (i % 2)))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * scale, f.y * scale);
    w[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  out[0] = make_uint4(w[0], w[1], w[2], w[3]);
  out[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kSlices = D / 16, kRows = kReadThreads / kSlices;  // threads of a row; rows at a time
  static_assert(kRows % kReadTok == 0 || kReadTok % kRows == 0, "whole heads at a time");
  __shared__ int page_of[kReadTok], at_of[kReadTok];  // page -1: zeros, -2: no row
  launch_dependents();
  wait_prerequisites();
  const long long t0 = static_cast<long long>(blockIdx.x) * kReadTok;
  const PagedView &c = p.cache;
  if (threadIdx.x < kReadTok) {
    const long long t = t0 + threadIdx.x;
    int page = -2, at = 0;
    int lo = 0, hi = c.B;  // the first sequence that ends behind t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (c.cu_seqlens[mid + 1] <= t) lo = mid + 1;
      else hi = mid;
    }
    if (t < p.total && lo < c.B && c.cu_seqlens[lo] <= t) {
      const long long max_keys = static_cast<long long>(c.max_pages) * c.page_size;
      const long long len = min(static_cast<long long>(c.kv_lens[lo]), max_keys);
      const long long key = t - max(c.cu_seqlens[lo], 0) + (p.first ? p.first[lo] : 0);
      page = -1;
      if (key >= 0 && key < len) {
        const int e = c.page_table[lo * c.table_stride + key / c.page_size];
        if (e >= 0 && e < c.n_pages) {
          page = e;
          at = static_cast<int>(key % c.page_size);
        }
      }
    }
    page_of[threadIdx.x] = page;
    at_of[threadIdx.x] = at;
  }
  __syncthreads();
  const int sl = threadIdx.x % kSlices;
  const int lines = 2 * c.Hkv * kReadTok;  // (K or V, head, row), row fastest
  const int per = ((lines / kReadTok + gridDim.y - 1) / gridDim.y) * kReadTok;
  const int l1 = min(lines, static_cast<int>(blockIdx.y + 1) * per);
#pragma unroll 4
  for (int line = blockIdx.y * per + threadIdx.x / kSlices; line < l1; line += kRows) {
    const int r = line % kReadTok, h = line / kReadTok % c.Hkv;
    const bool v = line >= c.Hkv * kReadTok;
    const int page = page_of[r];
    if (page == -2) continue;
    uint4 out[2] = {};
    if (page >= 0) {
      const long long at = page * c.page_stride + (static_cast<long long>(h) * c.page_size + at_of[r]) * D + 16 * sl;
      if constexpr (kE4m3) {
        const unsigned e = (v ? p.scales.v : p.scales.k)[page * p.scales.page_stride + h * static_cast<long long>(c.page_size) + at_of[r]];
        const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(v ? c.v_pages : c.k_pages) + at));
        widen(x, scale_value(e), out);
      } else {
        const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(v ? c.v_pages : c.k_pages) + at);
        out[0] = __ldcs(x);
        out[1] = __ldcs(x + 1);
      }
    }
    const long long t = t0 + r;
    uint4 *to = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(v ? p.v : p.k) + h * (v ? p.v_h : p.k_h) +
                                          t * (v ? p.v_s : p.k_s) + 16 * sl);
    __stcs(to, out[0]);
    __stcs(to + 1, out[1]);
  }
}

template <int D, bool kE4m3>
cudaError_t launch_typed_read(const ReadParams &p, cudaStream_t stream) {
  const int tiles = (p.total + kReadTok - 1) / kReadTok;
  // few tiles: K and V and their heads over more CTAs, 24 an SM (8: 51.7 us for the keys
  // above, 16: 46.6, 32: 43.9)
  const long long want = (static_cast<long long>(device_sm_count()) * 24 + tiles - 1) / tiles;
  const long long y = want < 2 * p.cache.Hkv ? want : 2 * p.cache.Hkv;
  return launch_dependent(read_kernel<D, kE4m3>, dim3(tiles, static_cast<unsigned>(y)), dim3(kReadThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_read(const ReadParams &p, int D, bool e4m3, cudaStream_t stream) {
  if (e4m3) return D == 64 ? launch_typed_read<64, true>(p, stream) : launch_typed_read<128, true>(p, stream);
  return D == 64 ? launch_typed_read<64, false>(p, stream) : launch_typed_read<128, false>(p, stream);
}

cudaError_t launch_rope(const RopeParams &p, const RopeTable &tbl, int D, bool f32, bool interleaved,
                        cudaStream_t stream) {
  if (f32) return D == 64 ? launch_typed_rope<float, 64, 0>(p, tbl, interleaved, stream)
                          : launch_typed_rope<float, 128, 0>(p, tbl, interleaved, stream);
  return D == 64 ? launch_typed_rope<__nv_bfloat16, 64, 0>(p, tbl, interleaved, stream)
                 : launch_typed_rope<__nv_bfloat16, 128, 0>(p, tbl, interleaved, stream);
}

cudaError_t launch_append(const RopeParams &p, const RopeTable &tbl, int D, bool e4m3, bool interleaved,
                          cudaStream_t stream) {
  if (e4m3) return D == 64 ? launch_typed_rope<__nv_bfloat16, 64, 2>(p, tbl, interleaved, stream)
                           : launch_typed_rope<__nv_bfloat16, 128, 2>(p, tbl, interleaved, stream);
  return D == 64 ? launch_typed_rope<__nv_bfloat16, 64, 1>(p, tbl, interleaved, stream)
                 : launch_typed_rope<__nv_bfloat16, 128, 1>(p, tbl, interleaved, stream);
}

}  // namespace seqattn
