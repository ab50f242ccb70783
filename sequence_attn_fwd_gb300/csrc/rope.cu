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

// The slot of token t of an append: its element offset in the pools, -1 if it has
// none; *live: whether the token belongs to a sequence. `one`: of the threads with
// this token, the one that writes for a guarded row.
__device__ __forceinline__ long long slot_of(const PagedView &c, int *guard, long long t, long long n_tok, int D,
                                             bool one, bool *live) {
  int lo = 0, hi = c.B;  // the first sequence that ends behind t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (c.cu_seqlens[mid + 1] <= t) lo = mid + 1;
    else hi = mid;
  }
  *live = lo < c.B && c.cu_seqlens[lo] <= t;
  if (!*live) return -1;
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
    if (refused) return -1;
  }
  if (slot < 0) return -1;
  const int page = c.page_table[lo * c.table_stride + slot / c.page_size];
  if (page < 0 || page >= c.n_pages) return -1;
  return static_cast<long long>(page) * c.page_stride + (slot % c.page_size) * D;
}

// blockIdx.x: tile of kTok tokens; blockIdx.y: share of the heads (those of q,
// then k, then, in an append, v). kStill: some pairs are copied, whatever they hold
// (turned by an angle of 0, an infinity would make its partner NaN). A variant of
// its own: tested in the one loop, it cost the others 17 %. Held to 64 registers,
// and to two rows in flight in fp32, it takes their time (32,768 tokens of 28 heads
// of 128, halves and neighbours as pairs: bf16 81 and 83 us, fp32 153 and 165; with
// 72 to 77 registers 94 and 96, 163 and 179; with four fp32 rows in flight 162 and 179).
template <typename T, int D, bool kInterleaved, bool kAppend, int kTok, bool kStill>
__global__ void __launch_bounds__(kRopeThreads, kStill ? 4 : 0)
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
  const long long slot = kAppend ? slot_of(p.cache, p.guard, t, n_tok, D, one, &live) : -1;
  float cn[8], sn[8];
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
      sincospif(static_cast<float>(turn) * 0x1p-63f, &sn[k], &cn[k]);
      if (p.inverse) sn[k] = -sn[k];
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
  } else if (slot >= 0) {
    const long long page_h = static_cast<long long>(p.cache.page_size) * D;
    rows(p.q.heads, p.k.heads, in(p.k), p.k.in_h, static_cast<T *>(p.cache.k_pages) + slot, page_h, p.positions != nullptr);
    rows(p.q.heads + p.k.heads, p.v.heads, in(p.v), p.v.in_h, static_cast<T *>(p.cache.v_pages) + slot, page_h, false);
  }
}

template <typename T, int D, bool kInterleaved, bool kAppend, int kTok, bool kStill>
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

template <typename T, int D, bool kAppend, bool kStill>
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

template <typename T, int D, bool kAppend>
cudaError_t launch_typed_rope(const RopeParams &p, const RopeTable &tbl, bool interleaved, cudaStream_t stream) {
  bool still = false;
  for (int i = 0; i < D / 2; ++i) still |= tbl.axis[i] < 0;
  return still ? launch_variant<T, D, kAppend, true>(p, tbl, interleaved, stream)
               : launch_variant<T, D, kAppend, false>(p, tbl, interleaved, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, const RopeTable &tbl, int D, bool f32, bool interleaved,
                        cudaStream_t stream) {
  if (f32) return D == 64 ? launch_typed_rope<float, 64, false>(p, tbl, interleaved, stream)
                          : launch_typed_rope<float, 128, false>(p, tbl, interleaved, stream);
  return D == 64 ? launch_typed_rope<__nv_bfloat16, 64, false>(p, tbl, interleaved, stream)
                 : launch_typed_rope<__nv_bfloat16, 128, false>(p, tbl, interleaved, stream);
}

cudaError_t launch_append(const RopeParams &p, const RopeTable &tbl, int D, bool interleaved, cudaStream_t stream) {
  return D == 64 ? launch_typed_rope<__nv_bfloat16, 64, true>(p, tbl, interleaved, stream)
                 : launch_typed_rope<__nv_bfloat16, 128, true>(p, tbl, interleaved, stream);
}

}  // namespace seqattn
