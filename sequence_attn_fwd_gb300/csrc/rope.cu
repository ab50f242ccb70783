// Rotary positions with several axes, alone and on the way into a paged cache.
//
// Pair i of a row is turned by positions[axis_i] * inv_freq_i. The angle is
// formed in turns, in 64-bit fixed point: f_i = inv_freq_i / 2 pi as a binary
// fraction of 64 bits (made on the host in double), position * f_i modulo 2^64
// by one integer product, so whole turns drop out exactly and a position of
// 10^6 costs no precision; the signed fraction, as a float, goes through
// sincospif.
//
// Memory-bound: every element is read and written once. A CTA takes a tile of
// kTok tokens and a share of the heads: the tile's sines and cosines are
// formed once in shared memory (D / 2 per token, instead of per head and
// token), then each thread takes 16 elements of one (head, token) row -- eight
// pairs, two 16-byte pieces in bf16, four in fp32 -- so that D / 16 threads
// cover a row with whole 32-byte sectors in either pairing.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kernels.h"

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

// The rows of one launch: heads [0, q.H) of q, then those of k, then those of v
// (v only in an append).
template <typename T, int D, bool kInterleaved, bool kAppend, int kTok>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeParams p, const __grid_constant__ RopeTable tbl) {
  __shared__ float2 cs[kTok][D / 2];
  __shared__ long long slot_at[kTok];  // append: element offset of the token's slot in the pools, -1: dropped
  __shared__ int live[kTok];           // append: the token belongs to a sequence
  const long long t0 = static_cast<long long>(blockIdx.x) * kTok;
  const long long n_tok = static_cast<long long>(p.B) * p.S;
  if (kAppend && threadIdx.x < kTok) {
    const long long t = t0 + threadIdx.x;
    const PagedView &c = p.cache;
    long long at = -1;
    int in = 0;
    if (t < n_tok) {
      // the last sequence that starts at or before t
      int lo = 0, hi = c.B;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (c.cu_seqlens[mid + 1] <= t) lo = mid + 1;
        else hi = mid;
      }
      if (lo < c.B && c.cu_seqlens[lo] <= t) {
        in = 1;
        const long long max_keys = static_cast<long long>(c.max_pages) * c.page_size;
        long long len = c.kv_lens[lo];
        len = len < 0 ? 0 : (len > max_keys ? max_keys : len);
        const long long end = c.cu_seqlens[lo + 1] < n_tok ? c.cu_seqlens[lo + 1] : n_tok;
        const long long slot = len - (end - t);
        if (slot >= 0) {
          const long long pi = slot / c.page_size;
          const int page = c.page_table[lo * c.table_stride + pi];
          if (page >= 0 && page < c.n_pages)
            at = static_cast<long long>(page) * c.page_stride + (slot % c.page_size) * D;
        }
      }
    }
    slot_at[threadIdx.x] = at;
    live[threadIdx.x] = in;
  }
  if (p.positions != nullptr) {
    for (int i = threadIdx.x; i < kTok * (D / 2); i += kRopeThreads) {
      const int tt = i / (D / 2), pr = i % (D / 2);
      const long long t = t0 + tt;
      if (t >= n_tok) break;
      const long long b = kAppend ? 0 : t / p.S, s = kAppend ? t : t - b * p.S;
      const int axis = tbl.axis[pr];
      const long long pos = axis < 0 ? 0 : p.positions[axis * p.pos_axis + b * p.pos_b + s];
      // position times turns per position, whole turns dropped: [-1/2, 1/2) turns in 64 bits
      const long long turn = static_cast<long long>(static_cast<uint64_t>(pos) * tbl.turns[pr]);
      float sn, cn;
      sincospif(static_cast<float>(turn) * 0x1p-63f, &sn, &cn);
      cs[tt][pr] = make_float2(cn, p.inverse ? -sn : sn);
    }
  }
  __syncthreads();

  constexpr int kSlices = D / 16;                          // threads per row
  constexpr int kRowsPerPass = kRopeThreads / kSlices;
  const int sl = threadIdx.x % kSlices;
  const int heads = p.q.heads + p.k.heads + (kAppend ? p.v.heads : 0);
  const int h_per = (heads + gridDim.y - 1) / gridDim.y;
  const int h0 = blockIdx.y * h_per, h1 = min(heads, h0 + h_per);
  const int n_rows = (h1 - h0) * kTok;
#pragma unroll 2
  for (int r = threadIdx.x / kSlices; r < n_rows; r += kRowsPerPass) {
    const int h = h0 + r / kTok, tt = r % kTok;
    const long long t = t0 + tt;
    if (t >= n_tok) continue;
    const bool is_q = h < p.q.heads;
    const bool is_v = kAppend && h >= p.q.heads + p.k.heads;
    const RopeView &x = is_q ? p.q : (is_v ? p.v : p.k);
    const int hh = is_q ? h : (is_v ? h - p.q.heads - p.k.heads : h - p.q.heads);
    const long long b = kAppend ? 0 : t / p.S, s = kAppend ? t : t - b * p.S;
    T *dst;
    if (kAppend) {
      if (is_q) {
        if (!live[tt]) continue;
        dst = static_cast<T *>(x.out) + hh * x.out_h + s * x.out_s;
      } else {
        if (slot_at[tt] < 0) continue;
        dst = static_cast<T *>(is_v ? p.cache.v_pages : p.cache.k_pages) + slot_at[tt] +
              static_cast<long long>(hh) * p.cache.page_size * D;
      }
    } else {
      dst = static_cast<T *>(x.out) + b * x.out_b + hh * x.out_h + s * x.out_s;
    }
    const T *src = static_cast<const T *>(x.in) + (kAppend ? 0 : b * x.in_b) + hh * x.in_h + s * x.in_s;
    constexpr int kPieces = Vec16<T>::kPieces;
    uint4 w[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      w[i] = __ldcs(reinterpret_cast<const uint4 *>(src + piece_at<T, D, kInterleaved>(sl, i)));
    if (p.positions != nullptr && !is_v) {
      float v[16], y[16];
      unpack(w, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 c = cs[tt][8 * sl + k];
        const int i1 = kInterleaved ? 2 * k : k, i2 = kInterleaved ? 2 * k + 1 : k + 8;
        y[i1] = fmaf(v[i1], c.x, -v[i2] * c.y);
        y[i2] = fmaf(v[i1], c.y, v[i2] * c.x);
      }
      pack(y, w);
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      *reinterpret_cast<uint4 *>(dst + piece_at<T, D, kInterleaved>(sl, i)) = w[i];
  }
}

template <typename T, int D, bool kInterleaved, bool kAppend, int kTok>
cudaError_t launch_tile(const RopeParams &p, const RopeTable &tbl, cudaStream_t stream) {
  const long long n_tok = static_cast<long long>(p.B) * p.S;
  const long long tiles = (n_tok + kTok - 1) / kTok;
  const int heads = p.q.heads + p.k.heads + (kAppend ? p.v.heads : 0);
  constexpr int kRowsPerPass = kRopeThreads / (D / 16);
  // few tiles: the heads are dealt over more CTAs, down to one pass each
  long long want = static_cast<long long>(device_sm_count()) * 4 / tiles;
  const long long most = (static_cast<long long>(heads) * kTok + kRowsPerPass - 1) / kRowsPerPass;
  want = want < 1 ? 1 : (want > most ? most : want);
  if (want > heads) want = heads;
  if (tiles > 0x7fffffffll || want > 65535) return cudaErrorInvalidValue;
  rope_kernel<T, D, kInterleaved, kAppend, kTok>
      <<<dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(want)), kRopeThreads, 0, stream>>>(p, tbl);
  return cudaGetLastError();
}

template <typename T, int D, bool kAppend>
cudaError_t launch_typed_rope(const RopeParams &p, const RopeTable &tbl, bool interleaved, cudaStream_t stream) {
  // Tiles of 16 tokens share their sines among the heads; with few tokens
  // tiles of 4 give more CTAs.
  const bool small = static_cast<long long>(p.B) * p.S < 16ll * 4 * device_sm_count();
  if (interleaved)
    return small ? launch_tile<T, D, true, kAppend, 4>(p, tbl, stream) : launch_tile<T, D, true, kAppend, 16>(p, tbl, stream);
  return small ? launch_tile<T, D, false, kAppend, 4>(p, tbl, stream) : launch_tile<T, D, false, kAppend, 16>(p, tbl, stream);
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
