// C-ABI entry points of the serving side (declared in include/seqattn_paged.h):
// argument validation, tensor maps and launches. Nothing here allocates or
// synchronises, and nothing is thrown.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/seqattn_paged.h"
#include "kernels.h"

namespace {

using seqattn::keep_cuda_error;

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int done(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : keep_cuda_error(e); }

constexpr long long kMaxKeys = 1ll << 30;

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

int check_cache(const paged_cache *c) {
  if (!c || c->B < 0 || c->Hkv <= 0 || c->n_pages <= 0 || c->max_pages < 0 || c->page_size <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return ATTN_ERR_UNSUPPORTED;
  if (c->page_size < 16 || (c->page_size & (c->page_size - 1))) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->max_pages) * c->page_size > kMaxKeys) return ATTN_ERR_UNSUPPORTED;
  if (c->B > seqattn::kPagedMaxSeqs || c->Hkv > 65535) return ATTN_ERR_UNSUPPORTED;
  const long long page = static_cast<long long>(c->Hkv) * c->page_size * c->D;
  if (c->page_stride < page || c->page_stride % 8 != 0) return ATTN_ERR_INVALID_ARG;
  if (c->table_stride < c->max_pages) return ATTN_ERR_INVALID_ARG;
  if (c->B == 0) return ATTN_OK;
  if (!c->k_pages || !c->v_pages || !aligned(c->k_pages, 16) || !aligned(c->v_pages, 16)) return ATTN_ERR_INVALID_ARG;
  if ((!c->page_table && c->max_pages > 0) || !c->kv_lens || !c->cu_seqlens || !aligned(c->page_table, 4) ||
      !aligned(c->kv_lens, 4) || !aligned(c->cu_seqlens, 4))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

seqattn::PagedView view_of(const paged_cache *c) {
  return {c->k_pages, c->v_pages, c->page_stride, c->page_table, c->table_stride, c->kv_lens,
          c->cu_seqlens, c->B, c->n_pages, c->page_size, c->max_pages, c->Hkv};
}

// 4-D bf16 map, dimension 0 contiguous, box 64 x b1 x b2 x 1, 128-byte swizzle.
bool make_map_4d(CUtensorMap *map, const void *base, const cuuint64_t (&dims)[4], const cuuint64_t (&strides)[3],
                 unsigned b1, unsigned b2) {
  using Fn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                          const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                          CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  Fn fn = reinterpret_cast<Fn>(seqattn::tensor_map_encoder());
  if (!fn) return false;
  const cuuint32_t box[4] = {64u, b1, b2, 1u}, one[4] = {1u, 1u, 1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a work item that can hold a token: two tiles of whole tokens, or all of them.
int rows_per_item(int G, int total_q) {
  const long long most = 2ll * (128 / G) * G, all = static_cast<long long>(total_q) * G;
  return static_cast<int>(all < most ? all : most);
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

struct Workspace {
  size_t lse, cuts, total;
};
Workspace workspace_of(int G, int total_q, int D) {
  const size_t rows = static_cast<size_t>(2 * seqattn::kPagedMaxCtas) * rows_per_item(G, total_q);
  const size_t lse = round256(rows * D * sizeof(float)), cuts = lse + round256(rows * sizeof(float));
  return {lse, cuts, cuts + round256(seqattn::kPagedMaxCtas * sizeof(int4))};
}

// A tensor of rows: strides in elements, multiples of 16 bytes (of dimensions
// longer than one: torch leaves the others arbitrary).
bool rows_ok(const rope_rows *x, bool with_out, int B, int S, int elem) {
  if (!x) return true;
  if (x->heads < 0) return false;
  if (x->heads == 0) return true;
  if (!x->in || !aligned(x->in, 16) || (with_out && (!x->out || !aligned(x->out, 16)))) return false;
  const long long unit = 16 / elem;
  auto ok = [&](long long b, long long h, long long s) {
    return (B <= 1 || b % unit == 0) && (x->heads <= 1 || h % unit == 0) && (S <= 1 || s % unit == 0);
  };
  return ok(x->in_b, x->in_h, x->in_s) && (!with_out || ok(x->out_b, x->out_h, x->out_s));
}
seqattn::RopeView rows_of(const rope_rows *x) {
  if (!x) return {nullptr, nullptr, 0, 0, 0, 0, 0, 0, 0};
  return {x->in, x->out, x->in_b, x->in_h, x->in_s, x->out_b, x->out_h, x->out_s, x->heads};
}

// Radians per position to turns per position modulo one, 64 fraction bits.
int make_table(seqattn::RopeTable *t, const double *inv_freq, const int *axes, int D, int n_axes) {
  if (!inv_freq || !axes || n_axes < 1) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < D / 2; ++i) {
    if (axes[i] < -1 || axes[i] >= n_axes || axes[i] > 127) return ATTN_ERR_INVALID_ARG;
    if (!isfinite(inv_freq[i])) return ATTN_ERR_INVALID_ARG;
    const double turns = inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    double frac = turns - floor(turns);
    if (frac >= 1.0) frac = 0.0;  // a tiny negative rounds up to a whole turn
    t->turns[i] = static_cast<uint64_t>(frac * 18446744073709551616.0);  // times 2^64, exact; below it, as frac < 1
    t->axis[i] = static_cast<signed char>(axes[i]);
  }
  return ATTN_OK;
}

int check_tables(const int *page_table, long long table_stride, int B, int max_pages, int n_pages) {
  if (B < 0 || max_pages < 0 || n_pages <= 0 || table_stride < max_pages) return ATTN_ERR_INVALID_ARG;
  if (B > seqattn::kPagedMaxRows || static_cast<long long>(B) * max_pages > 0x7fffffffll || n_pages > (1 << 28))
    return ATTN_ERR_UNSUPPORTED;
  if (B > 0 && max_pages > 0 && (!page_table || !aligned(page_table, 4))) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

int check_page_size(int page_size, int max_pages) {
  if (page_size <= 0) return ATTN_ERR_INVALID_ARG;
  if (page_size < 16 || (page_size & (page_size - 1))) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > kMaxKeys) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// The pools by value, empty ones left out.
int make_pools(seqattn::PoolList *list, const paged_pool *pools, int n, int n_pages) {
  if (n < 0 || (n > 0 && !pools)) return ATTN_ERR_INVALID_ARG;
  if (n > seqattn::kMaxPools) return ATTN_ERR_UNSUPPORTED;
  list->n = list->total_layers = 0;
  long long items = 0, layers = 0;  // at most 32 x 2^31
  for (int i = 0; i < n; ++i) {
    const paged_pool &p = pools[i];
    if (p.n_layers < 0 || p.page_bytes < 0) return ATTN_ERR_INVALID_ARG;
    if (p.n_layers == 0 || p.page_bytes == 0) continue;
    if (!p.base || !aligned(p.base, 16) || p.page_bytes % 16 != 0 || p.page_stride % 16 != 0 || p.layer_stride % 16 != 0)
      return ATTN_ERR_INVALID_ARG;
    if (n_pages > 1 && p.page_stride < p.page_bytes) return ATTN_ERR_INVALID_ARG;
    list->pool[list->n++] = {static_cast<unsigned char *>(p.base), p.layer_stride, p.page_stride, p.page_bytes, p.n_layers};
    layers += p.n_layers;
    items += (p.page_bytes - 1) / 16384 + 1;
  }
  // copies of 16 KB of one page
  if (items > (1 << 30) || layers > (1 << 30) || items * layers > (1 << 30)) return ATTN_ERR_UNSUPPORTED;
  list->total_layers = static_cast<int>(layers);
  return ATTN_OK;
}

}  // namespace

extern "C" {

size_t attn_paged_workspace_bytes(int Hq, int Hkv, int total_q, int D) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Hq / Hkv > 128 || total_q < 0 || (D != 64 && D != 128)) return 0;
  return workspace_of(Hq / Hkv, total_q > 0 ? total_q : 1, D).total;
}

int attn_paged(const void *q, long long q_head_stride, long long q_row_stride, const paged_cache *cache, void *o,
               long long o_head_stride, long long o_row_stride, float *lse, void *workspace, size_t workspace_bytes,
               int Hq, int total_q, int causal, float scale, attn_stream_t stream) {
  const int st = check_cache(cache);
  if (st != ATTN_OK) return st;
  if (Hq <= 0 || Hq % cache->Hkv != 0 || total_q < 0) return ATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (!isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  const int G = Hq / cache->Hkv, D = cache->D;
  if (G > 128 || total_q > kMaxKeys) return ATTN_ERR_UNSUPPORTED;
  // the key tiles of all items, and a few more each, are counted in 32 bits
  const long long items = (static_cast<long long>(total_q) / (2 * (128 / G)) + cache->B) * cache->Hkv;
  const long long tiles = (static_cast<long long>(cache->max_pages) * cache->page_size + 127) / 128;
  if (items > 0x7fffffffll / (tiles + 16)) return ATTN_ERR_UNSUPPORTED;
  if (cache->B == 0 || total_q == 0) return ATTN_OK;
  if (!q || !o || !workspace || !aligned(q, 16) || !aligned(o, 16) || !aligned(workspace, 16) || !aligned(lse, 4))
    return ATTN_ERR_INVALID_ARG;
  // strides of dimensions of one are not looked at; no other may make rows overlap
  if (Hq > 1 && (q_head_stride % 8 || o_head_stride % 8 || q_head_stride < D || o_head_stride < D)) return ATTN_ERR_INVALID_ARG;
  if (total_q > 1 && (q_row_stride % 8 || o_row_stride % 8 || q_row_stride < D || o_row_stride < D)) return ATTN_ERR_INVALID_ARG;
  const Workspace ws = workspace_of(G, total_q, D);
  if (workspace_bytes < ws.total) return ATTN_ERR_INVALID_ARG;

  const cuuint64_t uD = static_cast<cuuint64_t>(D);
  const cuuint64_t qh = Hq > 1 ? static_cast<cuuint64_t>(q_head_stride) : uD;
  const cuuint64_t qs = total_q > 1 ? static_cast<cuuint64_t>(q_row_stride) : uD;
  const int tok = 128 / G;
  CUtensorMap tq{}, tqn[3] = {}, tk, tv;
  const cuuint64_t q_dims[4] = {uD, static_cast<cuuint64_t>(G), static_cast<cuuint64_t>(total_q),
                                static_cast<cuuint64_t>(cache->Hkv)};
  const cuuint64_t q_strides[3] = {qh * 2, qs * 2, qh * 2 * G};
  const cuuint64_t kv_dims[4] = {uD, static_cast<cuuint64_t>(cache->page_size), static_cast<cuuint64_t>(cache->Hkv),
                                 static_cast<cuuint64_t>(cache->n_pages)};
  const cuuint64_t kv_strides[3] = {uD * 2, uD * 2 * cache->page_size, static_cast<cuuint64_t>(cache->page_stride) * 2};
  const unsigned box_rows = cache->page_size < 128 ? cache->page_size : 128;
  // the maps that the call can need: no sequence has more rows than all have
  const long long rows = static_cast<long long>(total_q) * G;
  for (int i = 0; i < 3; ++i) {
    const int few = (16 << i) / G;
    if ((i == 0 || rows > (8 << i)) && !make_map_4d(&tqn[i], q, q_dims, q_strides, G, few > 0 ? few : 1))
      return keep_cuda_error(cudaErrorInvalidValue);
  }
  if ((rows > 64 && !make_map_4d(&tq, q, q_dims, q_strides, G, tok)) ||
      !make_map_4d(&tk, cache->k_pages, kv_dims, kv_strides, box_rows, 1) ||
      !make_map_4d(&tv, cache->v_pages, kv_dims, kv_strides, box_rows, 1))
    return keep_cuda_error(cudaErrorInvalidValue);

  seqattn::PagedAttnParams p{};
  p.cache = view_of(cache);
  p.o = o;
  p.o_h = o_head_stride;
  p.o_s = o_row_stride;
  p.lse = lse;
  p.part_o = static_cast<float *>(workspace);
  p.part_lse = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + ws.lse);
  p.cuts = reinterpret_cast<int4 *>(static_cast<unsigned char *>(workspace) + ws.cuts);
  p.part_rows = rows_per_item(G, total_q);
  p.Hq = Hq;
  p.G = G;
  p.tok = tok;
  p.total_q = total_q;
  p.causal = causal;
  p.page_log2 = log2_of(cache->page_size);
  p.scale_log2 = scale * 1.4426950408889634f;
  return done(seqattn::launch_attn_paged(D, tq, tqn, tk, tv, p, reinterpret_cast<cudaStream_t>(stream)));
}

int rope_axes(const rope_rows *q, const rope_rows *k, const int *positions, long long pos_axis, long long pos_b,
              int n_axes, const double *inv_freq, const int *axes, int B, int S, int D, int dtype, int interleaved,
              int inverse, attn_stream_t stream) {
  if (B < 0 || S < 0 || (dtype != ATTN_BF16 && dtype != ATTN_F32)) return ATTN_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1)) return ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * S > kMaxKeys) return ATTN_ERR_UNSUPPORTED;
  seqattn::RopeTable tbl{};
  const int st = make_table(&tbl, inv_freq, axes, D, n_axes);
  if (st != ATTN_OK) return st;
  const int elem = dtype == ATTN_F32 ? 4 : 2;
  if (B == 0 || S == 0) return ATTN_OK;
  if (!rows_ok(q, true, B, S, elem) || !rows_ok(k, true, B, S, elem)) return ATTN_ERR_INVALID_ARG;
  if (!positions || !aligned(positions, 4)) return ATTN_ERR_INVALID_ARG;
  seqattn::RopeParams p{};
  p.q = rows_of(q);
  p.k = rows_of(k);
  if (p.q.heads + p.k.heads == 0) return ATTN_OK;
  p.positions = positions;
  p.pos_axis = pos_axis;
  p.pos_b = pos_b;
  p.B = B;
  p.S = S;
  p.inverse = inverse;
  return done(seqattn::launch_rope(p, tbl, D, dtype == ATTN_F32, interleaved != 0, reinterpret_cast<cudaStream_t>(stream)));
}

int paged_append(const rope_rows *q, const rope_rows *k, const rope_rows *v, const paged_cache *cache,
                 const int *positions, long long pos_axis, int n_axes, const double *inv_freq, const int *axes,
                 int total, int interleaved, attn_stream_t stream) {
  return paged_append_guarded(q, k, v, cache, positions, pos_axis, n_axes, inv_freq, axes, total, interleaved, nullptr,
                              stream);
}

int paged_append_guarded(const rope_rows *q, const rope_rows *k, const rope_rows *v, const paged_cache *cache,
                         const int *positions, long long pos_axis, int n_axes, const double *inv_freq, const int *axes,
                         int total, int interleaved, int *guard, attn_stream_t stream) {
  int st = check_cache(cache);
  if (st != ATTN_OK) return st;
  if (total < 0 || (interleaved != 0 && interleaved != 1)) return ATTN_ERR_INVALID_ARG;
  if (total > kMaxKeys) return ATTN_ERR_UNSUPPORTED;
  if (!k || !v || k->heads != cache->Hkv || v->heads != cache->Hkv) return ATTN_ERR_INVALID_ARG;
  if ((!positions && q && q->heads > 0) || !aligned(guard, 4)) return ATTN_ERR_INVALID_ARG;
  seqattn::RopeTable tbl{};
  if (positions) {
    if (!aligned(positions, 4)) return ATTN_ERR_INVALID_ARG;
    st = make_table(&tbl, inv_freq, axes, cache->D, n_axes);
    if (st != ATTN_OK) return st;
  }
  if (cache->B == 0 || total == 0) return ATTN_OK;
  if (!rows_ok(q, true, 1, total, 2) || !rows_ok(k, false, 1, total, 2) || !rows_ok(v, false, 1, total, 2))
    return ATTN_ERR_INVALID_ARG;
  seqattn::RopeParams p{};
  p.q = rows_of(q);
  p.k = rows_of(k);
  p.v = rows_of(v);
  p.cache = view_of(cache);
  p.guard = guard;
  p.positions = positions;
  p.pos_axis = pos_axis;
  p.B = 1;
  p.S = total;
  return done(seqattn::launch_append(p, tbl, cache->D, interleaved != 0, reinterpret_cast<cudaStream_t>(stream)));
}

int paged_reserve(int *page_table, long long table_stride, int *kv_lens, int *page_refs, const int *n_new, int *status,
                  int B, int max_pages, int n_pages, int page_size, attn_stream_t stream) {
  return paged_reserve_guarded(page_table, table_stride, kv_lens, page_refs, n_new, status, nullptr, B, max_pages,
                               n_pages, page_size, stream);
}

int paged_reserve_guarded(int *page_table, long long table_stride, int *kv_lens, int *page_refs, const int *n_new,
                          int *status, int *guard, int B, int max_pages, int n_pages, int page_size,
                          attn_stream_t stream) {
  int st = check_tables(page_table, table_stride, B, max_pages, n_pages);
  if (st == ATTN_OK) st = check_page_size(page_size, max_pages);
  if (st != ATTN_OK) return st;
  if (B == 0) return ATTN_OK;
  if (!kv_lens || !page_refs || !n_new || !status || !aligned(kv_lens, 4) || !aligned(page_refs, 4) ||
      !aligned(n_new, 4) || !aligned(status, 4) || !aligned(guard, 4))
    return ATTN_ERR_INVALID_ARG;
  const seqattn::PageTables t{page_table, table_stride, kv_lens, page_refs, B, max_pages, n_pages, log2_of(page_size)};
  return done(seqattn::launch_reserve(t, n_new, status, guard, reinterpret_cast<cudaStream_t>(stream)));
}

int paged_free(int *page_table, long long table_stride, int *kv_lens, int *page_refs, const int *rows, int n, int B,
               int max_pages, int n_pages, attn_stream_t stream) {
  const int st = check_tables(page_table, table_stride, B, max_pages, n_pages);
  if (st != ATTN_OK) return st;
  if (n < 0 || (n > 0 && !rows)) return ATTN_ERR_INVALID_ARG;
  if (n == 0) return ATTN_OK;
  if (!kv_lens || !page_refs || !aligned(kv_lens, 4) || !aligned(page_refs, 4)) return ATTN_ERR_INVALID_ARG;
  bool seen[seqattn::kPagedMaxRows] = {};
  for (int i = 0; i < n; ++i) {
    if (rows[i] < 0 || rows[i] >= B || seen[rows[i]]) return ATTN_ERR_INVALID_ARG;
    seen[rows[i]] = true;
  }
  const seqattn::PageTables t{page_table, table_stride, kv_lens, page_refs, B, max_pages, n_pages, 0};
  for (int first = 0; first < n; first += seqattn::kPageListMax) {
    seqattn::PageList list{};
    list.n = n - first < seqattn::kPageListMax ? n - first : seqattn::kPageListMax;
    for (int i = 0; i < list.n; ++i) list.a[i] = rows[first + i];
    const cudaError_t e = seqattn::launch_free(t, list, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return keep_cuda_error(e);
  }
  return ATTN_OK;
}

int paged_fork(const paged_pool *pools, int n_pools, int *page_table, long long table_stride, int *kv_lens,
               int *page_refs, const int *src, const int *dst, int *status, int n, int B, int max_pages, int n_pages,
               int page_size, attn_stream_t stream) {
  int st = check_tables(page_table, table_stride, B, max_pages, n_pages);
  if (st == ATTN_OK) st = check_page_size(page_size, max_pages);
  if (st != ATTN_OK) return st;
  seqattn::PoolList list{};
  st = make_pools(&list, pools, n_pools, n_pages);
  if (st != ATTN_OK) return st;
  if (n < 0 || (n > 0 && (!src || !dst))) return ATTN_ERR_INVALID_ARG;
  if (n == 0) return ATTN_OK;
  if (!kv_lens || !page_refs || !status || !aligned(kv_lens, 4) || !aligned(page_refs, 4) || !aligned(status, 4))
    return ATTN_ERR_INVALID_ARG;
  bool target[seqattn::kPagedMaxRows] = {};
  for (int i = 0; i < n; ++i) {
    if (src[i] < 0 || src[i] >= B || dst[i] < 0 || dst[i] >= B || target[dst[i]]) return ATTN_ERR_INVALID_ARG;
    target[dst[i]] = true;
  }
  for (int i = 0; i < n; ++i)
    if (target[src[i]]) return ATTN_ERR_INVALID_ARG;
  const seqattn::PageTables t{page_table, table_stride, kv_lens, page_refs, B, max_pages, n_pages, log2_of(page_size)};
  for (int first = 0; first < n; first += seqattn::kPageListMax) {
    seqattn::PageList pairs{};
    pairs.n = n - first < seqattn::kPageListMax ? n - first : seqattn::kPageListMax;
    for (int i = 0; i < pairs.n; ++i) {
      pairs.a[i] = src[first + i];
      pairs.b[i] = dst[first + i];
    }
    const cudaError_t e = seqattn::launch_fork(t, list, pairs, status + first, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return keep_cuda_error(e);
  }
  return ATTN_OK;
}

int paged_copy(const paged_pool *pools, int n_pools, const int *src, const int *dst, int n, int n_pages,
               attn_stream_t stream) {
  if (n < 0 || n_pages <= 0 || (n > 0 && (!src || !dst))) return ATTN_ERR_INVALID_ARG;
  seqattn::PoolList list{};
  const int st = make_pools(&list, pools, n_pools, n_pages);
  if (st != ATTN_OK) return st;
  for (int i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= n_pages || dst[i] < 0 || dst[i] >= n_pages) return ATTN_ERR_INVALID_ARG;
  // no page twice as a target, none both a source and a target: marked in a
  // bitmap of the launch's pages, a window of it at a time
  constexpr int kWindow = 1 << 15;
  unsigned char mark[kWindow];
  int lo = n_pages, hi = -1;
  for (int i = 0; i < n; ++i) {
    lo = dst[i] < lo ? dst[i] : lo;
    hi = dst[i] > hi ? dst[i] : hi;
  }
  for (long long w = lo; w <= hi; w += kWindow) {
    for (int i = 0; i < kWindow; ++i) mark[i] = 0;
    for (int i = 0; i < n; ++i)
      if (dst[i] >= w && dst[i] < w + kWindow) {
        if (mark[dst[i] - w]) return ATTN_ERR_INVALID_ARG;
        mark[dst[i] - w] = 1;
      }
    for (int i = 0; i < n; ++i)
      if (src[i] >= w && src[i] < w + kWindow && mark[src[i] - w]) return ATTN_ERR_INVALID_ARG;
  }
  if (n == 0 || list.total_layers == 0) return ATTN_OK;
  for (int first = 0; first < n; first += seqattn::kPageListMax) {
    seqattn::PageList pairs{};
    pairs.n = n - first < seqattn::kPageListMax ? n - first : seqattn::kPageListMax;
    for (int i = 0; i < pairs.n; ++i) {
      pairs.a[i] = src[first + i];
      pairs.b[i] = dst[first + i];
    }
    const cudaError_t e = seqattn::launch_copy(list, pairs, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return keep_cuda_error(e);
  }
  return ATTN_OK;
}

size_t paged_compact_workspace_bytes(int n_pages) {
  return n_pages <= 0 || n_pages > (1 << 28) ? 0 : round256(seqattn::compact_workspace_ints(n_pages) * sizeof(int));
}

int paged_compact(const paged_pool *pools, int n_pools, const int *page_table, int *out_table, long long table_stride,
                  const int *page_refs, int *out_refs, int *n_live, void *workspace, size_t workspace_bytes, int B,
                  int max_pages, int n_pages, attn_stream_t stream) {
  int st = check_tables(page_table, table_stride, B, max_pages, n_pages);
  if (st != ATTN_OK) return st;
  seqattn::PoolList list{};
  st = make_pools(&list, pools, n_pools, n_pages);
  if (st != ATTN_OK) return st;
  if (B > 0 && max_pages > 0 && (!out_table || !aligned(out_table, 4))) return ATTN_ERR_INVALID_ARG;
  if (!page_refs || !out_refs || !n_live || !aligned(page_refs, 4) || !aligned(out_refs, 4) || !aligned(n_live, 4))
    return ATTN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < paged_compact_workspace_bytes(n_pages))
    return ATTN_ERR_INVALID_ARG;
  return done(seqattn::launch_compact(list, page_table, out_table, table_stride, page_refs, out_refs, n_live,
                                      static_cast<int *>(workspace), B, max_pages, n_pages,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
