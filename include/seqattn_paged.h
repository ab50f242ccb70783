/*
 * seqattn, serving side -- attention over a paged K/V cache, rotary positions
 * with several axes, appending new tokens to the cache, and the management of
 * its pages, for GB300 (sm_103a). Part of libseqattn.so; the conventions of
 * seqattn.h (layout, GQA, scale, lse, ownership, errors, asynchrony) hold here
 * too, except where an entry point says otherwise.
 *
 * The cache
 *   Pools      K and V live in pages: bf16 [n_pages, Hkv, page_size, D], each
 *              page contiguous, pages page_stride elements apart (a layer of a
 *              larger allocation is a valid pool). page_size is a power of two
 *              from 16 on.
 *   Table      page_table[b * table_stride + i], int32 on the device, is the
 *              page with the keys i*page_size .. of sequence b. An entry outside
 *              [0, n_pages) is no page: its keys are not there (attention does
 *              not see them, an append to it is dropped).
 *   Lengths    kv_lens[b], int32 on the device: keys of sequence b, the new
 *              tokens of the call included. Taken as 0 if negative and as
 *              max_pages*page_size if larger. Slots at or past kv_lens[b] are
 *              never read as numbers: they may hold anything.
 *   New tokens are packed without padding: sequence b has rows cu_seqlens[b] ..
 *              cu_seqlens[b + 1] (int32 [B + 1] on the device, non-decreasing),
 *              the last of its kv_lens[b] keys. Rows at or past cu_seqlens[B]
 *              belong to no sequence and are left as they are. Entries outside
 *              [0, total] are clamped; if they decrease, results are unspecified
 *              but every access stays inside the tensors.
 * The kernels are launched as programmatic dependents of what is before them on
 * the stream and wait for it before they touch memory.
 * Everything that changes from step to step is read on the device, so a call
 * can be captured into a graph and replayed on new lengths and tables.
 */
#ifndef SEQATTN_PAGED_H
#define SEQATTN_PAGED_H

#include <stddef.h>

#include "seqattn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  void *k_pages, *v_pages;  /* bf16 pools, 16-byte aligned */
  long long page_stride;    /* elements from one page to the next, a multiple of 8 */
  const int *page_table;    /* device int32 [B, max_pages] */
  long long table_stride;   /* entries from one row of the table to the next */
  const int *kv_lens;       /* device int32 [B] */
  const int *cu_seqlens;    /* device int32 [B + 1] */
  int B, n_pages, page_size, max_pages, Hkv, D;
} paged_cache;

/*
 * attn_paged -- attention of new tokens over the paged cache: row t of
 * sequence b attends the keys j of its sequence, with causal != 0 those with
 * j <= kv_lens[b] - q_len(b) + t (the chunk is the end of its sequence), that
 * have a page. One token per sequence (decoding), whole prompts and any mix.
 *   q         bf16, row t of query head h at q + h*q_head_stride + t*q_row_stride
 *   o         bf16, likewise with its own strides (output)
 *   lse       fp32 [Hq, total_q] (output), natural logarithm; may be NULL
 *   workspace 16-byte aligned device memory of attn_paged_workspace_bytes(...)
 *             bytes; no other call may use it at the same time
 * Strides are in elements and multiples of 8. Rows that see no key: O = 0,
 * lse = -inf. Keys and values
 * inside kv_lens must be finite (a row with a NaN score comes out as NaN). Scores, sums and
 * accumulators are fp32; the exponentials are rounded to bf16 for the product with V, as in
 * attn_fwd, and summed before that. D 64 or 128, Hq / Hkv at
 * most 128, B at most 4096, max_pages * page_size at most 2^30, and at most
 * 2^31 tiles of 128 keys over all row blocks of 256 rows (else
 * ATTN_ERR_UNSUPPORTED). Two kernels: the attention itself, its key tiles
 * dealt evenly over the SMs whatever the lengths, and the merge of the rows
 * whose keys were split. The result does not depend on timing: the split is a
 * function of the lengths alone.
 */
int attn_paged(const void *q, long long q_head_stride, long long q_row_stride, const paged_cache *cache,
               void *o, long long o_head_stride, long long o_row_stride, float *lse, void *workspace,
               size_t workspace_bytes, int Hq, int total_q, int causal, float scale, attn_stream_t stream);

/* Workspace of attn_paged for these sizes, or 0 for sizes it refuses. */
size_t attn_paged_workspace_bytes(int Hq, int Hkv, int total_q, int D);

/* Rows of one tensor: element d of head h, row s of batch entry b at
 * in + b*in_b + h*in_h + s*in_s + d, its result at out + b*out_b + ... (strides
 * in elements, multiples of 16 bytes; out may be in). */
typedef struct {
  const void *in;
  void *out;
  long long in_b, in_h, in_s, out_b, out_h, out_s;
  int heads;
} rope_rows;

/*
 * rope_axes -- rotary positions with several axes (text: one; images: height
 * and width; video: time, height and width). Pair i of a row, i < D / 2, is
 * turned by positions[axes[i]] * inv_freq[i]:
 *   y1 = x1 cos - x2 sin,  y2 = x1 sin + x2 cos,
 * (x1, x2) = elements (i, i + D/2), or (2i, 2i + 1) with interleaved != 0.
 * inverse != 0 turns back: the gradient of the forward.
 *   q, k       rows to turn, dtype ATTN_BF16 or ATTN_F32; either may be NULL
 *   positions  device int32: axis a, batch entry b, row s at
 *              positions[a*pos_axis + b*pos_b + s] (pos_b = 0: shared)
 *   inv_freq, axes   host arrays of D / 2: radians per position, and the axis
 *              of each pair, 0 <= axis < n_axes, or -1 for a pair that is copied
 * The angle is reduced exactly (64-bit fixed point turns), so positions up to
 * 2^31 keep full precision. D 64 or 128 (else ATTN_ERR_UNSUPPORTED).
 */
int rope_axes(const rope_rows *q, const rope_rows *k, const int *positions, long long pos_axis,
              long long pos_b, int n_axes, const double *inv_freq, const int *axes, int B, int S, int D,
              int dtype, int interleaved, int inverse, attn_stream_t stream);

/*
 * paged_append -- writes new tokens' keys and values into their slots of the
 * cache, turning q and k by their positions on the way (rope_axes): token t of
 * sequence b goes to slot kv_lens[b] - q_len(b) + t. Tokens whose slot is
 * negative, past the table or on no page are dropped (their q is still
 * turned).
 *   q          rows to turn, or NULL; k, v: new tokens ("out" of k and v is not
 *              used; in_b, out_b are not used: rows are packed)
 *   positions  device int32 [n_axes] rows pos_axis apart of total tokens, or
 *              NULL: nothing is turned (then q must be NULL)
 */
int paged_append(const rope_rows *q, const rope_rows *k, const rope_rows *v, const paged_cache *cache,
                 const int *positions, long long pos_axis, int n_axes, const double *inv_freq,
                 const int *axes, int total, int interleaved, attn_stream_t stream);

/*
 * Page management. page_refs, int32 [n_pages] on the device, counts the table
 * entries that hold each page; a page with 0 is free. New pages are always the
 * lowest free ones, handed out in the order of the rows that need them.
 * kv_lens and the entries of the table change through these calls only: a
 * row's entries behind its length are -1 (pages behind a length that the caller
 * lowered would never be free again: there is no call that gives single tokens
 * back). Entries in front may be set to -1 (evicted) by the caller, who then counts
 * their references down; in an evicted page that is partly filled, tokens appended
 * later have no place either.
 * status (int32 per row or pair, device, output): 0 done, PAGED_NO_PAGES, or
 * the reason given below; a row or pair that is not done is left unchanged.
 * All rows of one call belong to one table; calls that change the same table
 * must be ordered on one stream.
 */
#define PAGED_NO_PAGES 1  /* not enough free pages */
#define PAGED_TOO_LONG 2  /* the row's table has no room */
#define PAGED_IN_USE 3    /* the fork's target row holds tokens */

/*
 * A step after a refused request. Append and attention place a sequence's new
 * tokens by counting back from kv_lens, which a refused request does not move: they
 * would lie over keys that the row has already, in pages that it may share. Either
 * leave the rows whose status is not 0 out of cu_seqlens (their ranges empty), or
 * give the step's calls a guard: device int32 [4][B], zeros at first, written by
 * these two calls only. Then the append drops the new tokens of a row that was
 * refused room since its last append if they would lie over keys from before its
 * requests (their q is still turned), and leaves in guard[3 B + b] the lengths to
 * give the attention as kv_lens: 0 for such a row, whose tokens then see no key (O =
 * 0, lse = -inf), else kv_lens[b]; of rows without new tokens, anything. A row that
 * was granted one request and refused another may still bring the tokens that it was
 * granted. With guard NULL these are the plain calls.
 */
int paged_reserve_guarded(int *page_table, long long table_stride, int *kv_lens, int *page_refs, const int *n_new,
                          int *status, int *guard, int B, int max_pages, int n_pages, int page_size,
                          attn_stream_t stream);
int paged_append_guarded(const rope_rows *q, const rope_rows *k, const rope_rows *v, const paged_cache *cache,
                         const int *positions, long long pos_axis, int n_axes, const double *inv_freq, const int *axes,
                         int total, int interleaved, int *guard, attn_stream_t stream);

/* A pool whose pages paged_fork, paged_copy and paged_compact move: n_layers
 * pools at layer_stride, pages page_stride apart, page_bytes each (all in bytes,
 * multiples of 16, base 16-byte aligned). */
typedef struct {
  void *base;
  long long layer_stride, page_stride, page_bytes;
  int n_layers;
} paged_pool;

#define PAGED_MAX_POOLS 32

/* Room for n_new[b] more tokens (device int32 [B], negative counts as 0) in
 * every row: pages are added to the table and kv_lens grows by n_new[b]. Rows are
 * served in order while the free pages last: behind one that gets PAGED_NO_PAGES
 * every row that needs a page gets it too, even if it needs fewer. B at most 4096. */
int paged_reserve(int *page_table, long long table_stride, int *kv_lens, int *page_refs, const int *n_new,
                  int *status, int B, int max_pages, int n_pages, int page_size, attn_stream_t stream);

/* Rows rows[0..n) (host array, distinct) give up their pages: references
 * counted down, entries set to -1, kv_lens to 0. */
int paged_free(int *page_table, long long table_stride, int *kv_lens, int *page_refs, const int *rows, int n,
               int B, int max_pages, int n_pages, attn_stream_t stream);

/* Row dst[i] becomes a copy of row src[i] (host arrays; dst distinct, none of
 * them in src; src may repeat): whole pages are shared, a partly filled last
 * page is copied to a page of its own in every pool, so that both rows can
 * grow (an evicted one stays evicted in both). A dst row must be empty (kv_lens
 * 0), else PAGED_IN_USE. */
int paged_fork(const paged_pool *pools, int n_pools, int *page_table, long long table_stride, int *kv_lens,
               int *page_refs, const int *src, const int *dst, int *status, int n, int B, int max_pages,
               int n_pages, int page_size, attn_stream_t stream);

/* Page dst[i] = page src[i] in every pool (host arrays; dst distinct and none
 * of them in src, all in [0, n_pages)). */
int paged_copy(const paged_pool *pools, int n_pools, const int *src, const int *dst, int n, int n_pages,
               attn_stream_t stream);

/* Moves the live pages with the highest ids into the lowest free ones, in
 * ascending order of both, until pages 0 .. n_live - 1 are the live ones; table
 * and references follow (out_table / out_refs may be the inputs; out_table has
 * the input's stride). What the left pages hold is unspecified.
 *   n_live     device int32 [1] (output)
 *   workspace  paged_compact_workspace_bytes(n_pages) bytes, 16-byte aligned */
int paged_compact(const paged_pool *pools, int n_pools, const int *page_table, int *out_table,
                  long long table_stride, const int *page_refs, int *out_refs, int *n_live, void *workspace,
                  size_t workspace_bytes, int B, int max_pages, int n_pages, attn_stream_t stream);
size_t paged_compact_workspace_bytes(int n_pages);

#ifdef __cplusplus
}
#endif
#endif /* SEQATTN_PAGED_H */
