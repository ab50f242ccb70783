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

/*
 * The 8-bit cache. Pools of e4m3 codes [n_pages, Hkv, page_size, D] (page_stride a
 * multiple of 16) and, for each key and value of each head, a scale that is a power
 * of two: biased exponents (the type e8m0: 2^(byte - 127), 1 <= byte <= 254) in
 * [n_pages, Hkv, page_size], pages page_stride bytes apart, K and V alike. An element
 * is code * scale, which bf16 holds exactly (if not below its smallest number).
 * Everything said of the bf16 cache holds for it: table, lengths, missing pages,
 * what slots past a length may hold (scales too). Pages of codes and of scales are
 * moved by paged_fork, paged_copy, paged_compact and paged_keep as pools like others.
 */
typedef struct {
  unsigned char *k, *v;
  long long page_stride; /* bytes from one page to the next */
} paged_scales;

/*
 * paged_append_e4m3 -- paged_append_guarded to an 8-bit cache: the turned keys and the
 * values are rounded once, from fp32, to code * scale with the least scale whose
 * largest number 448 scale reaches the row's largest size (2^-126 at the least, as
 * for a row of zeros). q is turned and written in bf16. A NaN becomes the NaN
 * code and does not count for the scale. An infinity becomes 448 2^120 with its sign, which
 * no bf16 or fp32 number reaches: paged_read gives an infinity back, as it does for sizes of
 * 248 2^120 (3.3e38) and more; of the rest of such a row only what the scale 2^120 leaves is kept
 * (a bf16 cache keeps it all), and attention must not see the row (its scores are finite, but mean nothing).
 */
int paged_append_e4m3(const rope_rows *q, const rope_rows *k, const rope_rows *v, const paged_cache *cache,
                      const paged_scales *scales, const int *positions, long long pos_axis, int n_axes,
                      const double *inv_freq, const int *axes, int total, int interleaved, int *guard,
                      attn_stream_t stream);

/*
 * paged_read -- keys and values out of the cache, dense: row t of sequence b, for
 * cache->cu_seqlens[b] <= t < cache->cu_seqlens[b + 1], is its key first[b] + t -
 * cu_seqlens[b]. Keys that are not there (past kv_lens[b], before 0, on no page)
 * come out as zeros; rows of no sequence are left as they are.
 *   scales  of an 8-bit cache, or NULL: a bf16 one
 *   first   device int32 [B], or NULL: 0
 *   k, v    bf16 (output): row t of head h at k + h*k_head_stride + t*k_row_stride,
 *           likewise v; strides in elements, multiples of 8, at least D
 *   total   rows of k and v
 */
int paged_read(const paged_cache *cache, const paged_scales *scales, const int *first, void *k, long long k_head_stride,
               long long k_row_stride, void *v, long long v_head_stride, long long v_row_stride, int total,
               attn_stream_t stream);

/*
 * Drafts. The new tokens of a sequence may be a tree: token t follows its parent, an
 * earlier one of the sequence's new tokens, or (parent negative, or not an earlier
 * one) the cached keys. A tree has at most 64 * words tokens, 1 <= words <=
 * DRAFT_MAX_WORDS; a sequence that brings more is none: its tokens follow each other,
 * as in a call without trees (a piece of a prompt beside the drafts of others).
 */
#define DRAFT_MAX_WORDS 4

/*
 * draft_tree -- masks and depths from parents (device int32 [total], numbers
 * within the sequence): bit i of the `words` 64-bit words masks[t*words ..]
 * is set for the ancestors of token t and itself; depths[t] (int32) counts its
 * ancestors, so its position is kv_lens[b] - q_len(b) + depths[t]. Of a sequence
 * of more than 64 * words tokens the masks are 0, the depths 0, 1, 2, ... Rows of no
 * sequence are left as they are.
 */
int draft_tree(const int *parents, const int *cu_seqlens, long long *masks, int *depths, int B, int total, int words,
               attn_stream_t stream);

/*
 * attn_paged_tree, attn_paged_e4m3 -- attn_paged (causal) for drafts, over a bf16 and
 * over an 8-bit cache: token t of a sequence of at most 64 * tree_words new tokens
 * sees its sequence's cached keys j < kv_lens[b] - q_len(b) and those of the new tokens
 * whose bits are set in tree[t*tree_words ..] (bits from q_len(b) on are not looked
 * at). Tokens of longer sequences see what they see in attn_paged. In
 * attn_paged_e4m3 tree may be NULL (tree_words 0), and causal is as in attn_paged
 * then. Workspace: attn_paged_workspace_bytes. Queries are bf16 in both.
 * Over the 8-bit cache, weights of sequences of at most 64 rows (new tokens times
 * Hq / Hkv) are rounded to 2^-9 of themselves for the product with V, if they and their value's
 * scale multiply to 2^-23 of the row's largest such product or more; below that, to steps of
 * 2^-31 of it (2^-44 of the largest scale that a row sees counts as the least scale there).
 * Weights of longer sequences are rounded to 2^-11 of themselves or to 2^-18 of the weights of
 * their 128 keys together (keys 128 i on; or 2^-70 of all), what is more. Values there are exact
 * down to scales of 2^-17 of the largest of these keys, held to 2^-27 of that down to 2^-26 (and to
 * 2^-60 of the largest of all), and may count as zeros below; keys down to 2^-22, 2^-32, 2^-31.
 */
int attn_paged_tree(const void *q, long long q_head_stride, long long q_row_stride, const paged_cache *cache, void *o,
                    long long o_head_stride, long long o_row_stride, float *lse, void *workspace,
                    size_t workspace_bytes, int Hq, int total_q, const long long *tree, int tree_words, float scale,
                    attn_stream_t stream);
int attn_paged_e4m3(const void *q, long long q_head_stride, long long q_row_stride, const paged_cache *cache,
                    const paged_scales *scales, void *o, long long o_head_stride, long long o_row_stride, float *lse,
                    void *workspace, size_t workspace_bytes, int Hq, int total_q, int causal, const long long *tree,
                    int tree_words, float scale, attn_stream_t stream);

/*
 * draft_accept -- the drafts that the model confirms. tokens[t] is the token that
 * row t brought, choices[t] the one that the model chose behind it (device int32
 * [total]). The first given[b] tokens of sequence b (device int32 [B], clamped to 1 ..
 * q_len; NULL: 1, the token that the step before chose) are kept whatever they are;
 * from the last of them on the path goes to the lowest child whose token is the choice, as
 * long as there is one.
 *   path    int32 [total] (output): the kept tokens' numbers within the sequence,
 *           ascending, in rows cu_seqlens[b] .., then -1
 *   n_keep  int32 [B] (output): how many; 0 for a sequence without new tokens
 *   last    int32 [B] (output): the choice behind the last kept token, or -1
 * Rows of path of no sequence are left as they are.
 *
 * draft_accept follows trees of any size, as they are given. The attention does not: a
 * sequence of more than 64 * tree_words tokens is a chain to it, and what the model chose
 * behind a token of another branch was chosen behind all tokens before it.
 * draft_accept_words takes such a sequence as the chain that it was attended as, whatever
 * its parents: `words` is that of the attention's masks (0: none, as draft_accept).
 */
int draft_accept(const int *parents, const int *cu_seqlens, const int *tokens, const int *choices, const int *given,
                 int *path, int *n_keep, int *last, int B, int total, attn_stream_t stream);
int draft_accept_words(const int *parents, const int *cu_seqlens, const int *tokens, const int *choices, const int *given,
                       int *path, int *n_keep, int *last, int B, int total, int words, attn_stream_t stream);

/*
 * paged_keep -- of the last q_len(b) keys of row b, those of a step's new tokens, only
 * path[cu_seqlens[b] + i], i < n_keep[b], stay (strictly ascending numbers within
 * them): they are moved together in every pool, in their order, behind the older keys,
 * kv_lens[b] shrinks by the others, and pages that hold no key any more are given
 * back. A kept token whose place, old or new, is on no page has none. The pools' pages hold
 * [heads[i]][page_size] slots (heads: host array [n_pools], page_bytes a multiple of
 * heads * page_size). All device memory but pools and heads.
 * status: 0 done; a row that is not done is left unchanged:
 *   PAGED_BAD_PATH  n_keep or path out of order or range, kv_lens past the table or
 *                   below q_len, or a token that would move out of a missing page
 *   PAGED_SHARED    a page that would be written, or that the row would end inside
 *                   of, is another row's too
 *   PAGED_REFUSED   the row was refused room for these tokens (guard, or NULL: that of
 *                   the step's paged_reserve_guarded)
 */
#define PAGED_BAD_PATH 4
#define PAGED_SHARED 5
#define PAGED_REFUSED 6
int paged_keep(const paged_pool *pools, const int *heads, int n_pools, int *page_table, long long table_stride,
               int *kv_lens, int *page_refs, const int *cu_seqlens, const int *path, const int *n_keep, int *status,
               int *guard, int total, int B, int max_pages, int n_pages, int page_size, attn_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SEQATTN_PAGED_H */
