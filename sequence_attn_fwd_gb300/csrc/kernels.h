// Host-side interface between the C-ABI layer (api.cu) and the kernel
// translation units. Not part of the public ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace seqattn {

// Parameters of one attention launch (attn_fwd or attn_partial).
struct AttnParams {
  void *o;            // [B, Hq, Sq, D] bf16 (attn_fwd) or fp32 (attn_partial)
  float *lse;         // [B, Hq, Sq]
  int B, Hq, Hkv, Sq, Skv;
  long long q_off, kv_off;  // global positions of query row 0 and key 0
  float scale_log2;   // softmax scale times log2(e)
  int causal;
  int n_qblocks;      // ceil(Sq / 256): two 128-row query tiles per CTA
  int skip_empty;     // rows that see no key: write lse = -inf only, leave O untouched
  long long o_rows;   // rows per head of O and lse (Sq for a single problem)
  float o_scale;      // e4m3 attention: the V scale applied to O (1 otherwise)
  int heads_per_chunk;  // single problems: items come in chunks of this many consecutive
                        // heads (whole GQA groups), all query blocks of a chunk before the next
};

// One block of attention: the queries in rows [q_row, q_row + Sq) of Q (per
// head) against the keys and values in rows [kv_row, kv_row + Skv) of K / V,
// written to rows [o_row, o_row + Sq) of part `part` of O and lse (O viewed as
// [parts][B * Hq heads][rows][D]). q_pos / kv_pos are the global positions of
// query row 0 and key 0 (the causal mask compares them).
struct BlockDesc {
  long long q_row, kv_row, o_row;
  long long q_pos, kv_pos;
  int Sq, Skv;
  int part;
};

// The blocks of one launch, passed by value in the kernel parameters.
// item_start[i] is the first work item of block i (items: B * Hq heads times
// ceil(Sq / 256) query blocks per block), item_start[n] the total.
constexpr int kMaxLaunchBlocks = 64;
struct BlockTable {
  int n;
  long long item_start[kMaxLaunchBlocks + 1];
  BlockDesc b[kMaxLaunchBlocks];
};

// Blocks that share their query rows (q_row, o_row, q_pos and Sq equal to
// block 0's), such as the key chunks of a ring pass: a work item is 256 of
// those rows of one (batch, head) taken against every block in turn, each
// block a segment of the item with its own partial, Q loaded once.
struct SegTable {
  int n;
  BlockDesc b[kMaxLaunchBlocks];
};

// Number of SMs of the current device (read once per device).
int device_sm_count();

// Tensor maps are 3-D views [heads][rows][D] built by the caller: q, k, v of
// bf16 data, box 64 columns x 128 rows x 1; o of the output type (fp32 when
// f32_out, else bf16), box 128 bytes x 32 rows x 1 (one warp's rows); all with
// 128-byte swizzle.
cudaError_t launch_attention(int D, bool f32_out, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                             const CUtensorMap &tm_v, const CUtensorMap &tm_o, const AttnParams &p,
                             cudaStream_t stream);

// Backward (head dim 64 or 128): gradients of a forward whose O and lse are given.
struct BwdParams {
  const float *lse;    // [B*Hq, S] natural log (the forward's)
  const float *delta;  // [B*Hq, S] workspace: <dO_i, O_i>, written by the first kernel
  void *dq, *dk, *dv;  // bf16 [B*Hq, S, D], [B*Hkv, S, D] x 2
  int B, Hq, Hkv, S;
  float scale;         // softmax scale
  int causal;
};

// delta, then dK / dV (grid: key tiles x B*Hkv), then dQ (grid: query tiles x
// B*Hq); maps over bf16 [heads][S][D], box 64 x 128 x 1, 128-byte swizzle.
cudaError_t launch_attention_bwd(int D, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                                 const CUtensorMap &tm_v, const CUtensorMap &tm_do,
                                 const void *o, const void *dout, float *delta,
                                 const BwdParams &p, cudaStream_t stream);

// e4m3 attention (D = 128, bf16 O): tq / tk over e4m3 [heads][S][128] with
// box 128 x 128 x 1, tvt over V^T e4m3 [kv heads][128][S] with box 128 (keys)
// x 128 x 1, all 128-byte swizzle; p.scale_log2 includes the Q and K scales,
// p.o_scale is the V scale.
cudaError_t launch_attention_fp8(const CUtensorMap &tq, const CUtensorMap &tk,
                                 const CUtensorMap &tvt, const CUtensorMap &to,
                                 const AttnParams &p, cudaStream_t stream);

// The single-SM persistent kernel over a table of blocks (row ranges of the
// maps' row dimension; p's Sq / Skv / q_off / kv_off / n_qblocks are unused).
cudaError_t launch_attention_blocks(int D, bool f32_out, const CUtensorMap &tm_q,
                                    const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                    const CUtensorMap &tm_o, const AttnParams &p,
                                    const BlockTable &tbl, cudaStream_t stream);

// The same kernel over a table of blocks that share their query rows (see
// SegTable; p's Sq / Skv / q_off / kv_off / n_qblocks are unused): fp32
// partials of blocks of at most 2048 keys (anything else is refused with
// cudaErrorInvalidValue).
cudaError_t launch_attention_segments(int D, bool f32_out, const CUtensorMap &tm_q,
                                      const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                      const CUtensorMap &tm_o, const AttnParams &p,
                                      const SegTable &tbl, cudaStream_t stream);

cudaError_t launch_lse_merge(const float *o_parts, const float *lse_parts, int P, long long nrows,
                             int D, void *o, bool bf16_out, float *lse, cudaStream_t stream);

// ---------------------------------------------------------------- paged cache
// The device view of a paged K/V cache (paged_cache of seqattn_paged.h).
struct PagedView {
  void *k_pages, *v_pages;
  long long page_stride;   // elements
  const int *page_table;
  long long table_stride;
  const int *kv_lens;
  const int *cu_seqlens;   // [B + 1] rows of the packed new tokens
  int B, n_pages, page_size, max_pages, Hkv;
};

// What a row's requests for room left for the step that follows them (null: no
// row is guarded). A request that was refused does not move kv_lens, so that the
// step's tokens, counted back from it, would lie over older keys.
//   base   the row's length before its first request after its last append
//   held   its length after the last one, plus 1, if one of them was refused, else 0
//   open   its length after the last one, plus 1, until an append comes, then 0
//   lens   what the attention of the step takes as its length, written by the append
// A length that differs from `open` was changed otherwise (freed, forked): the next
// request is a first one again; and one that differs from `held` is not guarded.
struct RowGuard {
  int *base, *held, *open, *lens;
#ifdef __CUDACC__
  __device__ __forceinline__ RowGuard(int *guard, int B)
      : base(guard), held(guard + B), open(guard + 2 * B), lens(guard + 3 * B) {}
  // Whether q_len new tokens of row b, which has kv_len keys, would lie over older ones.
  __device__ __forceinline__ bool refuses(int b, int kv_len, int q_len) const {
    return held[b] == kv_len + 1 && kv_len - q_len < base[b];
  }
  // After a request for tokens of row b, by one thread: its length before and after.
  __device__ __forceinline__ void request(int b, int len, int after, bool refused) const {
    const bool same = open[b] == len + 1;
    if (!same) base[b] = len;
    held[b] = refused || (same && held[b] != 0) ? after + 1 : 0;
    open[b] = after + 1;
  }
#endif
};

// The scales of an e4m3 cache: powers of two, biased exponents [n_pages][Hkv][page_size].
struct ScaleView {
  unsigned char *k, *v;
  long long page_stride;   // bytes
};
constexpr int kDraftWords = 4;  // 64-bit words of a draft's mask, at most

// Attention of packed new tokens over a paged cache. The rows of a KV head are
// numbered (token, query head of the group), group fastest; a 128-row tile has
// `tok` whole tokens (tok * G <= 128), a work item two tiles.
struct PagedAttnParams {
  PagedView cache;
  void *o;                 // bf16, row t of head h at h * o_h + t * o_s
  long long o_h, o_s;
  float *lse;              // [Hq, total_q] or null
  float *part_o;           // workspace: [2 * kPagedMaxCtas][part_rows][D]
  float *part_lse;         // workspace: [2 * kPagedMaxCtas][part_rows]
  int4 *cuts;              // workspace: [kPagedMaxCtas] the items that the CTAs begin and do not end
  int part_rows;           // rows of a work item that can hold a token
  int Hq, G, tok, total_q, causal;
  int page_log2;           // log2(page_size)
  float scale_log2;
  const unsigned long long *tree;  // [total_q][tree_words] drafts that a row sees, one bit each, or null
  int tree_words;
  ScaleView scales;        // of an e4m3 cache
  const void *q;           // bf16, row t of head h at h * q_h + t * q_s (the e4m3 form reads it without a map)
  long long q_h, q_s;
};
constexpr int kPagedMaxCtas = 160;   // CTAs of one launch (at most one per SM)
constexpr int kPagedMaxSeqs = 4096;  // sequences of one launch (their prefix sums sit in shared memory)
constexpr int kPagedMaxRows = 4096;  // rows of a page table

// Maps: q bf16 4-D [Hkv][total_q][G][D], box 64 x G x tok x 1, and the same with
// boxes of 16 / G, 32 / G, 64 / G tokens (at least one) for calls whose sequences
// have that few rows; k, v bf16 4-D [n_pages][Hkv][page_size][D], box 64 x
// min(page_size, 128) x 1 x 1; 128-byte swizzle. Two kernels: the attention and
// the merge of split rows.
cudaError_t launch_attn_paged(int D, const CUtensorMap &tm_q, const CUtensorMap (&tm_qn)[3], const CUtensorMap &tm_k,
                              const CUtensorMap &tm_v, const PagedAttnParams &p, cudaStream_t stream);
// The same over an e4m3 cache. Maps of bytes: box D x min(page_size, 128) x 1 x 1, swizzled
// over the D bytes of a row (128 or 64).
cudaError_t launch_attn_paged_e4m3(int D, const CUtensorMap &tm_k, const CUtensorMap &tm_v, const PagedAttnParams &p,
                                   cudaStream_t stream);

// ---------------------------------------------------------------- rotary positions, appends
struct RopeView {
  const void *in;
  void *out;
  long long in_b, in_h, in_s, out_b, out_h, out_s;  // elements
  int heads;                                        // 0: nothing
};
// Turns per position of each pair, as a fraction of 2^64, and its axis (-1: not turned).
struct RopeTable {
  uint64_t turns[64];
  signed char axis[64];
};
struct RopeParams {
  RopeView q, k, v;        // v: appends only
  PagedView cache;         // appends only
  ScaleView scales;        // appends to an e4m3 cache only
  int *guard;              // appends only: [4][B] or null, see RowGuard
  const int *positions;    // null: nothing is turned (appends only)
  long long pos_axis, pos_b;
  int B, S, inverse;       // appends: B = 1, S = the packed tokens
};
cudaError_t launch_rope(const RopeParams &p, const RopeTable &tbl, int D, bool f32, bool interleaved,
                        cudaStream_t stream);
cudaError_t launch_append(const RopeParams &p, const RopeTable &tbl, int D, bool e4m3, bool interleaved,
                          cudaStream_t stream);

// Keys and values out of a paged cache: the packed rows of cache.cu_seqlens are
// keys first[b] (0 if null) on of each sequence.
struct ReadParams {
  PagedView cache;
  ScaleView scales;        // of an e4m3 cache
  const int *first;
  void *k, *v;             // bf16, row t of head h at h * .._h + t * .._s
  long long k_h, k_s, v_h, v_s;
  int total;
};
cudaError_t launch_read(const ReadParams &p, int D, bool e4m3, cudaStream_t stream);

// ---------------------------------------------------------------- page management
struct PageTables {
  int *page_table;
  long long table_stride;
  int *kv_lens, *page_refs;
  int B, max_pages, n_pages, page_log2;
};
constexpr int kPageListMax = 512;  // rows, pairs or copies of one launch, passed by value
struct PageList {
  int n;
  int a[kPageListMax], b[kPageListMax];
};
struct PoolView {
  unsigned char *base;
  long long layer_stride, page_stride, page_bytes;
  int n_layers;
};
constexpr int kMaxPools = 32;
struct PoolList {
  int n, total_layers;
  PoolView pool[kMaxPools];
};
cudaError_t launch_reserve(const PageTables &t, const int *n_new, int *status, int *guard, cudaStream_t stream);
cudaError_t launch_free(const PageTables &t, const PageList &rows, cudaStream_t stream);
cudaError_t launch_fork(const PageTables &t, const PoolList &pools, const PageList &pairs, int *status,
                        cudaStream_t stream);
cudaError_t launch_copy(const PoolList &pools, const PageList &pairs, cudaStream_t stream);
cudaError_t launch_compact(const PoolList &pools, const int *page_table, int *out_table, long long table_stride,
                           const int *page_refs, int *out_refs, int *n_live, int *workspace, int B, int max_pages,
                           int n_pages, cudaStream_t stream);

size_t compact_workspace_ints(int n_pages);

// ---------------------------------------------------------------- drafts
cudaError_t launch_draft_tree(const int *parents, const int *cu, long long *masks, int *depths, int B, int total, int words,
                              cudaStream_t stream);
cudaError_t launch_draft_accept(const int *parents, const int *cu, const int *tokens, const int *choices, const int *given,
                                int *path, int *n_keep, int *last, int B, int total, int words, cudaStream_t stream);

// A pool as slots: pages of [heads][page_size] slots of slot_bytes.
struct SlotPool {
  unsigned char *base;
  long long layer_stride, page_stride;
  int slot_bytes, heads;
  int lines;  // n_layers * heads * pieces of a slot (16 bytes, or one where that does not divide it)
};
struct KeepParams {
  PageTables t;
  const int *cu, *path, *n_keep;
  int *status, *guard;     // guard: [4][B] or null, see RowGuard
  int total, n_pools, lines;
  SlotPool pool[kMaxPools];
};
cudaError_t launch_keep(const KeepParams &p, cudaStream_t stream);

// Launches a kernel that may start before the one ahead of it on the stream has
// finished; it calls wait_prerequisites() before it touches memory. Every kernel
// of the serving side is launched so and waits first; all but the merge of the
// attention let the next one start as soon as their own CTAs have: 1.5 to 2.5 us a
// call of a chain.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             Args &&...args) {
  cudaLaunchConfig_t cfg{};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// Shared by the C-ABI files: keeps the error for attn_last_cuda_error() and
// returns ATTN_ERR_CUDA; the driver's tensor-map encoder (null if not found).
int keep_cuda_error(cudaError_t e);
void *tensor_map_encoder();

// One CTA waits on an mbarrier nothing arrives at until timeout_us runs out.
cudaError_t launch_expire_wait(unsigned timeout_us, cudaStream_t stream);

// y[i] = 2^x[i] by the softmax's exponential routine (polynomial or MUFU).
cudaError_t launch_exp2_probe(const float *x, float *y, long long n, bool poly,
                              cudaStream_t stream);

// Reads and clears the device error word (after the caller synchronised).
cudaError_t read_and_clear_device_error(int *code);

}  // namespace seqattn
