/*
 * gdn_block.h -- C ABI of the operators that a hybrid stack puts next to its gated delta-rule layers (GB300,
 * sm_103a): attention of new tokens over a paged key/value cache, rotary positions (alone or behind a norm of each head), the upkeep of the cache's
 * pages, the root-mean-square norm of the residual stream, and a gated linear recurrence with one state per channel.
 *
 * A stack of gated delta-rule layers carries a softmax-attention layer after every few of them (onedev.kr summary
 * of the FlashQLA AICon 2026 talk, background paragraph: hybrids of three linear layers to one softmax layer).
 *
 * Conventions, as in gdn.h unless a function says otherwise
 *  - Tensor pointers are DEVICE pointers.  Shape structs are host structs.  The caller owns all memory; the library
 *    never allocates, and scratch memory is the caller's `workspace`, sized by the *_workspace_size queries.  A
 *    workspace needs no initialisation and keeps nothing between calls.
 *  - Strides are in ELEMENTS; the feature dimension is contiguous.  dtype is GDN_BF16 or GDN_FP32.
 *  - Calls are asynchronous on `stream` and never synchronise the host.  Argument errors are found on the host
 *    before any launch: GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_WORKSPACE; a failed launch returns
 *    GDN_ERR_CUDA; gdn_last_error_string() has the reason.
 *  - Results are deterministic (no floating-point atomics).
 *  - Lengths, page tables and page numbers live on the device, so the host cannot check them.  The kernels read and
 *    write nothing out of range whatever they hold: lengths are cut to the space there is, and a page number outside
 *    the pool is a missing page.
 */
#ifndef GDN_BLOCK_H_
#define GDN_BLOCK_H_

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ paged cache
 * The keys and values of all sequences lie in pages of `page_size` tokens: k_cache, v_cache [num_pages, page_size,
 * Hkv, D] with any strides (a head-major pool is the same with other strides).  Token t of sequence n is slot
 * t % page_size of page page_table[n, t / page_size]; unused table entries are -1.  kv_lens[n] counts the
 * sequence's tokens, the new ones of this call among them.
 */
typedef struct {
  int num_seqs;                /* N                                                            */
  int total_q;                 /* new tokens of all sequences                                  */
  int num_heads, num_kv_heads; /* Hq, Hkv: query head h reads key head h / (Hq / Hkv)          */
  int head_dim;                /* D: 64 or 128 (attention)                                     */
  int page_size;               /* a power of two, 16 .. 4096                                   */
  int num_pages;               /* pages of the pool                                            */
  int max_pages;               /* columns of page_table                                        */
  gdn_dtype dtype;             /* of q, k, v, o and both caches                                */
  int max_q;                   /* attention: longest new length of one sequence if the host    */
                               /* knows it, 0 otherwise; any value gives the same results (it  */
                               /* picks the kernel)                                            */
  int window;                  /* attention: keys a query sees, itself included; 0: no limit   */
  float scale;                 /* attention: logits are scale * q . k                          */
  int64_t table_stride;        /* of page_table rows; 0: one row for all sequences (read only)  */
  int64_t q_tok, q_head;       /* strides of q: token, head                                    */
  int64_t k_page, k_tok, k_head; /* strides of k_cache: page, slot, head                       */
  int64_t v_page, v_tok, v_head; /* strides of v_cache                                         */
  int64_t o_tok, o_head;       /* strides of o (attention) or q_out (append)                   */
  int64_t kn_tok, kn_head;     /* append: strides of the new keys                              */
  int64_t vn_tok, vn_head;     /* append: strides of the new values                            */
  int rot;                     /* append: leading features of q and k that turn, even, <= D    */
  int interleaved;             /* append: pairs (2i, 2i + 1) instead of (i, i + rot / 2)       */
  int table_rows;              /* append: positions of the rotary table                        */
  int reserved;                /* must be 0; attention: or GDN_DEBUG_WAIT_TIMEOUT              */
} gdn_paged_shape;

/*
 * Attention of new tokens over the cache (causal).  The new tokens of sequence n are rows cu_q[n] .. cu_q[n+1]-1 of
 * q [total_q, Hq, D] (cu_q device int32 [N+1], not decreasing; NULL: every sequence has total_q / N of them; rows that no
 * sequence names, and a batch whose cu_q goes back and names tokens many times, may be left without an output).  Query i of a
 * sequence with `ql` new tokens sits at position p = kv_lens[n] - ql + i and sees the keys at positions
 * max(0, p - window + 1) .. p, whose own keys and values the cache must hold already:
 *
 *     o = sum_j exp(s_j - lse) v_j,   s_j = scale q . k_j,   lse = log sum_j exp(s_j).
 *
 * A query that sees no key (p < 0, or an empty sequence) gets o = 0, lse = -inf.  lse fp32 [total_q, Hq], contiguous,
 * or NULL.  Slots outside what the queries see may hold anything, NaN included; a key that only some of the queries
 * computed together see (16, 32 or 256 (query, head) rows) must have a finite value vector.  A missing page counts as
 * keys and values of zero.
 * bf16: products in bf16 with fp32 sums, the weights rounded to bf16 before the second product.  fp32: products in
 * three TF32 parts each, about 2^-21 relative (less where a part of a factor is below 2^-126); a NaN or an infinity
 * reaches what it should (an infinity times a factor beyond 2^11 may come out as NaN).  q, k_cache, v_cache, o:
 * 16-byte aligned with strides of whole 16 bytes, those of the caches positive and below 2^37; at most 65535 query heads
 * per key head.  o and lse share no memory with the inputs.  workspace: 32-byte aligned (GDN_ERR_INVALID_ARG otherwise).
 */
size_t gdn_paged_attn_workspace_size(const gdn_paged_shape *shape);
int gdn_paged_attn_fwd(const gdn_paged_shape *shape, const void *q, const void *k_cache, const void *v_cache,
                       const int32_t *page_table, const int32_t *cu_q /* nullable */, const int32_t *kv_lens, void *o,
                       float *lse /* nullable */, void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/* The status word of the last gdn_paged_attn_fwd with this shape and workspace (synchronises the stream): 0, or 4 when a
 * bounded device wait ran past its limit (that call's outputs are not reliable; gdn_device_status_code maps it), or -1 on
 * an error.  workspace: the whole one that the call was given, at least gdn_paged_attn_workspace_size bytes.  With
 * GDN_DEBUG_WAIT_TIMEOUT in `reserved` (a test hook) a call only waits, with a short limit, for a barrier that nothing
 * arrives at, sets the status and returns without writing its outputs. */
int gdn_paged_attn_status(const gdn_paged_shape *shape, const void *workspace, gdn_stream_t stream);

/* gdn_paged_attn_fwd of a window whose sequences' first `sinks` keys stay visible: the query at position p sees the keys j <= p
 * with j > p - window or j < sinks.  Without a window (0, or one as long as a table row) they add nothing.  The same
 * workspace and status. */
int gdn_paged_attn_sinks_fwd(const gdn_paged_shape *shape, int sinks, const void *q, const void *k_cache, const void *v_cache,
                             const int32_t *page_table, const int32_t *cu_q /* nullable */, const int32_t *kv_lens, void *o,
                             float *lse /* nullable */, void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * gdn_paged_attn_fwd of groups of sequences that share a prefix (branches that gdn_pages_fork made, or requests behind one
 * system prompt), whose keys are read once for a group.  Group g is the sequences cu_seqs[g] .. cu_seqs[g+1]-1 (device int32
 * [groups + 1], not decreasing; NULL: num_seqs / groups each; sequences that no group names have no prefix).  The first
 * prefix_lens[g] tokens (device int32 [groups]) of all its sequences that have new tokens are the same: the rows of page_table
 * name the same pages there, and those of the first such sequence are read.  A prefix longer than what some sequence of the
 * group had cached before its new tokens is cut to that, so any value gives right results where the pages are the same.
 * Sequences without new tokens (branches that have ended among them) limit nothing, and their rows are not read.
 * The new tokens of a group's sequences follow one another in q (cu_q as in gdn_paged_attn_fwd; one that goes back leaves rows
 * without an output).  window must be 0.  max_group: most new tokens of a group if the host knows, 0 otherwise (picks the
 * kernel).  Batches in which sharing saves too little are computed as gdn_paged_attn_fwd does, from each sequence's own row:
 * those whose table rows (max_pages, not the lengths, which the host does not know) have room for little, so a table no wider
 * than need be makes small batches faster; and those with many new tokens to a sequence, which are bound by products.
 */
size_t gdn_prefix_attn_workspace_size(const gdn_paged_shape *shape, int groups, int max_group);
int gdn_prefix_attn_fwd(const gdn_paged_shape *shape, int groups, int max_group, const void *q, const void *k_cache,
                        const void *v_cache, const int32_t *page_table, const int32_t *cu_q /* nullable */,
                        const int32_t *kv_lens, const int32_t *cu_seqs /* nullable */, const int32_t *prefix_lens, void *o,
                        float *lse /* nullable */, void *workspace, size_t workspace_bytes, gdn_stream_t stream);
/* gdn_paged_attn_status of the last gdn_prefix_attn_fwd with these arguments. */
int gdn_prefix_attn_status(const gdn_paged_shape *shape, int groups, int max_group, const void *workspace, gdn_stream_t stream);

/* ------------------------------------------------------------------ rotary positions
 * The pair (a, b) of features at a position turns by the position's angle of that pair:
 *     (a, b) -> (a cos - b sin, b cos + a sin).
 * Pairs are (i, i + rot/2), or (2i, 2i+1) when interleaved, over the first `rot` features of a head; the others pass.
 * The angles come as a table, fp32 [rows, rot/2, 2] of (cos, sin), built once: row p, pair i holds
 * amplitude * (cos, sin)(p * freq[i]).
 */

/* Fills a table: freq fp64 [pairs] on the device (angle per position of each pair, in radians).  Angles and their
 * cos and sin are formed in fp64 and rounded once, so far positions keep their accuracy. */
int gdn_rotary_table(const double *freq, int pairs, int rows, double amplitude, float *table, gdn_stream_t stream);

typedef struct {
  int tokens;              /* T                                                          */
  int q_heads, k_heads;    /* heads of q and k; either may be 0 (its pointers NULL)      */
  int head_dim;            /* D >= 2                                                     */
  int rot;                 /* even, 2 <= rot <= D                                        */
  int interleaved;         /* 0 or 1                                                     */
  int inverse;             /* 1: turn by the opposite angle, which is the gradient of    */
                           /* the turn, and undoes it where the amplitude is 1           */
  int table_rows;
  gdn_dtype dtype;
  int reserved;            /* must be 0                                                  */
  int64_t q_tok, q_head, k_tok, k_head;     /* strides of the inputs                     */
  int64_t qo_tok, qo_head, ko_tok, ko_head; /* strides of the outputs                    */
} gdn_rotary_shape;

/* Turns q [T, q_heads, D] and k [T, k_heads, D] into q_out and k_out (which may be q and k themselves, with their
 * strides).  positions int32 [T]; a position outside the table leaves its token unturned. */
int gdn_rotary(const gdn_rotary_shape *shape, const void *q, const void *k, const float *table,
               const int32_t *positions, void *q_out, void *k_out, gdn_stream_t stream);

/* Rotary positions of new tokens and their write into a paged cache: token i of the `ql` new ones of sequence n has
 * position kv_lens[n] - ql + i; its query turns into q_out, its key turns into the cache's slot of that position, its
 * value goes there as it is.  q, k, v [total_q, heads, D] (Hq, Hkv, Hkv); cu_q as in gdn_paged_attn_fwd.  A token
 * whose position is below 0, past the page table or on a missing page is not written to the cache; one outside the
 * rotary table is not turned. */
int gdn_rotary_append(const gdn_paged_shape *shape, const void *q, const void *k, const void *v, const float *table,
                      void *k_cache, void *v_cache, const int32_t *page_table, const int32_t *cu_q /* nullable */,
                      const int32_t *kv_lens, void *q_out, gdn_stream_t stream);

/* ------------------------------------------------------------------ norm of heads with rotary positions
 * The root-mean-square norm of every head of q and k, and its turn, in one pass (y and all between in fp32, rounded once):
 *     r = 1 / sqrt(mean(x^2) + eps),   y = turn(x r (weight + weight_offset))
 * over the features of a head; turn, table and positions as in gdn_rotary (inverse must be 0); weights fp32 [D], one for
 * the heads of q and one for those of k.  head_dim at most 1024.  q_out and k_out may be q and k themselves, with
 * their strides. */
int gdn_norm_rotary(const gdn_rotary_shape *shape, float eps, float weight_offset, const void *q, const void *k,
                    const float *q_weight, const float *k_weight, const float *table, const int32_t *positions, void *q_out,
                    void *k_out, gdn_stream_t stream);

/* Gradients, given dq_out and dk_out (strides qo_*, ko_* of the shape) and the inputs q and k (q_*, k_*): dq [T, q_heads, D] and
 * dk [T, k_heads, D], contiguous, and dq_weight, dk_weight fp32 [D] (summed in a fixed order).  With u the turned-back gradient
 * and xhat = x r: dx = r (u w - xhat mean(u w xhat)), w = weight + weight_offset, dw = sum of u xhat. */
size_t gdn_norm_rotary_bwd_workspace_size(const gdn_rotary_shape *shape);
int gdn_norm_rotary_bwd(const gdn_rotary_shape *shape, float eps, float weight_offset, const void *dq_out, const void *dk_out,
                        const void *q, const void *k, const float *q_weight, const float *k_weight, const float *table,
                        const int32_t *positions, void *dq, void *dk, float *dq_weight, float *dk_weight, void *workspace,
                        size_t workspace_bytes, gdn_stream_t stream);

/* gdn_rotary_append with the heads of q and k normed before they turn. */
int gdn_norm_rotary_append(const gdn_paged_shape *shape, float eps, float weight_offset, const void *q, const void *k,
                           const void *v, const float *q_weight, const float *k_weight, const float *table, void *k_cache,
                           void *v_cache, const int32_t *page_table, const int32_t *cu_q /* nullable */,
                           const int32_t *kv_lens, void *q_out, gdn_stream_t stream);

/* ------------------------------------------------------------------ pages
 * Bookkeeping on the device: page_table int32 [num_seqs, max_pages] (-1: none), seq_lens int32 [num_seqs] (tokens),
 * refcount int32 [num_pages] (table entries that name the page; 0: free).  New pages are the free ones of lowest
 * number, given out in the order of the request list.  A page that is not full belongs to one sequence only (fork
 * copies it), so appending never writes into a shared page.
 */
typedef struct {
  int num_seqs, max_pages, num_pages, page_size;
  int64_t table_stride;
  int reserved[2]; /* must be 0 */
} gdn_pages_shape;

/* A device array of equal slots that are copied whole (one layer's keys, or the per-sequence recurrent states):
 * slot i occupies bytes [i * stride, i * stride + bytes).  base 16-byte aligned; stride and bytes multiples of 16. */
typedef struct {
  void *base;
  int64_t stride, bytes;
  int64_t slots; /* gdn_slots_copy leaves out pairs that name a slot outside [0, slots); fork and compact refuse a  */
                 /* pool of fewer slots than pages, and a state pool of fewer than sequences                        */
} gdn_slot_pool;

/* Copies slot src[i] to slot dst[i] in every pool, i < count.  No dst may appear twice or among the src. */
int gdn_slots_copy(const gdn_slot_pool *pools, int num_pools, const int32_t *src, const int32_t *dst, int count,
                   gdn_stream_t stream);

/* Grows sequences: seqs int32 [m] (distinct), add int32 [m] tokens.  ok int32 [m] gets 1, or 0 where the sequence is
 * left as it was: a bad number, no room in its table row (or in 31 bits), a last page that is shared, or not enough free pages (once
 * the list has asked for more pages than there are, that request and the later ones that need pages get none). */
size_t gdn_pages_workspace_size(const gdn_pages_shape *shape, int m);
int gdn_pages_extend(const gdn_pages_shape *shape, int32_t *page_table, int32_t *seq_lens, int32_t *refcount,
                     const int32_t *seqs, const int32_t *add, int m, int32_t *ok, void *workspace,
                     size_t workspace_bytes, gdn_stream_t stream);

/* Branches sequences: children[i] (empty, distinct, no parent of the same call) becomes a copy of parents[i].  Full
 * pages are shared; a partly filled last page is copied to a new page in every pool; slot children[i] of every state
 * pool becomes a copy of slot parents[i].  new_page int32 [m] gets the copied page's number, -1 where none was
 * needed, -2 where the fork was left out (bad numbers, child not empty, no free page). */
int gdn_pages_fork(const gdn_pages_shape *shape, int32_t *page_table, int32_t *seq_lens, int32_t *refcount,
                   const int32_t *parents, const int32_t *children, int m, const gdn_slot_pool *pools, int num_pools,
                   const gdn_slot_pool *states, int num_states, int32_t *new_page, void *workspace,
                   size_t workspace_bytes, gdn_stream_t stream);

/* Ends sequences: their pages lose one reference each, their rows become -1, their lengths 0. */
int gdn_pages_free(const gdn_pages_shape *shape, int32_t *page_table, int32_t *seq_lens, int32_t *refcount,
                   const int32_t *seqs, int m, gdn_stream_t stream);

/* Moves the live pages to the front: with L pages in use, the i-th page in use of number >= L (ascending) moves to the
 * i-th free number below L, in every pool, in the table and in the counts.  The results go to page_table_out (rows of
 * table_stride too) and refcount_out, which may be the inputs themselves; moves int32 [1] gets the number of moved
 * pages, or NULL. */
int gdn_pages_compact(const gdn_pages_shape *shape, const int32_t *page_table, const int32_t *refcount,
                      int32_t *page_table_out, int32_t *refcount_out, const gdn_slot_pool *pools, int num_pools,
                      int32_t *moves /* nullable */, void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/* ------------------------------------------------------------------ root-mean-square norm */
typedef struct {
  int64_t rows;            /* T                                                               */
  int dim;                 /* D, 1 .. 65536                                                   */
  gdn_dtype dtype;         /* x, residual, h; y when it is not 8-bit; dy, dh, dx              */
  int fp8;                 /* 1: y is e4m3 with scales                                        */
  int group;               /* fp8: features per scale, 128 (D a multiple of it) or 0: the row */
  float eps;               /* > 0                                                             */
  float weight_offset;     /* y = h rstd (weight + weight_offset): 0, or 1 for zero-centred   */
  int64_t x_row, r_row, h_row, y_row; /* row strides of x, residual, h, y (backward: h = x_row, dy = y_row, */
                                      /* dh = r_row, dx = h_row)                              */
  int reserved[2];         /* must be 0                                                       */
} gdn_norm_shape;

/* h = x + residual (just x without one), rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd (weight + weight_offset).
 * residual and h_out may be NULL (h_out may be x or residual); rstd fp32 [T] or NULL; weight fp32 [D].  The norm is
 * that of the fp32 sum, before its rounding to h_out.  fp8: scale fp32 [T, D / group] (or [T]) = amax / 448 of the
 * unrounded y, amax not below 1e-30, and y in e4m3 = round(y * (448 / amax)), products and quotients in fp32 (as far from
 * the exact quotient as y / scale in fp32; where that lies next to a tie the two may be an e4m3 step apart). */
int gdn_rmsnorm_fwd(const gdn_norm_shape *shape, const void *x, const void *residual, const float *weight, void *h_out,
                    void *y, float *scale, float *rstd, gdn_stream_t stream);

/* Gradients of h and weight, given dy, the stored h, its rstd, and dh (NULL: zero), the gradient that reaches h along
 * the residual stream: dx = rstd w dy - h rstd^3 <w dy, h> / D + dh (the gradient of x and of residual),
 * dw[i] = sum over rows of dy h rstd (fp32 [D], summed in a fixed order).  dx may be dy or dh. */
size_t gdn_rmsnorm_bwd_workspace_size(const gdn_norm_shape *shape);
int gdn_rmsnorm_bwd(const gdn_norm_shape *shape, const void *dy, const void *h, const float *weight, const float *rstd,
                    const void *dh, void *dx, float *dw, void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/* ------------------------------------------------------------------ gated linear recurrence
 * The elementwise sister of the delta rule: one state per channel, the gate in its logarithm,
 *     h_t = exp(g_t) h_{t-1} + x_t,   y_t = h_t.
 * x, g, y [tokens, D] (row strides), the sequences one behind the other: token b * T + t of N equal ones of
 * T = tokens / N, or cu_seqlens device int32 [N + 1] (not decreasing; outputs' rows in front of the first sequence and behind
 * the last one are left as they were, or become zeros with zero_rest, as what sums over all rows needs it).
 * h0 and final fp32 [N, D], contiguous: the states before and after each sequence (an empty one's passes through).
 * Gates are meant to be <= 0 (-inf forgets); with larger ones every product of gates over consecutive tokens of a
 * sequence has to stay finite.  Sums and states are fp32; a NaN or an infinity reaches what follows in its sequence and
 * channel.  No output may share memory with an input.
 */
typedef struct {
  int num_seqs;         /* N >= 1                                                        */
  int tokens;           /* of all sequences; without cu_seqlens a multiple of N          */
  int dim;              /* D, 1 .. 2^20                                                  */
  gdn_dtype dtype;      /* of x, y, dy, dx                                               */
  gdn_dtype gate_dtype; /* of g, dg: dtype or GDN_FP32                                   */
  int reserved;         /* must be 0                                                     */
  int64_t x_row, g_row; /* row strides                                                   */
  int64_t y_row;        /* of y; backward: of dx                                         */
  int64_t dy_row, dg_row; /* backward                                                    */
  int64_t state_row;    /* step: of the state                                            */
  int zero_rest;        /* 1: zeros in the rows that no sequence names; 0: these stay    */
  int reserved1;        /* must be 0                                                     */
} gdn_scan_shape;

/* states fp32 [gdn_scan_states_rows, D] or NULL: gets the state before every 16th token of the line, for the backward.
 * h0 NULL: zeros.  final NULL: not wanted. */
int64_t gdn_scan_states_rows(const gdn_scan_shape *shape);
int gdn_scan_fwd(const gdn_scan_shape *shape, const void *x, const void *g, const float *h0 /* nullable */,
                 const int32_t *cu_seqlens /* nullable */, void *y, float *final /* nullable */, float *states /* nullable */,
                 gdn_stream_t stream);

/* Gradients, given dy, d_final (of the final states; NULL: zero) and the forward's x, g, h0 and states:
 *     d_t = dy_t + exp(g_{t+1}) d_{t+1} (the last token's: dy + d_final),  dx = d,  dg_t = exp(g_t) d_t h_{t-1},
 *     dh0 = exp(g_0) d_0 (NULL: not wanted). */
int gdn_scan_bwd(const gdn_scan_shape *shape, const void *dy, const void *x, const void *g, const float *states,
                 const float *h0 /* nullable */, const float *d_final /* nullable */, const int32_t *cu_seqlens /* nullable */,
                 void *dx, void *dg, float *dh0 /* nullable */, gdn_stream_t stream);

/* One token of each sequence (tokens = N): state [N, D] fp32 (state_row) is updated in place, y is the new state. */
int gdn_scan_step(const gdn_scan_shape *shape, const void *x, const void *g, float *state, void *y, gdn_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* GDN_BLOCK_H_ */
