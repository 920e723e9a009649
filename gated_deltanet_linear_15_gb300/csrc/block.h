// Host-visible launchers of the operators declared in include/gdn_block.h (internal to the library).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdn_block.h"

namespace gdn {

constexpr int ROPE_THREADS = 128;  // of a CTA, which holds at least a head's 32-byte units

// ---- rotary positions
// One head group of a launch: heads of one tensor, turned (or only copied, when `turn` is 0) from src to dst; dst NULL
// for the keys and values of an append, which go to the cache.
struct RopeGroup {
  const void *src;
  void *dst;
  long long s_tok, s_head, d_tok, d_head, d_page;  // elements; with d_page != 0: d_tok is the slot stride in a page
  int heads, turn;
};
struct RopeArgs {
  RopeGroup grp[3];
  int ngrp, tokens, heads, D, rot, interleaved, inverse, rows;
  const float *table;
  const int *positions;                 // NULL: positions from cu_q and kv_lens
  const int *cu_q, *kv_lens, *pages;    // append
  long long table_stride;
  int N, per_seq, log2P, num_pages, max_pages;
};
cudaError_t launch_rope(const RopeArgs &a, bool bf16_type, bool vec, cudaStream_t st);
cudaError_t launch_rope_table(const double *freq, int pairs, int rows, double amplitude, float *table, cudaStream_t st);

// ---- pages
constexpr int MAX_POOLS = 64;  // pools of one launch
struct PoolList {
  gdn_slot_pool p[MAX_POOLS];
  int list[MAX_POOLS];              // which of the launch's two pair lists a pool follows
  long long chunk0[MAX_POOLS + 1];  // chunks of the pools before, per pair
  int n;
};
struct PairList {
  const int *src, *dst;  // slot src[i] -> dst[i]; negative numbers are left out
};
struct PagesArgs {
  int S, W, NP, P;
  long long ts;
  int *table, *lens, *ref;
};
// what a copy launch does to the tables first: nothing, the rows of forked children, or the renaming of moved pages
struct TableJob {
  enum { NONE, FORK, REMAP } kind;
  PagesArgs a;
  const int *psrc, *pdst, *new_page;  // FORK: parent, child, copied page of every fork
  int m;
  const int *table_in, *ref_in, *map, *front;  // REMAP: new number of every moved page, pages in use
};
// pairs i < (count_dev ? min(count, *count_dev) : count) of both lists
cudaError_t launch_slots_copy(const PoolList &pl, const PairList (&pairs)[2], int count, const int *count_dev, const TableJob &job,
                              cudaStream_t st);
cudaError_t launch_pages_extend(const PagesArgs &a, const int *seqs, const int *add, int m, int *ok, int *ws,
                                cudaStream_t st);
cudaError_t launch_pages_fork_plan(const PagesArgs &a, const int *parents, const int *children, int m, int *new_page,
                                   int *src, int *psrc, int *pdst, cudaStream_t st);
cudaError_t launch_pages_free(const PagesArgs &a, const int *seqs, int m, cudaStream_t st);
cudaError_t launch_pages_compact_plan(const PagesArgs &a, const int *ref_in, int *map, int *src, int *dst, int *moves,
                                      int *front, cudaStream_t st);

// ---- norm
struct NormArgs {
  const void *x, *res;      // backward: dy, dh
  const void *h;            // backward
  const float *weight;
  void *h_out, *y;          // backward: dx in y
  float *scale, *rstd;
  const float *rstd_in;
  float *dw, *part;
  long long T, x_row, r_row, h_row, y_row;
  int D, group, fp8;
  float eps, off;
};
int norm_bwd_ctas(const NormArgs &a, bool bf16_type, bool vec, int sms);
cudaError_t launch_norm_fwd(const NormArgs &a, bool bf16_type, bool vec, int sms, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormArgs &a, bool bf16_type, bool vec, int sms, cudaStream_t st);

}  // namespace gdn
