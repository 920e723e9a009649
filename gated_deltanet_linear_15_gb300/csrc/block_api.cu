// C entry points of include/gdn_block.h: argument checks, workspace layout and launches of the operators next to the
// delta rule (paged attention, rotary positions, cache pages, root-mean-square norm, gated linear recurrence).
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <vector>

#include "block.h"
#include "host.h"
#include "paged.cuh"

using namespace gdn;

namespace {

typedef cudaStream_t Stream;

size_t esize(gdn_dtype d) { return d == GDN_BF16 ? 2 : 4; }
bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
int ilog2(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

int need_ptr(const void *p, const char *name) {
  return p ? GDN_OK : fail(GDN_ERR_INVALID_ARG, "%s is NULL", name);
}
int need_aligned(const void *p, const char *name) {
  if (!p) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", name);
  return aligned16(p) ? GDN_OK : fail(GDN_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
}
#define TRY(e)            \
  do {                    \
    const int rc_ = (e);  \
    if (rc_) return rc_;  \
  } while (0)

// ------------------------------------------------------------------ paged shapes
int check_paged(const gdn_paged_shape *s, bool attn) {
  if (!s) return fail(GDN_ERR_INVALID_ARG, "shape is NULL");
  if (s->reserved && !(attn && (uint32_t)s->reserved == (uint32_t)GDN_DEBUG_WAIT_TIMEOUT))
    return fail(GDN_ERR_INVALID_ARG, "reserved fields must be 0");
  if (s->dtype != GDN_BF16 && s->dtype != GDN_FP32) return fail(GDN_ERR_INVALID_ARG, "unknown dtype");
  if (s->num_seqs < 0 || s->total_q < 0) return fail(GDN_ERR_INVALID_ARG, "need num_seqs >= 0, total_q >= 0");
  if (s->num_heads < 1 || s->num_kv_heads < 1 || s->num_heads % s->num_kv_heads)
    return fail(GDN_ERR_INVALID_ARG, "num_heads (%d) must be a positive multiple of num_kv_heads (%d)", s->num_heads, s->num_kv_heads);
  if (!pow2(s->page_size) || s->page_size < 16 || s->page_size > 4096)
    return fail(GDN_ERR_UNSUPPORTED, "page_size must be a power of two from 16 to 4096 (got %d)", s->page_size);
  if (s->num_pages < 1 || s->max_pages < 0) return fail(GDN_ERR_INVALID_ARG, "need num_pages >= 1, max_pages >= 0");
  if (s->max_pages > 0 && s->num_seqs > 1 && s->table_stride != 0 && s->table_stride < s->max_pages)
    return fail(GDN_ERR_INVALID_ARG, "table_stride is smaller than max_pages");
  return GDN_OK;
}

int check_attn(const gdn_paged_shape *s) {
  TRY(check_paged(s, true));
  if (s->head_dim != 64 && s->head_dim != 128) return fail(GDN_ERR_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", s->head_dim);
  if (s->window < 0) return fail(GDN_ERR_INVALID_ARG, "window must be >= 0");
  if (s->max_q < 0) return fail(GDN_ERR_INVALID_ARG, "max_q must be >= 0");
  if (!std::isfinite(s->scale)) return fail(GDN_ERR_INVALID_ARG, "scale must be finite");
  if ((long long)s->total_q * (s->num_heads / s->num_kv_heads) > 0x7fffffffll)
    return fail(GDN_ERR_UNSUPPORTED, "too many query rows");
  if (s->num_heads / s->num_kv_heads > 65535)  // a cut item's header has 16 bits for the place in the group
    return fail(GDN_ERR_UNSUPPORTED, "more than 65535 query heads per key head");
  const int v = 16 / (int)esize(s->dtype);
  const struct { int64_t v; const char *name; } st[] = {
      {s->q_tok, "q_tok"}, {s->q_head, "q_head"}, {s->k_page, "k_page"}, {s->k_tok, "k_tok"}, {s->k_head, "k_head"},
      {s->v_page, "v_page"}, {s->v_tok, "v_tok"}, {s->v_head, "v_head"}, {s->o_tok, "o_tok"}, {s->o_head, "o_head"}};
  for (const auto &x : st) {
    if (x.v < 0) return fail(GDN_ERR_INVALID_ARG, "stride %s is negative", x.name);
    if ((x.name[0] == 'k' || x.name[0] == 'v') && (x.v == 0 || x.v >= (1ll << 37)))  // what a tensor map can hold
      return fail(GDN_ERR_UNSUPPORTED, "stride %s must be positive and below 2^37", x.name);
    if (x.v % v) return fail(GDN_ERR_INVALID_ARG, "stride %s is not a multiple of 16 bytes", x.name);
  }
  return GDN_OK;
}

// The kernel of a call and its grid: bf16 with more than 32 (query, head) rows per key head in the longest sequence
// takes the tensor-core kernel (256 rows, one CTA per SM), everything else the row kernel (16 or 32 rows).  Sequences of
// 16384 tokens, 8 key heads of 128, 4 heads each, row kernel / tensor-core kernel: 8 new tokens (32 rows) of one sequence
// 22 / 29 us, of 16 ragged ones 105 / 136 us; 9 new tokens 30 / 28 and 185 / 136 us; 16 new tokens 33 / 30 and 192 / 132 us.
struct AttnPlan {
  bool tc;
  int MT, ctas;
  size_t off_status, off_part, total;
};
AttnPlan attn_plan(const gdn_paged_shape *s) {
  AttnPlan p;
  const int G = s->num_heads / s->num_kv_heads;
  const long long mean = ((long long)s->total_q + s->num_seqs - 1) / std::max(1, s->num_seqs);
  const long long rows = (s->max_q > 0 ? s->max_q : mean) * G;
  const bool bf = s->dtype == GDN_BF16;
  p.tc = bf && rows > 32;
  p.MT = p.tc ? 256 : attn_rows_tile(bf, s->head_dim, (int)std::min(rows, 1ll << 20));
  p.ctas = num_sms() * (p.tc ? 1 : attn_rows_per_sm(bf, s->head_dim, p.MT));
  p.off_status = up256((size_t)p.ctas * sizeof(int4));
  p.off_part = p.off_status + up256((size_t)p.ctas * sizeof(int));
  p.total = p.off_part + up256((size_t)p.ctas * 2 * record_floats(p.MT, s->head_dim) * 4);
  return p;
}

// keys or values as [pages, slots, heads, features], box = 128 bytes of one head's features, `slots` slots
int cache_map(CUtensorMap *m, const void *p, const gdn_paged_shape *s, int64_t page, int64_t tok, int64_t head, int slots) {
  const int es = (int)esize(s->dtype);
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(GDN_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[4] = {(cuuint64_t)s->head_dim, (cuuint64_t)s->num_kv_heads, (cuuint64_t)s->page_size, (cuuint64_t)s->num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)head * es, (cuuint64_t)tok * es, (cuuint64_t)page * es};
  const cuuint32_t box[4] = {(cuuint32_t)(128 / es), 1, (cuuint32_t)slots, 1}, step[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<void *>(p),
                        dims, strides, box, step,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GDN_OK : fail(GDN_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

// ------------------------------------------------------------------ pages
int check_pages(const gdn_pages_shape *s) {
  if (!s) return fail(GDN_ERR_INVALID_ARG, "shape is NULL");
  if (s->reserved[0] || s->reserved[1]) return fail(GDN_ERR_INVALID_ARG, "reserved fields must be 0");
  if (s->num_seqs < 1 || s->max_pages < 1) return fail(GDN_ERR_INVALID_ARG, "need num_seqs >= 1, max_pages >= 1");
  if (s->num_pages < 1 || s->num_pages > (1 << 20)) return fail(GDN_ERR_UNSUPPORTED, "num_pages must be 1 .. 2^20 (got %d)", s->num_pages);
  if (s->page_size < 1 || s->page_size > (1 << 20)) return fail(GDN_ERR_INVALID_ARG, "page_size must be 1 .. 2^20");
  if (s->table_stride < s->max_pages) return fail(GDN_ERR_INVALID_ARG, "table_stride is smaller than max_pages");
  return GDN_OK;
}
PagesArgs pages_args(const gdn_pages_shape *s, int *table, int *lens, int *ref) {
  PagesArgs a;
  a.S = s->num_seqs;
  a.W = s->max_pages;
  a.NP = s->num_pages;
  a.P = s->page_size;
  a.ts = s->table_stride;
  a.table = table;
  a.lens = lens;
  a.ref = ref;
  return a;
}
// least: slots that each has to have
int check_pools(const gdn_slot_pool *p, int n, const char *what, int least) {
  if (n < 0) return fail(GDN_ERR_INVALID_ARG, "negative number of %s", what);
  if (n && !p) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", what);
  for (int i = 0; i < n; ++i) {
    if (!p[i].base) return fail(GDN_ERR_INVALID_ARG, "%s[%d].base is NULL", what, i);
    if (p[i].bytes < 0 || p[i].slots < 0 || p[i].stride < p[i].bytes)
      return fail(GDN_ERR_INVALID_ARG, "%s[%d]: need 0 <= bytes <= stride and slots >= 0", what, i);
    if (!aligned16(p[i].base) || p[i].stride % 16 || p[i].bytes % 16)
      return fail(GDN_ERR_INVALID_ARG, "%s[%d]: base, stride and bytes must be multiples of 16", what, i);
    if (p[i].slots < least)
      return fail(GDN_ERR_INVALID_ARG, "%s[%d] has %lld slots where %d are named", what, i, (long long)p[i].slots, least);
  }
  return GDN_OK;
}
// the copies of a call, MAX_POOLS pools to a launch, the first of which does the job on the tables too
int copy_slots(const gdn_slot_pool *p, int n, const gdn_slot_pool *q, int nq, const PairList (&pairs)[2], int count,
               const int *count_dev, TableJob job, Stream st) {
  int b = 0;
  do {
    PoolList l;
    l.n = std::min(MAX_POOLS, n + nq - b);
    for (int i = 0; i < l.n; ++i) {
      l.list[i] = b + i >= n;
      l.p[i] = b + i < n ? p[b + i] : q[b + i - n];
    }
    PROF("slots_copy");
    CK(launch_slots_copy(l, pairs, count, count_dev, job, st));
    job.kind = TableJob::NONE;
    b += l.n;
  } while (b < n + nq);
  return GDN_OK;
}

// ------------------------------------------------------------------ norm
int check_norm(const gdn_norm_shape *s, bool bwd) {
  if (!s) return fail(GDN_ERR_INVALID_ARG, "shape is NULL");
  if (s->reserved[0] || s->reserved[1]) return fail(GDN_ERR_INVALID_ARG, "reserved fields must be 0");
  if (s->dtype != GDN_BF16 && s->dtype != GDN_FP32) return fail(GDN_ERR_INVALID_ARG, "unknown dtype");
  if (s->rows < 0) return fail(GDN_ERR_INVALID_ARG, "rows must be >= 0");
  if (s->dim < 1 || s->dim > 65536) return fail(GDN_ERR_UNSUPPORTED, "dim must be 1 .. 65536 (got %d)", s->dim);
  if (!std::isfinite(s->weight_offset)) return fail(GDN_ERR_INVALID_ARG, "weight_offset must be finite");
  if (s->x_row < 0 || s->r_row < 0 || s->h_row < 0 || s->y_row < 0) return fail(GDN_ERR_INVALID_ARG, "row strides must be >= 0");
  if (bwd) return GDN_OK;
  if (!(s->eps > 0.f) || !std::isfinite(s->eps)) return fail(GDN_ERR_INVALID_ARG, "eps must be finite and > 0");
  if (s->fp8 != 0 && s->fp8 != 1) return fail(GDN_ERR_INVALID_ARG, "fp8 must be 0 or 1");
  if (s->group != 0 && (!s->fp8 || s->group != 128)) return fail(GDN_ERR_UNSUPPORTED, "group must be 0, or 128 with fp8 (got %d)", s->group);
  if (s->group && s->dim % s->group) return fail(GDN_ERR_UNSUPPORTED, "dim (%d) is not a multiple of group (%d)", s->dim, s->group);
  return GDN_OK;
}
// rows written must not overlap one another
int check_row(int64_t row, const gdn_norm_shape *s, const char *name) {
  return s->rows > 1 && row < s->dim ? fail(GDN_ERR_INVALID_ARG, "%s is smaller than dim", name) : GDN_OK;
}
bool vec_ok(const void *p, int64_t row, int v) { return !p || (aligned16(p) && row % v == 0); }

// ------------------------------------------------------------------ attention
// the arguments of every attention
int check_attn_args(const gdn_paged_shape *s, const void *q, const void *k, const void *v, const int32_t *table, const int32_t *cu_q,
                    const int32_t *kv_lens, const void *o) {
  if (!cu_q && s->total_q % s->num_seqs) return fail(GDN_ERR_INVALID_ARG, "without cu_q, total_q must be a multiple of num_seqs");
  TRY(need_aligned(q, "q"));
  TRY(need_aligned(k, "k_cache"));
  TRY(need_aligned(v, "v_cache"));
  TRY(need_aligned(o, "o"));
  if (s->max_pages > 0) TRY(need_ptr(table, "page_table"));
  return need_ptr(kv_lens, "kv_lens");
}
int check_attn_memory(const void *q, const void *k, const void *v, const void *o, const void *ws, size_t ws_bytes, size_t need) {
  if (!ws || ws_bytes < need) return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
  // a cut item's record leaves in 32-byte stores (attn_chunk_tc.cu); every part of the workspace is a multiple of that
  if (reinterpret_cast<uintptr_t>(ws) & 31) return fail(GDN_ERR_INVALID_ARG, "workspace is not 32-byte aligned");
  // a CTA reads queries and cache rows after another wrote its outputs
  if (o == q || o == k || o == v) return fail(GDN_ERR_INVALID_ARG, "o is one of the inputs");
  return GDN_OK;
}
PagedArgs attn_args(const gdn_paged_shape *s, const void *q, const void *k, const void *v, const int32_t *table, const int32_t *cu_q,
                    const int32_t *kv_lens, void *o, float *lse) {
  PagedArgs a = {};
  a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
  a.table = table; a.cu_q = cu_q; a.kv_lens = kv_lens;
  a.table_stride = s->table_stride;
  a.q_tok = s->q_tok; a.q_head = s->q_head;
  a.k_page = s->k_page; a.k_tok = s->k_tok; a.k_head = s->k_head;
  a.v_page = s->v_page; a.v_tok = s->v_tok; a.v_head = s->v_head;
  a.o_tok = s->o_tok; a.o_head = s->o_head;
  a.N = s->num_seqs; a.total_q = s->total_q; a.per_seq = cu_q ? 0 : s->total_q / s->num_seqs;
  a.Hq = s->num_heads; a.Hkv = s->num_kv_heads; a.G = s->num_heads / s->num_kv_heads;
  a.log2P = ilog2(s->page_size);
  a.num_pages = s->num_pages; a.max_pages = s->max_pages;
  // a window as long as a table row limits nothing; what stays is far from where differences of positions would wrap
  a.window = s->window < (long long)s->max_pages * s->page_size ? s->window : 0;
  a.scale_log2 = s->scale * 1.4426950408889634f;
  a.expire = s->reserved != 0;
  return a;
}
// a kernel's part of the workspace, from `ws` on
void attn_scratch(PagedArgs &a, const AttnPlan &p, void *ws) {
  a.hdr = static_cast<int4 *>(ws);
  a.part = reinterpret_cast<float *>(static_cast<char *>(ws) + p.off_part);
  a.status = reinterpret_cast<int *>(static_cast<char *>(ws) + p.off_status);
}
int run_attn(const gdn_paged_shape *s, const AttnPlan &p, const PagedArgs &a, Part part, Stream st) {
  const bool bf = s->dtype == GDN_BF16;
  CUtensorMap tk, tv;
  const int slots = p.tc ? std::min(s->page_size, 128) : attn_rows_box(bf, p.MT, s->page_size);
  TRY(cache_map(&tk, a.k, s, s->k_page, s->k_tok, s->k_head, slots));
  TRY(cache_map(&tv, a.v, s, s->v_page, s->v_tok, s->v_head, slots));
  if (p.tc) {
    PROF("attn_chunk");
    CK(launch_attn_chunk_tc(a, part, tk, tv, s->head_dim, p.ctas, st));
  } else {
    PROF("attn_rows");
    CK(launch_attn_rows(a, part, tk, tv, bf, s->head_dim, p.MT, p.ctas, st));
  }
  return GDN_OK;
}
int run_attn_join(const gdn_paged_shape *s, const AttnPlan &p, const PagedArgs &a, Stream st) {
  // tiles: every sequence has at most one that is not full
  const long long tiles = s->num_seqs + (long long)s->total_q * a.G / p.MT;
  PROF("attn_join");
  CK(launch_attn_join(a, s->dtype == GDN_BF16, s->head_dim, p.MT, p.ctas, (int)std::min(tiles * s->num_kv_heads, (long long)p.ctas), st));
  return GDN_OK;
}
int paged_attn(const gdn_paged_shape *s, int sinks, const void *q, const void *k, const void *v, const int32_t *table, const int32_t *cu_q,
               const int32_t *kv_lens, void *o, float *lse, void *ws, size_t ws_bytes, Stream st) {
  TRY(check_attn_args(s, q, k, v, table, cu_q, kv_lens, o));
  const AttnPlan p = attn_plan(s);
  TRY(check_attn_memory(q, k, v, o, ws, ws_bytes, p.total));
  PagedArgs a = attn_args(s, q, k, v, table, cu_q, kv_lens, o, lse);
  // sinks beyond the table's room stand for all of it; without a window they add nothing
  a.sinks = (int)std::min((long long)sinks, (long long)s->max_pages * s->page_size);
  attn_scratch(a, p, ws);
  TRY(run_attn(s, p, a, a.window && a.sinks ? SINKS : ALL, st));
  return run_attn_join(s, p, a, st);
}
// the words of the CTAs of one kernel
int attn_status_words(const AttnPlan &p, const void *ws) {
  try {
    std::vector<int> st(p.ctas);
    if (cudaMemcpy(st.data(), static_cast<const char *>(ws) + p.off_status, st.size() * sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
      return -1;
    int word = 0;
    for (int x : st) word |= x ? 4 : 0;
    return word;
  } catch (...) {
    return -1;
  }
}

// ------------------------------------------------------------------ attention behind a shared prefix
// Where sharing saves no more than this many bytes, a batch is computed as if its sequences shared nothing.  Two parts take
// three launches more, some 10 us; reading shared keys again, mostly from L2, costs 1 us for 13 MB in bf16 and for 7 in fp32.
// One new token, caches cold, us as one / in two parts: bf16, 8 key heads of 128: 16 sequences behind 1024 tokens (67 MB)
// 25 / 34, 32 (138 MB) 29 / 32, 8 behind 4096 (119 MB) 31 / 28, 4 behind 16384 (202 MB) 48 / 39, 64 behind 4096 (1.1 GB)
// 120 / 43; fp32, 2 key heads of 128: 64 behind 256 (41 MB) 28 / 35, 8 behind 4096 (59 MB) 37 / 41, 64 behind 512 (74 MB)
// 40 / 37, 4 behind 16384 (101 MB) 54 / 49.
// (The host knows the room of a table row, not the lengths: behind a table of 32768 tokens the first of these, and 4 samples
// after 992 tokens, go in two parts too: 34 instead of 25 us, 26 instead of 17.)
double prefix_min_bytes(gdn_dtype d) { return d == GDN_BF16 ? 128e6 : 80e6; }
// Query rows of a sequence and key head, on the mean, from which on a batch is computed in one part: they fill half a tile of the
// chunk kernel (fp32: one of the row kernel) by themselves, so the products are as many with the prefix shared, and two parts
// add their fp32 sums.  Us in one / two parts, caches cold: bf16, 8 sequences behind 8192 tokens, 8 key heads of 128, 4 heads each:
// 8 new tokens (32 rows) 55 / 47, 24: 73 / 65, 32: 59 / 71, 40: 85 / 78, 64: 67 / 98, 80: 129 / 110, 128: 104 / 149, 1024: 656 / 962;
// 64 behind 2048, 2 heads each, 48 (96 rows): 143 / 141, 64: 110 / 164; fp32, 16 behind 4096, 4 key heads of 128, 4 heads each:
// 1: 93 / 47, 4: 93 / 92, 8 (32 rows): 109 / 145, 64: 720 / 936; 32 behind 2048, 2 key heads of 64, 8 heads each, 4 (32 rows): 44 / 57.
int prefix_max_rows(gdn_dtype d) { return d == GDN_BF16 ? 128 : 32; }
struct PrefixLayout {
  bool split;  // in two parts; otherwise as sequences that share nothing
  gdn_paged_shape groups;  // the batch of heads
  AttnPlan head, tail;
  size_t off_head, off_tail, off_info, off_sums[2], off_mass[2], off_loc[2], total;
};
int check_prefix(const gdn_paged_shape *s, int groups, int max_group) {
  TRY(check_attn(s));
  if (s->window) return fail(GDN_ERR_UNSUPPORTED, "a window and a shared prefix do not go together");
  if (groups < 0 || (groups == 0 && s->num_seqs > 0) || groups > s->num_seqs)
    return fail(GDN_ERR_INVALID_ARG, "need 1 <= groups <= num_seqs (got %d, %d)", groups, s->num_seqs);
  if (max_group < 0) return fail(GDN_ERR_INVALID_ARG, "max_group must be >= 0");
  return GDN_OK;
}
PrefixLayout prefix_layout(const gdn_paged_shape *s, int groups, int max_group) {
  PrefixLayout l = {};
  l.tail = attn_plan(s);
  // bytes that sharing can save at most, as far as the host knows: the sequences of a group read what its first one reads
  const double saved = (double)(s->num_seqs - groups) * s->max_pages * s->page_size * s->num_kv_heads * s->head_dim * 2 * (double)esize(s->dtype);
  const double mean = (double)s->total_q * (s->num_heads / s->num_kv_heads) / std::max(1, s->num_seqs);
  l.split = saved > prefix_min_bytes(s->dtype) && mean < prefix_max_rows(s->dtype);
  if (!l.split) {
    l.total = l.tail.total;
    return l;
  }
  l.groups = *s;
  l.groups.num_seqs = groups;
  l.groups.max_q = max_group;
  l.head = attn_plan(&l.groups);
  const size_t rows = (size_t)s->total_q * s->num_heads;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += up256(bytes);
    return x;
  };
  l.off_tail = take(l.tail.total);
  l.off_head = take(l.head.total);
  l.off_info = take(((size_t)groups + s->num_seqs + 2) * sizeof(int4));
  for (int i = 0; i < 2; ++i) {
    l.off_sums[i] = take(rows * s->head_dim * sizeof(float));
    l.off_mass[i] = take(rows * sizeof(float2));
    l.off_loc[i] = take(rows * sizeof(int2));
  }
  l.total = at;
  return l;
}

// What a part costs, for the sharing of the SMs: a line through times taken with different shares.  Chunk kernel: 19 us and
// 1.5 for 256 rows and 128 keys (D = 64: 1.1).  Row kernel: 8 us and an SM's bytes at 71 GB/s, 33 with two groups of rows, 40 in
// fp32, but 0.4 at least for a block.
PrefixPlan::Share part_share(const gdn_paged_shape *s, const AttnPlan &p) {
  const bool bf = s->dtype == GDN_BF16;
  PrefixPlan::Share x;
  x.MT = p.MT;
  x.BN = p.tc ? 128 : attn_rows_block(bf, p.MT);
  x.per_sm = p.ctas / num_sms();
  x.start = p.tc ? 19.f : 8.f;
  x.setup = p.tc ? 5 : 2;
  x.cost = p.tc ? (s->head_dim == 64 ? 1.1f : 1.5f)
                : std::max(0.4f, x.BN * s->head_dim * 2 * esize(s->dtype) / (p.MT == 32 ? 33e3f : bf ? 71e3f : 40e3f));
  return x;
}

// ------------------------------------------------------------------ rotary positions
int check_rotary(const gdn_rotary_shape *s) {
  if (!s) return fail(GDN_ERR_INVALID_ARG, "shape is NULL");
  if (s->reserved) return fail(GDN_ERR_INVALID_ARG, "reserved fields must be 0");
  if (s->dtype != GDN_BF16 && s->dtype != GDN_FP32) return fail(GDN_ERR_INVALID_ARG, "unknown dtype");
  if (s->tokens < 0 || s->q_heads < 0 || s->k_heads < 0) return fail(GDN_ERR_INVALID_ARG, "negative size");
  if (s->head_dim < 2 || s->rot < 2 || s->rot % 2 || s->rot > s->head_dim)
    return fail(GDN_ERR_INVALID_ARG, "need an even rot with 2 <= rot <= head_dim (got rot %d, head_dim %d)", s->rot, s->head_dim);
  if (s->head_dim > 65536) return fail(GDN_ERR_UNSUPPORTED, "head_dim must be at most 65536");
  if (s->table_rows < 0) return fail(GDN_ERR_INVALID_ARG, "table_rows must be >= 0");
  if ((s->interleaved | s->inverse) & ~1) return fail(GDN_ERR_INVALID_ARG, "interleaved and inverse must be 0 or 1");
  if ((long long)(s->q_heads + (long long)s->k_heads) * s->head_dim > (1 << 28)) return fail(GDN_ERR_UNSUPPORTED, "too many heads");
  return GDN_OK;
}
int check_rotary_args(const gdn_rotary_shape *s, const void *q, const void *k, const float *table, const int32_t *positions,
                      const void *q_out, const void *k_out) {
  if (s->q_heads) {
    TRY(need_ptr(q, "q"));
    TRY(need_ptr(q_out, "q_out"));
  }
  if (s->k_heads) {
    TRY(need_ptr(k, "k"));
    TRY(need_ptr(k_out, "k_out"));
  }
  if (s->table_rows) TRY(need_aligned(table, "table"));
  return need_ptr(positions, "positions");
}
// vec: every access may take 16 bytes
RopeArgs rotary_args(const gdn_rotary_shape *s, const void *q, const void *k, const float *table, const int32_t *positions, void *q_out,
                     void *k_out, bool &vec) {
  RopeArgs a = {};
  const int v = 16 / (int)esize(s->dtype);
  vec = s->head_dim % (2 * v) == 0 && s->rot % (2 * v) == 0 && s->head_dim <= ROPE_THREADS * 2 * v;  // a CTA holds a head
  auto add = [&](const void *src, void *dst, int heads, int64_t st_, int64_t sh, int64_t dt, int64_t dh) {
    if (!heads) return;
    a.grp[a.ngrp++] = {src, dst, st_, sh, dt, dh, 0, heads, 1};
    a.heads += heads;
    vec = vec && aligned16(src) && aligned16(dst) && st_ % v == 0 && sh % v == 0 && dt % v == 0 && dh % v == 0;
  };
  add(q, q_out, s->q_heads, s->q_tok, s->q_head, s->qo_tok, s->qo_head);
  add(k, k_out, s->k_heads, s->k_tok, s->k_head, s->ko_tok, s->ko_head);
  a.tokens = s->tokens; a.D = s->head_dim; a.rot = s->rot; a.interleaved = s->interleaved; a.inverse = s->inverse;
  a.rows = s->table_rows; a.table = table; a.positions = positions;
  return a;
}
int check_append(const gdn_paged_shape *s) {
  TRY(check_paged(s, false));
  if (s->head_dim < 2 || s->rot < 2 || s->rot % 2 || s->rot > s->head_dim)
    return fail(GDN_ERR_INVALID_ARG, "need an even rot with 2 <= rot <= head_dim (got rot %d, head_dim %d)", s->rot, s->head_dim);
  if (s->head_dim > 65536 || (long long)s->num_heads * s->head_dim > (1 << 26)) return fail(GDN_ERR_UNSUPPORTED, "too many heads");
  if (s->interleaved & ~1) return fail(GDN_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (s->table_rows < 0) return fail(GDN_ERR_INVALID_ARG, "table_rows must be >= 0");
  return GDN_OK;
}
int check_append_args(const gdn_paged_shape *s, const void *q, const void *k, const void *v, const float *table, const void *k_cache,
                      const void *v_cache, const int32_t *page_table, const int32_t *cu_q, const int32_t *kv_lens, const void *q_out) {
  if (!cu_q && s->total_q % s->num_seqs) return fail(GDN_ERR_INVALID_ARG, "without cu_q, total_q must be a multiple of num_seqs");
  TRY(need_ptr(q, "q"));
  TRY(need_ptr(k, "k"));
  TRY(need_ptr(v, "v"));
  TRY(need_ptr(k_cache, "k_cache"));
  TRY(need_ptr(v_cache, "v_cache"));
  TRY(need_ptr(q_out, "q_out"));
  if (s->max_pages > 0) TRY(need_ptr(page_table, "page_table"));
  TRY(need_ptr(kv_lens, "kv_lens"));
  if (s->table_rows) TRY(need_aligned(table, "table"));
  if (s->k_page < 1 || s->v_page < 1) return fail(GDN_ERR_INVALID_ARG, "page strides must be positive");
  return GDN_OK;
}
RopeArgs append_args(const gdn_paged_shape *s, const void *q, const void *k, const void *v, const float *table, void *k_cache, void *v_cache,
                     const int32_t *page_table, const int32_t *cu_q, const int32_t *kv_lens, void *q_out, bool &vec) {
  RopeArgs a = {};
  const int w = 16 / (int)esize(s->dtype);
  vec = s->head_dim % (2 * w) == 0 && s->rot % (2 * w) == 0 && s->head_dim <= ROPE_THREADS * 2 * w;  // a CTA holds a head
  auto add = [&](const void *src, void *dst, int heads, int turn, int64_t st_, int64_t sh, int64_t dt, int64_t dh, int64_t dp) {
    a.grp[a.ngrp++] = {src, dst, st_, sh, dt, dh, dp, heads, turn};
    a.heads += heads;
    vec = vec && aligned16(src) && aligned16(dst) && st_ % w == 0 && sh % w == 0 && dt % w == 0 && dh % w == 0 && dp % w == 0;
  };
  add(q, q_out, s->num_heads, 1, s->q_tok, s->q_head, s->o_tok, s->o_head, 0);
  add(k, k_cache, s->num_kv_heads, 1, s->kn_tok, s->kn_head, s->k_tok, s->k_head, s->k_page);
  add(v, v_cache, s->num_kv_heads, 0, s->vn_tok, s->vn_head, s->v_tok, s->v_head, s->v_page);
  a.tokens = s->total_q; a.D = s->head_dim; a.rot = s->rot; a.interleaved = s->interleaved;
  a.rows = s->table_rows; a.table = table;
  a.cu_q = cu_q; a.kv_lens = kv_lens; a.pages = page_table; a.table_stride = s->table_stride;
  a.N = s->num_seqs; a.per_seq = cu_q ? 0 : s->total_q / s->num_seqs;
  a.log2P = ilog2(s->page_size); a.num_pages = s->num_pages; a.max_pages = s->max_pages;
  return a;
}
int check_head_norm(int head_dim, int inverse, float eps, float off) {
  if (head_dim > NORM_ROPE_MAX_DIM) return fail(GDN_ERR_UNSUPPORTED, "head_dim must be at most %d with a norm (got %d)", NORM_ROPE_MAX_DIM, head_dim);
  if (inverse) return fail(GDN_ERR_INVALID_ARG, "inverse must be 0 with a norm");
  if (!(eps > 0.f) || !std::isfinite(eps)) return fail(GDN_ERR_INVALID_ARG, "eps must be finite and > 0");
  if (!std::isfinite(off)) return fail(GDN_ERR_INVALID_ARG, "weight_offset must be finite");
  return GDN_OK;
}
// the 32-byte units of a head are a power of two, in one warp
bool head_in_warp(int head_dim, gdn_dtype d) {
  const int units = head_dim * (int)esize(d) / 32;
  return pow2(units) && units <= 32;
}

// ------------------------------------------------------------------ gated linear recurrence
int check_scan(const gdn_scan_shape *s) {
  if (!s) return fail(GDN_ERR_INVALID_ARG, "shape is NULL");
  if (s->reserved || s->reserved1) return fail(GDN_ERR_INVALID_ARG, "reserved fields must be 0");
  if (s->zero_rest & ~1) return fail(GDN_ERR_INVALID_ARG, "zero_rest must be 0 or 1");
  if (s->dtype != GDN_BF16 && s->dtype != GDN_FP32) return fail(GDN_ERR_INVALID_ARG, "unknown dtype");
  if (s->gate_dtype != s->dtype && s->gate_dtype != GDN_FP32) return fail(GDN_ERR_INVALID_ARG, "gate_dtype must be dtype or fp32");
  if (s->num_seqs < 1 || s->tokens < 0) return fail(GDN_ERR_INVALID_ARG, "need num_seqs >= 1, tokens >= 0");
  if (s->tokens > 0x7fff0000) return fail(GDN_ERR_UNSUPPORTED, "too many tokens");
  if (s->dim < 1 || s->dim > (1 << 20)) return fail(GDN_ERR_UNSUPPORTED, "dim must be 1 .. 2^20 (got %d)", s->dim);
  if (s->x_row < 0 || s->g_row < 0 || s->y_row < 0 || s->dy_row < 0 || s->dg_row < 0 || s->state_row < 0)
    return fail(GDN_ERR_INVALID_ARG, "row strides must be >= 0");
  return GDN_OK;
}
// rows written must not overlap one another
int check_scan_row(int64_t row, const gdn_scan_shape *s, const char *name) {
  return s->tokens > 1 && row < s->dim ? fail(GDN_ERR_INVALID_ARG, "%s is smaller than dim", name) : GDN_OK;
}
ScanArgs scan_args(const gdn_scan_shape *s, const void *x, const void *g, const int32_t *cu) {
  ScanArgs a = {};
  a.x = x;
  a.g = g;
  a.cu = cu;
  a.N = s->num_seqs;
  a.tokens = s->tokens;
  a.T = cu ? 0 : s->tokens / s->num_seqs;
  a.D = s->dim;
  a.x_row = s->x_row;
  a.g_row = s->g_row;
  a.y_row = s->y_row;
  a.dy_row = s->dy_row;
  a.dg_row = s->dg_row;
  a.h_row = s->state_row;
  a.zero_rest = s->zero_rest;
  return a;
}
// whether rows and pointer allow accesses of `bytes` that do not leave the row's features
struct Access {
  int move = 16;
  void add(const void *p, int64_t row, int es, int dim) {
    for (; move > 2; move = move == 16 ? 4 : 2)
      if (reinterpret_cast<uintptr_t>(p) % move == 0 && row * es % move == 0 && (int64_t)dim * es % move == 0) return;
  }
};
// the bytes of an access for a call: rows as in m; the fp32 states go by pairs of channels then, or singly with single ones
int scan_move(const Access &m, const gdn_scan_shape *s, std::initializer_list<const float *> states) {
  int move = m.move;
  for (const float *p : states)
    if (p && reinterpret_cast<uintptr_t>(p) % 8) move = std::min(move, s->dtype == GDN_FP32 ? 4 : 2);
  // without 16-byte pieces, channels of bf16 go in pairs and of fp32 singly; rows of both types at once go singly
  if (move == 4 && s->dtype != s->gate_dtype) move = 2;
  return move;
}
// no tokens at all: every state passes through
int scan_no_tokens(const gdn_scan_shape *s, const float *in, float *out, Stream st) {
  const size_t n = (size_t)s->num_seqs * s->dim * sizeof(float);
  if (out && in) CK(cudaMemcpyAsync(out, in, n, cudaMemcpyDeviceToDevice, st));
  else if (out) CK(cudaMemsetAsync(out, 0, n, st));
  return GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_paged_attn_workspace_size(const gdn_paged_shape *s) {
  if (check_attn(s)) return 0;
  return attn_plan(s).total;
}

int gdn_paged_attn_fwd(const gdn_paged_shape *s, const void *q, const void *k, const void *v, const int32_t *table,
                       const int32_t *cu_q, const int32_t *kv_lens, void *o, float *lse, void *ws, size_t ws_bytes,
                       gdn_stream_t stream) {
  TRY(check_attn(s));
  if (s->total_q == 0 || s->num_seqs == 0) return GDN_OK;
  return paged_attn(s, 0, q, k, v, table, cu_q, kv_lens, o, lse, ws, ws_bytes, (Stream)stream);
}

int gdn_paged_attn_sinks_fwd(const gdn_paged_shape *s, int sinks, const void *q, const void *k, const void *v, const int32_t *table,
                             const int32_t *cu_q, const int32_t *kv_lens, void *o, float *lse, void *ws, size_t ws_bytes,
                             gdn_stream_t stream) {
  TRY(check_attn(s));
  if (sinks < 0) return fail(GDN_ERR_INVALID_ARG, "sinks must be >= 0");
  if (s->total_q == 0 || s->num_seqs == 0) return GDN_OK;
  return paged_attn(s, sinks, q, k, v, table, cu_q, kv_lens, o, lse, ws, ws_bytes, (Stream)stream);
}

size_t gdn_prefix_attn_workspace_size(const gdn_paged_shape *s, int groups, int max_group) {
  if (check_prefix(s, groups, max_group)) return 0;
  return prefix_layout(s, groups, max_group).total;
}

int gdn_prefix_attn_fwd(const gdn_paged_shape *s, int groups, int max_group, const void *q, const void *k, const void *v,
                        const int32_t *table, const int32_t *cu_q, const int32_t *kv_lens, const int32_t *cu_seqs,
                        const int32_t *prefix_lens, void *o, float *lse, void *ws, size_t ws_bytes, gdn_stream_t stream) {
  TRY(check_prefix(s, groups, max_group));
  if (s->total_q == 0 || s->num_seqs == 0) return GDN_OK;
  if (!cu_seqs && s->num_seqs % groups) return fail(GDN_ERR_INVALID_ARG, "without cu_seqs, num_seqs must be a multiple of groups");
  TRY(check_attn_args(s, q, k, v, table, cu_q, kv_lens, o));
  TRY(need_ptr(prefix_lens, "prefix_lens"));
  const PrefixLayout l = prefix_layout(s, groups, max_group);
  TRY(check_attn_memory(q, k, v, o, ws, ws_bytes, l.total));
  const Stream st = (Stream)stream;
  if (!l.split) return paged_attn(s, 0, q, k, v, table, cu_q, kv_lens, o, lse, ws, ws_bytes, st);
  char *w = static_cast<char *>(ws);
  PagedArgs tail = attn_args(s, q, k, v, table, cu_q, kv_lens, o, lse), head = tail;
  head.N = groups;
  attn_scratch(head, l.head, w + l.off_head);
  attn_scratch(tail, l.tail, w + l.off_tail);
  PrefixPlan plan;
  plan.cu_seqs = cu_seqs;
  plan.prefix_lens = prefix_lens;
  plan.groups = groups;
  plan.head = reinterpret_cast<int4 *>(w + l.off_info);
  plan.tail = plan.head + groups;
  plan.ctas = reinterpret_cast<int *>(plan.tail + s->num_seqs);
  plan.blocks = reinterpret_cast<unsigned long long *>(plan.ctas + 4);
  plan.sms = num_sms();
  plan.together = head.together = tail.together = !(l.head.tc && l.tail.tc);
  plan.share[0] = part_share(s, l.head);
  plan.share[1] = part_share(s, l.tail);
  head.info = plan.head;
  tail.info = plan.tail;
  head.ctas = plan.ctas;
  tail.ctas = plan.ctas + 1;
  PagedArgs *parts[2] = {&head, &tail};
  for (int i = 0; i < 2; ++i) {
    parts[i]->sums = reinterpret_cast<float *>(w + l.off_sums[i]);
    parts[i]->mass = reinterpret_cast<float2 *>(w + l.off_mass[i]);
    parts[i]->loc = reinterpret_cast<int2 *>(w + l.off_loc[i]);
  }
  {
    PROF("prefix_plan");
    CK(launch_prefix_plan(tail, plan, head.loc, tail.loc, st));
  }
  TRY(run_attn(&l.groups, l.head, head, HEAD, st));
  TRY(run_attn(s, l.tail, tail, TAIL, st));
  PROF("prefix_join");
  CK(launch_prefix_join(head, tail, s->dtype == GDN_BF16, s->head_dim, l.head.MT, l.tail.MT, l.head.ctas, l.tail.ctas, st));
  return GDN_OK;
}

int gdn_prefix_attn_status(const gdn_paged_shape *s, int groups, int max_group, const void *ws, gdn_stream_t stream) {
  if (check_prefix(s, groups, max_group) || need_ptr(ws, "workspace")) return -1;
  const PrefixLayout l = prefix_layout(s, groups, max_group);
  if (cudaStreamSynchronize((Stream)stream) != cudaSuccess) return -1;
  if (s->total_q == 0 || s->num_seqs == 0) return 0;
  const int tail = attn_status_words(l.tail, static_cast<const char *>(ws) + l.off_tail);
  const int head = l.split ? attn_status_words(l.head, static_cast<const char *>(ws) + l.off_head) : 0;
  return tail < 0 || head < 0 ? -1 : tail | head;
}

int gdn_paged_attn_status(const gdn_paged_shape *s, const void *ws, gdn_stream_t stream) {
  if (check_attn(s) || need_ptr(ws, "workspace")) return -1;
  if (cudaStreamSynchronize((Stream)stream) != cudaSuccess) return -1;
  if (s->total_q == 0 || s->num_seqs == 0) return 0;
  return attn_status_words(attn_plan(s), ws);
}

int gdn_rotary_table(const double *freq, int pairs, int rows, double amplitude, float *table, gdn_stream_t stream) {
  if (pairs < 1 || rows < 0) return fail(GDN_ERR_INVALID_ARG, "need pairs >= 1, rows >= 0");
  if ((long long)pairs * rows > 0x7fffffffll * 64) return fail(GDN_ERR_UNSUPPORTED, "table too large");
  if (!std::isfinite(amplitude)) return fail(GDN_ERR_INVALID_ARG, "amplitude must be finite");
  if (rows == 0) return GDN_OK;
  TRY(need_ptr(freq, "freq"));
  TRY(need_aligned(table, "table"));
  const Stream st = (Stream)stream;
  PROF("rope_table");
  CK(launch_rope_table(freq, pairs, rows, amplitude, table, st));
  return GDN_OK;
}

int gdn_rotary(const gdn_rotary_shape *s, const void *q, const void *k, const float *table, const int32_t *positions,
               void *q_out, void *k_out, gdn_stream_t stream) {
  TRY(check_rotary(s));
  if (s->tokens == 0 || s->q_heads + s->k_heads == 0) return GDN_OK;
  TRY(check_rotary_args(s, q, k, table, positions, q_out, k_out));
  bool vec;
  const RopeArgs a = rotary_args(s, q, k, table, positions, q_out, k_out, vec);
  const Stream st = (Stream)stream;
  PROF("rope");
  CK(launch_rope(a, s->dtype == GDN_BF16, vec, st));
  return GDN_OK;
}

int gdn_rotary_append(const gdn_paged_shape *s, const void *q, const void *k, const void *v, const float *table,
                      void *k_cache, void *v_cache, const int32_t *page_table, const int32_t *cu_q,
                      const int32_t *kv_lens, void *q_out, gdn_stream_t stream) {
  TRY(check_append(s));
  if (s->total_q == 0 || s->num_seqs == 0) return GDN_OK;
  TRY(check_append_args(s, q, k, v, table, k_cache, v_cache, page_table, cu_q, kv_lens, q_out));
  bool vec;
  const RopeArgs a = append_args(s, q, k, v, table, k_cache, v_cache, page_table, cu_q, kv_lens, q_out, vec);
  const Stream st = (Stream)stream;
  PROF("rope_append");
  CK(launch_rope(a, s->dtype == GDN_BF16, vec, st));
  return GDN_OK;
}

int gdn_norm_rotary(const gdn_rotary_shape *s, float eps, float off, const void *q, const void *k, const float *wq, const float *wk,
                    const float *table, const int32_t *positions, void *q_out, void *k_out, gdn_stream_t stream) {
  TRY(check_rotary(s));
  TRY(check_head_norm(s->head_dim, s->inverse, eps, off));
  if (s->tokens == 0 || s->q_heads + s->k_heads == 0) return GDN_OK;
  TRY(check_rotary_args(s, q, k, table, positions, q_out, k_out));
  if (s->q_heads) TRY(need_ptr(wq, "q_weight"));
  if (s->k_heads) TRY(need_ptr(wk, "k_weight"));
  bool vec;
  NormRopeArgs n = {};
  n.r = rotary_args(s, q, k, table, positions, q_out, k_out, vec);
  n.w[0] = s->q_heads ? wq : wk;
  n.w[1] = s->q_heads && s->k_heads ? wk : nullptr;
  n.eps = eps;
  n.off = off;
  const Stream st = (Stream)stream;
  PROF("norm_rope");
  CK(launch_norm_rope(n, s->dtype == GDN_BF16, vec && head_in_warp(s->head_dim, s->dtype), st));
  return GDN_OK;
}

size_t gdn_norm_rotary_bwd_workspace_size(const gdn_rotary_shape *s) {
  if (check_rotary(s) || check_head_norm(s->head_dim, s->inverse, 1.f, 0.f)) return 0;
  return up256((size_t)norm_rope_bwd_ctas(s->tokens, s->q_heads + s->k_heads, num_sms()) * s->head_dim * sizeof(float));
}

int gdn_norm_rotary_bwd(const gdn_rotary_shape *s, float eps, float off, const void *dq_out, const void *dk_out, const void *q,
                        const void *k, const float *wq, const float *wk, const float *table, const int32_t *positions, void *dq, void *dk,
                        float *dwq, float *dwk, void *ws, size_t ws_bytes, gdn_stream_t stream) {
  TRY(check_rotary(s));
  TRY(check_head_norm(s->head_dim, s->inverse, eps, off));
  const Stream st = (Stream)stream;
  if (s->q_heads) TRY(need_ptr(dwq, "dq_weight"));
  if (s->k_heads) TRY(need_ptr(dwk, "dk_weight"));
  // a weight that no head takes has a gradient of zero
  const bool none = s->tokens == 0;
  if (dwq && (none || !s->q_heads)) CK(cudaMemsetAsync(dwq, 0, s->head_dim * sizeof(float), st));
  if (dwk && (none || !s->k_heads)) CK(cudaMemsetAsync(dwk, 0, s->head_dim * sizeof(float), st));
  if (none || s->q_heads + s->k_heads == 0) return GDN_OK;
  TRY(check_rotary_args(s, q, k, table, positions, dq, dk));
  if (s->q_heads) {
    TRY(need_ptr(dq_out, "dq_out"));
    TRY(need_ptr(wq, "q_weight"));
  }
  if (s->k_heads) {
    TRY(need_ptr(dk_out, "dk_out"));
    TRY(need_ptr(wk, "k_weight"));
  }
  if (s->q_heads && s->k_heads && dwq == dwk) return fail(GDN_ERR_INVALID_ARG, "dq_weight and dk_weight need memory of their own");
  const size_t need = gdn_norm_rotary_bwd_workspace_size(s);
  if (!ws || ws_bytes < need) return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
  TRY(need_aligned(ws, "workspace"));
  gdn_rotary_shape o = *s;  // of the outputs
  o.qo_tok = (int64_t)s->q_heads * s->head_dim;
  o.ko_tok = (int64_t)s->k_heads * s->head_dim;
  o.qo_head = o.ko_head = s->head_dim;
  bool vec;
  NormRopeArgs n = {};
  n.r = rotary_args(&o, q, k, table, positions, dq, dk, vec);
  n.r.inverse = 1;
  const int v = 16 / (int)esize(s->dtype);
  int g = 0;
  auto add = [&](const void *dy, int64_t tok, int64_t head, const float *w) {
    n.w[g] = w;
    n.dy[g] = dy;
    n.dy_tok[g] = tok;
    n.dy_head[g++] = head;
    vec = vec && aligned16(dy) && tok % v == 0 && head % v == 0;
  };
  if (s->q_heads) add(dq_out, s->qo_tok, s->qo_head, wq);
  if (s->k_heads) add(dk_out, s->ko_tok, s->ko_head, wk);
  n.eps = eps;
  n.off = off;
  n.part = static_cast<float *>(ws);
  PROF("norm_rope_bwd");
  CK(launch_norm_rope_bwd(n, s->dtype == GDN_BF16, vec && head_in_warp(s->head_dim, s->dtype),
                          norm_rope_bwd_ctas(s->tokens, s->q_heads + s->k_heads, num_sms()), s->q_heads ? dwq : dwk,
                          s->q_heads && s->k_heads ? dwk : nullptr, st));
  return GDN_OK;
}

int gdn_norm_rotary_append(const gdn_paged_shape *s, float eps, float off, const void *q, const void *k, const void *v, const float *wq,
                           const float *wk, const float *table, void *k_cache, void *v_cache, const int32_t *page_table,
                           const int32_t *cu_q, const int32_t *kv_lens, void *q_out, gdn_stream_t stream) {
  TRY(check_append(s));
  TRY(check_head_norm(s->head_dim, 0, eps, off));
  if (s->total_q == 0 || s->num_seqs == 0) return GDN_OK;
  TRY(check_append_args(s, q, k, v, table, k_cache, v_cache, page_table, cu_q, kv_lens, q_out));
  TRY(need_ptr(wq, "q_weight"));
  TRY(need_ptr(wk, "k_weight"));
  bool vec;
  NormRopeArgs n = {};
  n.r = append_args(s, q, k, v, table, k_cache, v_cache, page_table, cu_q, kv_lens, q_out, vec);
  n.w[0] = wq;
  n.w[1] = wk;
  n.eps = eps;
  n.off = off;
  const Stream st = (Stream)stream;
  PROF("norm_rope_append");
  CK(launch_norm_rope(n, s->dtype == GDN_BF16, vec && head_in_warp(s->head_dim, s->dtype), st));
  return GDN_OK;
}

int gdn_slots_copy(const gdn_slot_pool *pools, int num_pools, const int32_t *src, const int32_t *dst, int count, gdn_stream_t stream) {
  TRY(check_pools(pools, num_pools, "pools", 0));
  if (count < 0) return fail(GDN_ERR_INVALID_ARG, "count must be >= 0");
  if (count == 0 || num_pools == 0) return GDN_OK;
  TRY(need_ptr(src, "src"));
  TRY(need_ptr(dst, "dst"));
  const PairList pairs[2] = {{src, dst}, {src, dst}};
  return copy_slots(pools, num_pools, nullptr, 0, pairs, count, nullptr, TableJob{}, (Stream)stream);
}

size_t gdn_pages_workspace_size(const gdn_pages_shape *s, int m) {
  if (check_pages(s)) return 0;
  if (m < 0) {
    fail(GDN_ERR_INVALID_ARG, "m must be >= 0");
    return 0;
  }
  // extend: prefix [m + 1]; fork: src, parents, children and a list [m]; compact: map, src, dst [pages], two counts
  return up256(std::max((size_t)5 * m + 1, (size_t)3 * s->num_pages + 2) * 4);
}
#define CHECK_WS(need)                                                                                                   \
  if (!ws || ws_bytes < (need))                                                                                          \
    return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", (size_t)(need), ws ? ws_bytes : (size_t)0); \
  TRY(need_aligned(ws, "workspace"))

int gdn_pages_extend(const gdn_pages_shape *s, int32_t *table, int32_t *lens, int32_t *ref, const int32_t *seqs,
                     const int32_t *add, int m, int32_t *ok, void *ws, size_t ws_bytes, gdn_stream_t stream) {
  TRY(check_pages(s));
  if (m < 0) return fail(GDN_ERR_INVALID_ARG, "m must be >= 0");
  if (m == 0) return GDN_OK;
  TRY(need_ptr(table, "page_table"));
  TRY(need_ptr(lens, "seq_lens"));
  TRY(need_ptr(ref, "refcount"));
  TRY(need_ptr(seqs, "seqs"));
  TRY(need_ptr(add, "add"));
  TRY(need_ptr(ok, "ok"));
  CHECK_WS(gdn_pages_workspace_size(s, m));
  const Stream st = (Stream)stream;
  PROF("pages_extend");
  CK(launch_pages_extend(pages_args(s, table, lens, ref), seqs, add, m, ok, static_cast<int *>(ws), st));
  return GDN_OK;
}

int gdn_pages_fork(const gdn_pages_shape *s, int32_t *table, int32_t *lens, int32_t *ref, const int32_t *parents,
                   const int32_t *children, int m, const gdn_slot_pool *pools, int num_pools, const gdn_slot_pool *states,
                   int num_states, int32_t *new_page, void *ws, size_t ws_bytes, gdn_stream_t stream) {
  TRY(check_pages(s));
  TRY(check_pools(pools, num_pools, "pools", s->num_pages));
  TRY(check_pools(states, num_states, "states", s->num_seqs));
  if (m < 0) return fail(GDN_ERR_INVALID_ARG, "m must be >= 0");
  if (m == 0) return GDN_OK;
  TRY(need_ptr(table, "page_table"));
  TRY(need_ptr(lens, "seq_lens"));
  TRY(need_ptr(ref, "refcount"));
  TRY(need_ptr(parents, "parents"));
  TRY(need_ptr(children, "children"));
  TRY(need_ptr(new_page, "new_page"));
  CHECK_WS(gdn_pages_workspace_size(s, m));
  const Stream st = (Stream)stream;
  int *src = static_cast<int *>(ws), *psrc = src + m, *pdst = src + 2 * (size_t)m;
  const PagesArgs a = pages_args(s, table, lens, ref);
  {
    PROF("pages_fork_plan");
    CK(launch_pages_fork_plan(a, parents, children, m, new_page, src, psrc, pdst, st));
  }
  TableJob job = {};
  job.kind = TableJob::FORK;
  job.a = a;
  job.psrc = psrc;
  job.pdst = pdst;
  job.new_page = new_page;
  job.m = m;
  const PairList pairs[2] = {{src, new_page}, {psrc, pdst}};
  return copy_slots(pools, num_pools, states, num_states, pairs, m, nullptr, job, st);
}

int gdn_pages_free(const gdn_pages_shape *s, int32_t *table, int32_t *lens, int32_t *ref, const int32_t *seqs, int m, gdn_stream_t stream) {
  TRY(check_pages(s));
  if (m < 0) return fail(GDN_ERR_INVALID_ARG, "m must be >= 0");
  if (m == 0) return GDN_OK;
  TRY(need_ptr(table, "page_table"));
  TRY(need_ptr(lens, "seq_lens"));
  TRY(need_ptr(ref, "refcount"));
  TRY(need_ptr(seqs, "seqs"));
  const Stream st = (Stream)stream;
  PROF("pages_free");
  CK(launch_pages_free(pages_args(s, table, lens, ref), seqs, m, st));
  return GDN_OK;
}

int gdn_pages_compact(const gdn_pages_shape *s, const int32_t *table, const int32_t *ref, int32_t *table_out,
                      int32_t *ref_out, const gdn_slot_pool *pools, int num_pools, int32_t *moves, void *ws,
                      size_t ws_bytes, gdn_stream_t stream) {
  TRY(check_pages(s));
  TRY(check_pools(pools, num_pools, "pools", s->num_pages));
  TRY(need_ptr(table, "page_table"));
  TRY(need_ptr(ref, "refcount"));
  TRY(need_ptr(table_out, "page_table_out"));
  TRY(need_ptr(ref_out, "refcount_out"));
  CHECK_WS(gdn_pages_workspace_size(s, 0));
  const Stream st = (Stream)stream;
  int *map = static_cast<int *>(ws), *src = map + s->num_pages, *dst = src + s->num_pages, *count = dst + s->num_pages, *front = count + 1;
  if (!moves) moves = count;
  const PagesArgs a = pages_args(s, table_out, nullptr, ref_out);
  {
    PROF("pages_compact_plan");
    CK(launch_pages_compact_plan(a, ref, map, src, dst, moves, front, st));
  }
  TableJob job = {};
  job.kind = TableJob::REMAP;
  job.a = a;
  job.table_in = table;
  job.ref_in = ref;
  job.map = map;
  job.front = front;
  const PairList pairs[2] = {{src, dst}, {src, dst}};
  return copy_slots(pools, num_pools, nullptr, 0, pairs, s->num_pages / 2, moves, job, st);
}

int gdn_rmsnorm_fwd(const gdn_norm_shape *s, const void *x, const void *residual, const float *weight, void *h_out,
                    void *y, float *scale, float *rstd, gdn_stream_t stream) {
  TRY(check_norm(s, false));
  if (s->rows == 0) return GDN_OK;
  TRY(need_ptr(x, "x"));
  TRY(need_ptr(weight, "weight"));
  TRY(need_ptr(y, "y"));
  if (s->fp8) TRY(need_ptr(scale, "scale"));
  TRY(check_row(s->y_row, s, "y_row"));
  if (h_out) TRY(check_row(s->h_row, s, "h_row"));
  NormArgs a = {};
  a.x = x; a.res = residual; a.weight = weight; a.h_out = h_out; a.y = y; a.scale = scale; a.rstd = rstd;
  a.T = s->rows; a.D = s->dim; a.group = s->group; a.fp8 = s->fp8; a.eps = s->eps; a.off = s->weight_offset;
  a.x_row = s->x_row; a.r_row = s->r_row; a.h_row = s->h_row; a.y_row = s->y_row;
  const int v = 16 / (int)esize(s->dtype);
  const bool vec = s->dim % v == 0 && vec_ok(x, s->x_row, v) && vec_ok(residual, s->r_row, v) &&
                   vec_ok(h_out, s->h_row, v) && vec_ok(y, s->y_row, v) && aligned16(weight);
  const Stream st = (Stream)stream;
  PROF("rmsnorm_fwd");
  CK(launch_norm_fwd(a, s->dtype == GDN_BF16, vec, num_sms(), st));
  return GDN_OK;
}

static NormArgs bwd_args(const gdn_norm_shape *s, const void *dy, const void *h, const float *weight, const void *dh, void *dx, bool &vec) {
  NormArgs a = {};
  a.x = dy; a.h = h; a.weight = weight; a.res = dh; a.y = dx;
  a.T = s->rows; a.D = s->dim; a.off = s->weight_offset;
  a.x_row = s->x_row; a.r_row = s->r_row; a.h_row = s->h_row; a.y_row = s->y_row;
  const int v = 16 / (int)esize(s->dtype);
  vec = s->dim % v == 0 && vec_ok(dy, s->y_row, v) && vec_ok(h, s->x_row, v) && vec_ok(dh, s->r_row, v) &&
        vec_ok(dx, s->h_row, v) && aligned16(weight);
  return a;
}

size_t gdn_rmsnorm_bwd_workspace_size(const gdn_norm_shape *s) {
  if (check_norm(s, true)) return 0;
  return up256((size_t)num_sms() * 4 * s->dim * 4);  // one partial row of dw for each of at most four CTAs per SM
}

int gdn_rmsnorm_bwd(const gdn_norm_shape *s, const void *dy, const void *h, const float *weight, const float *rstd,
                    const void *dh, void *dx, float *dw, void *ws, size_t ws_bytes, gdn_stream_t stream) {
  TRY(check_norm(s, true));
  TRY(need_ptr(weight, "weight"));
  TRY(need_ptr(dw, "dw"));
  if (s->rows) {
    TRY(need_ptr(dy, "dy"));
    TRY(need_ptr(h, "h"));
    TRY(need_ptr(rstd, "rstd"));
    TRY(need_ptr(dx, "dx"));
    TRY(check_row(s->h_row, s, "h_row"));
  }
  CHECK_WS(gdn_rmsnorm_bwd_workspace_size(s));
  bool vec;
  NormArgs a = bwd_args(s, dy, h, weight, dh, dx, vec);
  a.rstd_in = rstd; a.dw = dw; a.part = static_cast<float *>(ws);
  const Stream st = (Stream)stream;
  PROF("rmsnorm_bwd");
  CK(launch_norm_bwd(a, s->dtype == GDN_BF16, vec, num_sms(), st));
  return GDN_OK;
}

int64_t gdn_scan_states_rows(const gdn_scan_shape *s) {
  if (check_scan(s)) return -1;
  return ((int64_t)s->tokens + SCAN_SEG - 1) / SCAN_SEG;
}

int gdn_scan_fwd(const gdn_scan_shape *s, const void *x, const void *g, const float *h0, const int32_t *cu, void *y, float *final,
                 float *states, gdn_stream_t stream) {
  TRY(check_scan(s));
  if (!cu && s->tokens % s->num_seqs) return fail(GDN_ERR_INVALID_ARG, "without cu_seqlens, tokens must be a multiple of num_seqs");
  TRY(check_scan_row(s->y_row, s, "y_row"));
  const Stream st = (Stream)stream;
  if (s->tokens == 0) return scan_no_tokens(s, h0, final, st);
  TRY(need_ptr(x, "x"));
  TRY(need_ptr(g, "g"));
  TRY(need_ptr(y, "y"));
  if (y == x || y == g) return fail(GDN_ERR_INVALID_ARG, "y is one of the inputs");
  if (final && final == h0) return fail(GDN_ERR_INVALID_ARG, "final is h0");
  ScanArgs a = scan_args(s, x, g, cu);
  a.y = y;
  a.h0 = h0;
  a.hT = final;
  a.states = states;
  const int e = (int)esize(s->dtype), eg = (int)esize(s->gate_dtype);
  Access m;
  m.add(x, s->x_row, e, s->dim);
  m.add(g, s->g_row, eg, s->dim);
  m.add(y, s->y_row, e, s->dim);
  PROF("scan_fwd");
  CK(launch_scan(a, s->dtype == GDN_BF16, s->gate_dtype == GDN_BF16, scan_move(m, s, {h0, final, states}), false, num_sms(), st));
  return GDN_OK;
}

int gdn_scan_bwd(const gdn_scan_shape *s, const void *dy, const void *x, const void *g, const float *states, const float *h0,
                 const float *d_final, const int32_t *cu, void *dx, void *dg, float *dh0, gdn_stream_t stream) {
  TRY(check_scan(s));
  if (!cu && s->tokens % s->num_seqs) return fail(GDN_ERR_INVALID_ARG, "without cu_seqlens, tokens must be a multiple of num_seqs");
  TRY(check_scan_row(s->y_row, s, "y_row"));
  TRY(check_scan_row(s->dg_row, s, "dg_row"));
  const Stream st = (Stream)stream;
  if (s->tokens == 0) return scan_no_tokens(s, d_final, dh0, st);
  TRY(need_ptr(dy, "dy"));
  TRY(need_ptr(x, "x"));
  TRY(need_ptr(g, "g"));
  TRY(need_ptr(states, "states"));
  TRY(need_ptr(dx, "dx"));
  TRY(need_ptr(dg, "dg"));
  if (dx == dg || dx == dy || dx == x || dx == g || dg == dy || dg == x || dg == g)
    return fail(GDN_ERR_INVALID_ARG, "dx and dg need memory of their own");
  if (dh0 && (dh0 == d_final || dh0 == h0)) return fail(GDN_ERR_INVALID_ARG, "dh0 is one of the inputs");
  ScanArgs a = scan_args(s, x, g, cu);
  a.dy = dy;
  a.y = dx;
  a.dg = dg;
  a.h0 = h0;
  a.dhT = d_final;
  a.dh0 = dh0;
  a.states = const_cast<float *>(states);
  const int e = (int)esize(s->dtype), eg = (int)esize(s->gate_dtype);
  Access m;
  m.add(x, s->x_row, e, s->dim);
  m.add(dy, s->dy_row, e, s->dim);
  m.add(g, s->g_row, eg, s->dim);
  m.add(dx, s->y_row, e, s->dim);
  m.add(dg, s->dg_row, eg, s->dim);
  PROF("scan_bwd");
  CK(launch_scan(a, s->dtype == GDN_BF16, s->gate_dtype == GDN_BF16, scan_move(m, s, {h0, d_final, dh0, states}), true, num_sms(), st));
  return GDN_OK;
}

int gdn_scan_step(const gdn_scan_shape *s, const void *x, const void *g, float *state, void *y, gdn_stream_t stream) {
  TRY(check_scan(s));
  if (s->tokens != s->num_seqs) return fail(GDN_ERR_INVALID_ARG, "a step takes one token of each sequence");
  TRY(check_scan_row(s->y_row, s, "y_row"));
  TRY(check_scan_row(s->state_row, s, "state_row"));
  TRY(need_ptr(x, "x"));
  TRY(need_ptr(g, "g"));
  TRY(need_ptr(state, "state"));
  TRY(need_ptr(y, "y"));
  if (y == x || y == g || y == state || state == x || state == g) return fail(GDN_ERR_INVALID_ARG, "y and state need memory of their own");
  ScanArgs a = scan_args(s, x, g, nullptr);
  a.y = y;
  a.hT = state;
  auto four = [&](const void *p, int64_t row, size_t es) { return reinterpret_cast<uintptr_t>(p) % (4 * es) == 0 && row % 4 == 0; };
  const bool vec = s->dim % 4 == 0 && four(x, s->x_row, esize(s->dtype)) && four(g, s->g_row, esize(s->gate_dtype)) &&
                   four(y, s->y_row, esize(s->dtype)) && four(state, s->state_row, 4);
  const Stream st = (Stream)stream;
  PROF("scan_step");
  CK(launch_scan_step(a, s->dtype == GDN_BF16, s->gate_dtype == GDN_BF16, vec, st));
  return GDN_OK;
}

}  // extern "C"
