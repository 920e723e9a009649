// The row kernel of every key that a query sees, the choice among its variants, and the join of cut items.
#include "attn_rows.cuh"

namespace gdn {

extern template cudaError_t launch_attn_rows_part<SINKS>(const PagedArgs &, const CUtensorMap &, const CUtensorMap &, bool, int, int, int, cudaStream_t);
extern template cudaError_t launch_attn_rows_part<HEAD>(const PagedArgs &, const CUtensorMap &, const CUtensorMap &, bool, int, int, int, cudaStream_t);
extern template cudaError_t launch_attn_rows_part<TAIL>(const PagedArgs &, const CUtensorMap &, const CUtensorMap &, bool, int, int, int, cudaStream_t);
template cudaError_t launch_attn_rows_part<ALL>(const PagedArgs &, const CUtensorMap &, const CUtensorMap &, bool, int, int, int, cudaStream_t);

// Joins the pieces of cut items.  Block (j, y): rows of the j-th of them, which began in some CTA c and went on in the
// next ones (the block looks for c in the headers, so that the grid need not be larger than the number of items), a row
// of every gridDim.y, or four neighbours where a warp has one for itself.  JW warps share a row (8 or 4 where few items are
// cut into many pieces each, 1 where many are cut into a few): each takes every JW-th batch of pieces (JW, or 2 where a
// warp has the row alone and there are seldom more: 2048 new tokens after 8192 take 6 us less than with 8), asks for all of
// a batch before it uses any, and weights the batch by the running maximum; the warps' results meet in shared memory.  The
// order of the sums is fixed.
template <typename I, int D, int JW>
__global__ void __launch_bounds__(JW == 1 ? 128 : 32 * JW) attn_join_kernel(PagedArgs a, int MT, int C) {
  constexpr int WARPS = JW == 1 ? 4 : JW, RW = WARPS / JW, E = D / 32, BATCH = JW == 1 ? 2 : JW;
  __shared__ float sh[WARPS][32 * E + 2];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int c = -1, left = blockIdx.x;
  if ((int)gridDim.x == C) c = left;  // as many blocks as CTAs: no search
  for (int b = 0; b < C && c < 0; b += 256) {
    int x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = b + 32 * i + lane < C ? a.hdr[b + 32 * i + lane].x : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const unsigned m = __ballot_sync(0xffffffffu, x[i] != 0);
      const unsigned me = __ballot_sync(0xffffffffu, x[i] != 0 && __popc(m & ((1u << lane) - 1)) == left);
      if (c < 0 && me) c = b + 32 * i + __ffs(me) - 1;
      left -= __popc(m);
    }
  }
  if (c < 0) return;
  const int4 h = a.hdr[c];
  const int np = h.x, rows = h.w >> 16, gr = h.w & 0xffff;
  const int sub = warp % JW;
  if (np == 0) return;
  const long long rf = (long long)record_floats(MT, D);
  // piece 0 is slot 1 of CTA c, piece i slot 0 of CTA c + i
  const float *p0 = a.part + ((long long)c * 2 + 1) * rf, *p1 = a.part + (long long)c * 2 * rf;
  for (int r0 = blockIdx.y * RW; r0 < rows; r0 += gridDim.y * RW) {
    const int r = r0 + warp / JW;
    float M = -INFINITY, L = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    if (r < rows) {
      for (int b = sub * BATCH; b < np; b += JW * BATCH) {
        float m[BATCH], l[BATCH], v[BATCH][E];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          m[i] = -INFINITY;
          l[i] = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) v[i][e] = 0.f;
          if (b + i < np) {
            const float *p = b + i == 0 ? p0 : p1 + (b + i) * 2 * rf;
            m[i] = p[MT * D + r];
            l[i] = p[MT * D + MT + r];
            if constexpr (D == 128) {
              const float4 t = *reinterpret_cast<const float4 *>(p + r * D + 4 * lane);
              v[i][0] = t.x; v[i][1] = t.y; v[i][2] = t.z; v[i][3] = t.w;
            } else {
              const float2 t = *reinterpret_cast<const float2 *>(p + r * D + 2 * lane);
              v[i][0] = t.x; v[i][1] = t.y;
            }
          }
        }
        float mn = M;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) mn = fmaxf(mn, m[i]);
        // Nothing seen yet: every factor below is 0.  M stays -inf then: a row whose first pieces lie outside its window
        // may have its maximum far below 0.
        const float ref = mn == -INFINITY ? 0.f : mn;
        float f = ex2(M - ref);
        L *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          f = ex2(m[i] - ref);
          L += f * l[i];
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] += f * v[i][e];
        }
        M = mn;
      }
    }
    if constexpr (JW > 1) {
      if (lane == 0) {
        sh[warp][32 * E] = M;
        sh[warp][32 * E + 1] = L;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) sh[warp][E * lane + e] = o[e];
      __syncthreads();
      float mw[JW], mn = -INFINITY;
#pragma unroll
      for (int w = 0; w < JW; ++w) {
        mw[w] = sh[w][32 * E];
        mn = fmaxf(mn, mw[w]);
      }
      const float ref = mn == -INFINITY ? 0.f : mn;
      L = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
      for (int w = 0; w < JW; ++w) {
        const float f = ex2(mw[w] - ref);
        L += f * sh[w][32 * E + 1];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += f * sh[w][E * lane + e];
      }
      M = mn;
      __syncthreads();  // all have read
    }
    if (r >= rows || sub != 0) continue;
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // nothing seen: zeros; a NaN stays
    const int tok = h.y + (gr + r) / a.G, head = h.z * a.G + (gr + r) % a.G;
    I *op = static_cast<I *>(a.o) + tok * a.o_tok + head * a.o_head + E * lane;
#pragma unroll
    for (int e = 0; e < E; e += 2) st2(op + e, o[e] * inv, o[e + 1] * inv);
    if (a.lse && lane == 0) a.lse[(long long)tok * a.Hq + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
}

// 16 rows a tile where that is enough, and in fp32 with D = 64 always: 96 KB of rings (fp32, D = 128: 192 KB) and then two
// CTAs per SM.  More rows: two row groups and 192 KB of rings, so that a key or value is fetched and, in fp32, split into
// its two parts half as often (fp32: D = 64, 8 sequences of up to 256 new tokens: 44 us with 16 rows, 47 us with 32, the last
// 1024 of 4096 tokens: 313 and 324 us; D = 128, 512 new tokens after 3584: 530 us with 16 rows, 317 us with 32; both sides
// before the guard in split_tf32, which adds 1 to 3 %).
int attn_rows_tile(bool bf, int D, int rows) { return rows <= 16 || (!bf && D == 64) ? 16 : 32; }
int attn_rows_box(bool bf, int MT, int page) { return bf && MT == 32 && page >= 32 ? 32 : 16; }
int attn_rows_block(bool bf, int MT) { return bf && MT == 32 ? 128 : 64; }
int attn_rows_per_sm(bool bf, int D, int MT) { return MT == 16 && (bf || D == 64) ? 2 : 1; }
cudaError_t launch_attn_rows(const PagedArgs &a, Part part, const CUtensorMap &tk, const CUtensorMap &tv, bool bf, int D, int MT, int ctas,
                             cudaStream_t st) {
  switch (part) {
    case ALL: return launch_attn_rows_part<ALL>(a, tk, tv, bf, D, MT, ctas, st);
    case SINKS: return launch_attn_rows_part<SINKS>(a, tk, tv, bf, D, MT, ctas, st);
    case HEAD: return launch_attn_rows_part<HEAD>(a, tk, tv, bf, D, MT, ctas, st);
    default: return launch_attn_rows_part<TAIL>(a, tk, tv, bf, D, MT, ctas, st);
  }
}

namespace {
template <typename I, int D> cudaError_t launch_join(const PagedArgs &a, int MT, int ctas, int items, cudaStream_t st) {
  const int n = items < ctas ? items : ctas;  // cut items at most
  // Row blocks of an item, each of which walks over rows: in all as many as there is room for at once, since starting a
  // block costs more than a row (one sequence, 64 new tokens, 16 items of 256 rows: 43 us with 32 blocks to an item, 35
  // with 64, 38 with 256; 32 new tokens, 8 items: 29 us with 64, 20 with 256).
  const int rows = std::min(MT, std::max(16, 152 * 8 / n));
  // few items: many pieces each (8 new tokens of 8 sequences, fp32, 32 items on 304 CTAs: 14.8 us with four warps to a
  // row, 18.3 with one)
  if (items * 8 <= ctas) return launch_pdl(attn_join_kernel<I, D, 8>, dim3(n, rows), dim3(256), 0, st, a, MT, ctas);
  if (items * 4 <= ctas) return launch_pdl(attn_join_kernel<I, D, 4>, dim3(n, rows), dim3(128), 0, st, a, MT, ctas);
  return launch_pdl(attn_join_kernel<I, D, 1>, dim3(n, std::min((MT + 3) / 4, 32)), dim3(128), 0, st, a, MT, ctas);
}
}  // namespace

cudaError_t launch_attn_join(const PagedArgs &a, bool bf, int D, int MT, int ctas, int items, cudaStream_t st) {
  if (bf) return D == 64 ? launch_join<bf16, 64>(a, MT, ctas, items, st) : launch_join<bf16, 128>(a, MT, ctas, items, st);
  return D == 64 ? launch_join<float, 64>(a, MT, ctas, items, st) : launch_join<float, 128>(a, MT, ctas, items, st);
}

}  // namespace gdn
