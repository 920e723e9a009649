// Attention of a few query rows per key head over a paged cache (decoding, drafted tokens, and every fp32 call):
//   o_r = sum_j p_rj v_j,  p_rj = exp2(z_rj - max) / sum,  z = scale log2(e) q_r . k_j.
// Background of the softmax layer in a hybrid stack: onedev.kr summary of the FlashQLA talk, linear-attention
// background paragraph.
//
// Bound by the bytes of the cache: each key and value is used by MT = 16 or 32 rows only (16 flops per byte at four
// query heads per key head), far below the tensor cores' ratio.  So the kernel is a stream: the units of the whole
// batch are split evenly over the CTAs (paged.cuh), and inside a CTA each of the four warps owns a 16-token slice of
// every 64-token block with its own ring of cp.async stages, its own running maximum, mass and sums, and no barrier
// with the other warps until the piece ends.  The query rows stay in registers as mma.sync A fragments; scores come
// out in the layout that the second product takes as its A operand.  tcgen05 has no use here: its 128-row tile would
// be one eighth full, and the softmax would leave registers for TMEM and come back.
//
// The sums are rescaled only when a row's maximum rises by more than 8 (a factor of 256 that fp32 sums and bf16
// weights carry without loss), so most slices skip that pass over the accumulator.
//
// fp32: every product as three TF32 mma.sync parts, x = hi + lo (hi rounded to 11 bits, lo the exact rest):
// hi hi + hi lo + lo hi leaves about 2^-21 of a product.
#include "paged.cuh"

namespace gdn {

namespace {

constexpr int WARPS = 4, NT = WARPS * 32, SL = 16, BN = WARPS * SL;
constexpr float RAISE = 8.f;  // log2 of the growth of a row's maximum that is left in its weights

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
template <int K> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(K) : "memory"); }

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;  // to 11 significant bits, halves away from zero
  lo = __float_as_uint(x - __uint_as_float(hi));
}
// c += a b with both operands in two TF32 parts
__device__ __forceinline__ void mma_3tf32(float (&c)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], float b0, float b1) {
  uint32_t h0, l0, h1, l1;
  split_tf32(b0, h0, l0);
  split_tf32(b1, h1, l1);
  mma_tf32(c, al, h0, h1);
  mma_tf32(c, ah, l0, l1);
  mma_tf32(c, ah, h0, h1);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// byte offset of 16-byte chunk c of row r in a [16][D] slice: chunks of a row change places by the row's low three
// bits, so that eight rows at one column lie in eight different bank groups
template <int RB> __device__ __forceinline__ uint32_t slice_off(int r, int c) { return r * RB + ((c ^ (r & 7)) << 4); }

}  // namespace

template <typename I, int D, int MI, int STAGES>
__global__ void __launch_bounds__(NT, (sizeof(I) == 2 ? 2 : 1)) attn_rows_kernel(PagedArgs a) {
  constexpr int MT = 16 * MI, RB = D * sizeof(I), CPR = RB / 16, SLB = SL * RB;  // row bytes, chunks, slice bytes
  constexpr bool F32 = sizeof(I) == 4;
  constexpr int KS = F32 ? D / 8 : D / 16;  // k steps of q . k
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long pre[2][NT + 1];
  __shared__ long long scan_sh[NT / 32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, qd = lane & 3;
  const int cta = blockIdx.x;
  const int P = 1 << a.log2P;
  int used = 0;  // record slots written
  Cursor cur;
  bool more = cursor_begin<NT, MT, BN>(a, cur, pre, scan_sh);
  uint8_t *ring = smem + warp * (STAGES * 2 * SLB);
  const uint32_t ring_u = smem_u32(ring);
  const I *Q = static_cast<const I *>(a.q);
  const char *Kb = static_cast<const char *>(a.k), *Vb = static_cast<const char *>(a.v);

  while (more) {
    int b0, b1;
    bool first, last;
    const int n = cursor_piece(cur, b0, b1, first, last);
    const Tile w = cur.w;
    // ---- the slices of this piece: lane l copies chunks l, l + 32, ... of the keys and of the values
    const int *trow = a.table + (long long)cur.n * a.table_stride;
    auto page_of = [&](int b) {  // page of the warp's slice of block b, -1 where nothing is to be read
      const int t0 = (w.blk0 + b) * BN + warp * SL;
      if (b >= b1 || t0 >= w.hi || t0 + SL <= w.lo) return -1;
      const int pg = trow[t0 >> a.log2P];
      return (unsigned)pg < (unsigned)a.num_pages ? pg : -1;
    };
    auto issue = [&](int b, int pg, int stage) {
      const int t0 = (w.blk0 + b) * BN + warp * SL;
      if (b < b1) {
        const long long kb = ((long long)max(pg, 0) * a.k_page + (long long)(t0 & (P - 1)) * a.k_tok + cur.h * a.k_head) * (int)sizeof(I);
        const long long vb = ((long long)max(pg, 0) * a.v_page + (long long)(t0 & (P - 1)) * a.v_tok + cur.h * a.v_head) * (int)sizeof(I);
        uint8_t *ks = ring + stage * 2 * SLB, *vs = ks + SLB;
#pragma unroll
        for (int i = 0; i < SLB / 512; ++i) {
          const int r = (lane + 32 * i) / CPR, c = (lane + 32 * i) % CPR;
          const bool ok = pg >= 0 && t0 + r >= w.lo && t0 + r < w.hi;  // other slots read as zeros
          const int rr = ok ? r : 0;
          cp_async16(ks + slice_off<RB>(r, c), Kb + kb + (rr * a.k_tok * (int)sizeof(I) + c * 16), ok);
          cp_async16(vs + slice_off<RB>(r, c), Vb + vb + (rr * a.v_tok * (int)sizeof(I) + c * 16), ok);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) issue(b0 + s, page_of(b0 + s), s);
    int pg_next = page_of(b0 + STAGES - 1);

    // ---- query fragments: rows g and g + 8 of each 16-row tile
    uint32_t qf[MI][KS][4];
    int pos[MI][2];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 16 * i + g + 8 * e;
        const bool ok = r < w.rows;
        int tok, head;
        row_place(a, cur, MT, ok ? r : 0, tok, head);
        pos[i][e] = cur.s.kv - cur.s.qlen + tok - cur.s.qbeg;
        const I *p = Q + tok * a.q_tok + head * a.q_head;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          if constexpr (F32) {
            qf[i][k][e] = ok ? __float_as_uint(p[8 * k + qd]) : 0u;
            qf[i][k][e + 2] = ok ? __float_as_uint(p[8 * k + qd + 4]) : 0u;
          } else {
            qf[i][k][e] = ok ? *reinterpret_cast<const uint32_t *>(p + 16 * k + 2 * qd) : 0u;
            qf[i][k][e + 2] = ok ? *reinterpret_cast<const uint32_t *>(p + 16 * k + 2 * qd + 8) : 0u;
          }
        }
      }
    const int pos_last = cur.s.kv - cur.s.qlen + (int)(((long long)cur.t * MT + w.rows - 1) / a.G);

    float acc[MI][D / 8][4], m[MI][2], l[MI][2];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
    }

    int stage = 0;
    for (int b = b0; b < b1; ++b) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();
      {
        const int nx = stage == 0 ? STAGES - 1 : stage - 1;
        issue(b + STAGES - 1, pg_next, nx);
        pg_next = page_of(b + STAGES);
      }
      const uint32_t ks = ring_u + stage * 2 * SLB, vs = ks + SLB;
      const uint8_t *vsp = ring + stage * 2 * SLB + SLB, *ksp = ring + stage * 2 * SLB;
      stage = stage == STAGES - 1 ? 0 : stage + 1;
      const int t0 = (w.blk0 + b) * BN + warp * SL;
      if (t0 >= w.hi || t0 + SL <= w.lo) continue;
      // ---- scores of 16 tokens: tiles 0 (tokens 0-7) and 1 (8-15)
      float s[MI][2][4];
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][j][e] = 0.f;
      if constexpr (!F32) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t bk[4];
          const uint32_t ad = ks + slice_off<RB>((lane & 7) + 8 * (lane >> 4), 2 * k + ((lane >> 3) & 1));
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                       : "=r"(bk[0]), "=r"(bk[1]), "=r"(bk[2]), "=r"(bk[3]) : "r"(ad) : "memory");
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            mma_bf16(s[i][0], qf[i][k], bk[0], bk[1]);
            mma_bf16(s[i][1], qf[i][k], bk[2], bk[3]);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          float bk[2][2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              bk[j][e] = *reinterpret_cast<const float *>(ksp + slice_off<RB>(g + 8 * j, 2 * k + e) + qd * 4);
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            uint32_t ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split_tf32(__uint_as_float(qf[i][k][e]), ah[e], al[e]);
#pragma unroll
            for (int j = 0; j < 2; ++j) mma_3tf32(s[i][j], ah, al, bk[j][0], bk[j][1]);
          }
        }
      }
      // ---- softmax: thread holds rows g, g + 8 (e >> 1), tokens 8 j + 2 qd + (e & 1)
      const bool mask = t0 + SL - 1 > w.pos0 || (a.window && t0 < pos_last - a.window + 1);
      float mx[MI][2];
      bool raise = false;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float z = s[i][j][e] * a.scale_log2;
            if (mask) {
              const int key = t0 + 8 * j + 2 * qd + (e & 1), p = pos[i][e >> 1];
              if (key > p || (a.window && key <= p - a.window)) z = -INFINITY;
            }
            s[i][j][e] = z;
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[i][e] = quad_max(fmaxf(fmaxf(s[i][0][2 * e], s[i][0][2 * e + 1]), fmaxf(s[i][1][2 * e], s[i][1][2 * e + 1])));
          raise |= mx[i][e] > m[i][e] + RAISE;
        }
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mn = fmaxf(m[i][e], mx[i][e]);
            const float f = mn == -INFINITY ? 1.f : ex2(m[i][e] - mn);
            m[i][e] = mn;
            l[i][e] *= f;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
              acc[i][j][2 * e] *= f;
              acc[i][j][2 * e + 1] *= f;
            }
          }
      }
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mm = m[i][e] == -INFINITY ? 0.f : m[i][e];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float p = ex2(s[i][j][2 * e + x] - mm);
              l[i][e] += p;
              s[i][j][2 * e + x] = p;
            }
        }
      // ---- sums += weights x values
      if constexpr (!F32) {
        uint32_t pa[MI][4];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          pa[i][0] = pack2(s[i][0][0], s[i][0][1]);
          pa[i][1] = pack2(s[i][0][2], s[i][0][3]);
          pa[i][2] = pack2(s[i][1][0], s[i][1][1]);
          pa[i][3] = pack2(s[i][1][2], s[i][1][3]);
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          uint32_t bv[4];
          const uint32_t ad = vs + slice_off<RB>((lane & 7) + 8 * ((lane >> 3) & 1), 2 * j + (lane >> 4));
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                       : "=r"(bv[0]), "=r"(bv[1]), "=r"(bv[2]), "=r"(bv[3]) : "r"(ad) : "memory");
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            mma_bf16(acc[i][2 * j], pa[i], bv[0], bv[1]);
            mma_bf16(acc[i][2 * j + 1], pa[i], bv[2], bv[3]);
          }
        }
      } else {
        // the 8 tokens of score tile jt are the k of one step: index qd is token 2 qd and qd + 4 is token 2 qd + 1,
        // in the weights (as the scores came out) and in the values alike
#pragma unroll
        for (int jt = 0; jt < 2; ++jt) {
          uint32_t ph[MI][4], pl[MI][4];
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            split_tf32(s[i][jt][0], ph[i][0], pl[i][0]);
            split_tf32(s[i][jt][2], ph[i][1], pl[i][1]);
            split_tf32(s[i][jt][1], ph[i][2], pl[i][2]);
            split_tf32(s[i][jt][3], ph[i][3], pl[i][3]);
          }
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            const int r = 8 * jt + 2 * qd, c = 2 * j + (g >> 2);
            const float v0 = *reinterpret_cast<const float *>(vsp + slice_off<RB>(r, c) + (g & 3) * 4);
            const float v1 = *reinterpret_cast<const float *>(vsp + slice_off<RB>(r + 1, c) + (g & 3) * 4);
#pragma unroll
            for (int i = 0; i < MI; ++i) mma_3tf32(acc[i][j], ph[i], pl[i], v0, v1);
          }
        }
      }
    }
    cp_async_wait_all();
    __syncthreads();

    // ---- the four warps' sums meet in shared memory (over the rings, which are empty)
    float *om = reinterpret_cast<float *>(smem) + warp * (MT * (D + 2));
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 16 * i + g + 8 * e;
        const float ls = quad_sum(l[i][e]);
        if (qd == 0) {
          om[MT * D + r] = m[i][e];
          om[MT * D + MT + r] = ls;
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
          *reinterpret_cast<float2 *>(om + r * D + 8 * j + 2 * qd) = make_float2(acc[i][j][2 * e], acc[i][j][2 * e + 1]);
      }
    __syncthreads();
    constexpr int LPR = D / 4;  // lanes of a row
    const float *all = reinterpret_cast<const float *>(smem);
    const int slot = first ? 1 : 0;
    float *rec = a.part + ((long long)cta * 2 + slot) * record_floats(MT, D);
    for (int r = warp * (32 / LPR) + lane / LPR; r < w.rows; r += WARPS * (32 / LPR)) {
      const int c = lane % LPR;
      float mw[WARPS], M = -INFINITY;
#pragma unroll
      for (int x = 0; x < WARPS; ++x) {
        mw[x] = all[x * (MT * (D + 2)) + MT * D + r];
        M = fmaxf(M, mw[x]);
      }
      float L = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < WARPS; ++x) {
        const float f = mw[x] == -INFINITY ? 0.f : ex2(mw[x] - M);
        const float *base = all + x * (MT * (D + 2));
        const float4 v = *reinterpret_cast<const float4 *>(base + r * D + 4 * c);
        L += f * base[MT * D + MT + r];
        o.x += f * v.x;
        o.y += f * v.y;
        o.z += f * v.z;
        o.w += f * v.w;
      }
      if (first && last) {
        int tok, head;
        row_place(a, cur, MT, r, tok, head);
        const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // nothing seen: zeros; a NaN stays
        I *op = static_cast<I *>(a.o) + tok * a.o_tok + head * a.o_head + 4 * c;
        if constexpr (F32) {
          *reinterpret_cast<float4 *>(op) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        } else {
          *reinterpret_cast<uint2 *>(op) = make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv));
        }
        if (a.lse && c == 0)
          a.lse[(long long)tok * a.Hq + head] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      } else {
        *reinterpret_cast<float4 *>(rec + r * D + 4 * c) = o;
        if (c == 0) {
          rec[MT * D + r] = M;
          rec[MT * D + MT + r] = L;
        }
      }
    }
    if (!(first && last)) {
      used |= 1 << slot;
      if (tid == 0) {
        const long long r0 = (long long)cur.t * MT;
        a.hdr[cta * 2 + slot] = make_int4(last ? 1 : 2, cur.s.qbeg + (int)(r0 / a.G), cur.h, w.rows << 16 | (int)(r0 % a.G));
      }
    }
    more = cursor_next<MT, BN>(a, cur, n);
    __syncthreads();
  }
  if (tid < 2 && !(used >> tid & 1)) a.hdr[cta * 2 + tid] = make_int4(0, 0, 0, 0);
}

// Joins the pieces of cut items.  Block (c, y): the item that began in CTA c and went on; its warps take rows
// y * 4 + warp, + 4 gridDim.y, ...  A row's pieces are weighted by their maxima and added in the order of the CTAs.
template <typename I, int D>
__global__ void __launch_bounds__(128) attn_join_kernel(PagedArgs a, int MT, int C) {
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 h = a.hdr[c * 2 + 1];
  if (h.x != 2) return;
  const int rows = h.w >> 16, gr = h.w & 0xffff;
  // the piece after CTA c's own is slot 0 of c + 1, and so on until one that ends the item
  int np = 0;
  for (int x = c + 1; x < C; x += 32) {
    const bool end = x + lane < C && a.hdr[(x + lane) * 2].x != 2;
    const unsigned b = __ballot_sync(0xffffffffu, end);
    if (b) {
      np = x + __ffs(b) - 1 - c + 1;
      break;
    }
  }
  if (np == 0) np = C - c;
  const size_t rf = record_floats(MT, D);
  auto rec = [&](int i) { return a.part + ((long long)(c + i) * 2 + (i == 0 ? 1 : 0)) * rf; };
  for (int r = blockIdx.y * 4 + warp; r < rows; r += 4 * gridDim.y) {
    float M = -INFINITY;
    for (int i = lane; i < np; i += 32) M = fmaxf(M, rec(i)[(size_t)MT * D + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f, o[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int i = 0; i < np; ++i) {
      const float *p = rec(i);
      const float mi = p[(size_t)MT * D + r], li = p[(size_t)MT * D + MT + r];
      const float f = mi == -INFINITY ? 0.f : ex2(mi - M);
      L += f * li;
      if constexpr (D == 128) {
        const float4 v = *reinterpret_cast<const float4 *>(p + (size_t)r * D + 4 * lane);
        o[0] += f * v.x; o[1] += f * v.y; o[2] += f * v.z; o[3] += f * v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2 *>(p + (size_t)r * D + 2 * lane);
        o[0] += f * v.x; o[1] += f * v.y;
      }
    }
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    const int tok = h.y + (gr + r) / a.G, head = h.z * a.G + (gr + r) % a.G;
    I *op = static_cast<I *>(a.o) + tok * a.o_tok + head * a.o_head + (D / 32) * lane;
#pragma unroll
    for (int e = 0; e < D / 32; e += 2) st2(op + e, o[e] * inv, o[e + 1] * inv);
    if (a.lse && lane == 0)
      a.lse[(long long)tok * a.Hq + head] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
}

namespace {
template <typename I, int D, int MI, int STAGES> cudaError_t launch_rows(const PagedArgs &a, int ctas, cudaStream_t st) {
  constexpr size_t ring = (size_t)WARPS * STAGES * 2 * SL * D * sizeof(I);
  constexpr size_t meet = (size_t)WARPS * record_floats(16 * MI, D) * 4;
  constexpr size_t smem = ring > meet ? ring : meet;
  auto *k = attn_rows_kernel<I, D, MI, STAGES>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(ctas), dim3(NT), smem, st, a);
}
}  // namespace

// bf16: rings of 96 KB, so that two CTAs share an SM; fp32: 16 rows, and 96 KB (D = 64) or 192 KB rings
cudaError_t launch_attn_rows(const PagedArgs &a, bool bf, int D, int MT, int ctas, cudaStream_t st) {
  if (!bf) return D == 64 ? launch_rows<float, 64, 1, 3>(a, ctas, st) : launch_rows<float, 128, 1, 3>(a, ctas, st);
  if (D == 64) return MT == 16 ? launch_rows<bf16, 64, 1, 6>(a, ctas, st) : launch_rows<bf16, 64, 2, 6>(a, ctas, st);
  return MT == 16 ? launch_rows<bf16, 128, 1, 3>(a, ctas, st) : launch_rows<bf16, 128, 2, 3>(a, ctas, st);
}

cudaError_t launch_attn_join(const PagedArgs &a, bool bf, int D, int MT, int ctas, cudaStream_t st) {
  const dim3 grid(ctas, MT <= 32 ? MT / 4 : 16);
  if (bf)
    return D == 64 ? launch_pdl(attn_join_kernel<bf16, 64>, grid, dim3(128), 0, st, a, MT, ctas)
                   : launch_pdl(attn_join_kernel<bf16, 128>, grid, dim3(128), 0, st, a, MT, ctas);
  return D == 64 ? launch_pdl(attn_join_kernel<float, 64>, grid, dim3(128), 0, st, a, MT, ctas)
                 : launch_pdl(attn_join_kernel<float, 128>, grid, dim3(128), 0, st, a, MT, ctas);
}

}  // namespace gdn
