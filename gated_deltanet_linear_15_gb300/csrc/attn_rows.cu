// Attention of a few query rows per key head over a paged cache (decoding, drafted tokens, and every fp32 call):
//   o_r = sum_j p_rj v_j,  p_rj = exp2(z_rj - max) / sum,  z = scale log2(e) q_r . k_j.
// Background of the softmax layer in a hybrid stack: onedev.kr summary of the FlashQLA talk, linear-attention
// background paragraph.
//
// Bound by the bytes of the cache: each key and value is used by a few rows only (16 flops per byte at four query heads
// per key head), far below the tensor cores' ratio.  So the kernel is a stream: the units of the whole batch are split
// evenly over the CTAs (paged.cuh), and a CTA's blocks are cut into four slices of 16 NS tokens.  A slice belongs to RG
// warps, each with 16 of the tile's rows (MT = 16 RG), and has its own ring of TMA stages; every warp has its own running
// maximum, mass and sums, and meets the other slices only when the piece ends.  The query rows stay in registers as
// mma.sync A fragments; scores come out in the layout that the second product takes as its A operand.  tcgen05 has no use
// here: its 128-row tile would be an eighth full, and the softmax would leave registers for TMEM and come back.
//
// 16 tokens a slice keep the units small, which evens out ragged batches (64 sequences of 512 .. 16384 tokens, one new,
// 2.16 GB: 325 to 338 us, 6.4 to 6.6 TB/s; one new token of a sequence of 1024: 9.5 us, nearly all of it launches and
// latencies in a row).  With two row groups a step of 16 tokens is bound by its chain of latencies (wait, score, maximum,
// weight), and 32 tokens halve the steps: 4 new tokens after 65527 (32 rows, 67 MB) took 25.0 us instead of 26.4 (23.7 now
// with the split's setup units), after 262140 54 us (5.0 TB/s with the fixed costs, 6.9 without) instead of 60.
//
// A slice is loaded by one lane, a box of 16 or 32 tokens by 128 bytes each, with the 128-byte swizzle, which is what the
// fragment reads want.  (Sixteen-byte copies by every lane took 40 % of the instructions of the loop.)  Rows of a slice
// outside what the tile sees are cleared in shared memory; a missing page is loaded from an out-of-range coordinate,
// which fills zeros.  At a piece's end the sums go into the stages read last, while the first slices and the queries of
// the next piece are on their way to the others.
//
// The sums are rescaled only when a row's maximum rises by more than 8 (a factor of 256 that fp32 sums and bf16
// weights carry without loss), so most slices skip that pass over the accumulator.
//
// fp32: every product as three TF32 mma.sync parts, x = hi + lo (hi rounded to 11 bits, lo the rest):
// hi hi + hi lo + lo hi leaves about 2^-21 of a product.  Bound by instructions and the latency of the products' chains
// (8 sequences of 1 .. 256 new tokens, D = 64, window 1024: 45 us, issue slots 34 % busy, tensor pipe 29 %, 17 MB).
#include <algorithm>

#include "paged.cuh"
#include "umma.cuh"

namespace gdn {

using namespace umma;

namespace {

constexpr int SLICES = 4;
constexpr float RAISE = 8.f;  // log2 of the growth of a row's maximum that is left in its weights

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo: hi has 11 significant bits, rounded with halves away from zero, and what is left has 12, of which the product
// reads 11 (it ignores the low 13 bits of a word).  Rounding may carry into infinity or past a NaN, so hi stops at the
// largest value of its sign (one minimum of signed and one of unsigned numbers for the two signs): an infinity or a NaN is
// one in lo.  Without them, and with lo rounded by an integer sum, the NaN that fp32 arithmetic makes (0x7fffffff) came out
// as zero and the largest values as inf - inf; they cost 1 to 3 % (512 new tokens after 3584, 32 heads of 128: 637 to 652 us;
// 8 sequences of 1 .. 256, D = 64: 43.8 to 45.0 us).  Weights are below 2^9 or NaN, and need none.
__device__ __forceinline__ uint32_t round_tf32(float x) { return __float_as_uint(x) + 0x1000u; }
__device__ __forceinline__ void rest_tf32(float x, uint32_t &hi, uint32_t &lo) {
  hi &= 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
  hi = min((uint32_t)min((int)round_tf32(x), 0x7f7fffff), 0xff7fffffu);
  rest_tf32(x, hi, lo);
}
__device__ __forceinline__ void split_weight(float x, uint32_t &hi, uint32_t &lo) {
  hi = round_tf32(x);
  rest_tf32(x, hi, lo);
}
// sum of c[] += a b with both operands in two TF32 parts; N accumulators, so that the parts wait for one another less
template <int N>
__device__ __forceinline__ void mma_3tf32(float (&c)[N][4], const uint32_t (&ah)[4], const uint32_t (&al)[4], float b0, float b1) {
  uint32_t h0, l0, h1, l1;
  split_tf32(b0, h0, l0);
  split_tf32(b1, h1, l1);
  mma_tf32(c[0], al, h0, h1);
  mma_tf32(c[1 % N], ah, l0, l1);
  mma_tf32(c[2 % N], ah, h0, h1);
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// byte offset of 16-byte chunk c of row r in a tile of `ROWS` rows: boxes of 128 bytes by ROWS rows, 128-byte swizzle
template <int ROWS> __device__ __forceinline__ uint32_t tile_off(int r, int c) {
  return (c >> 3) * (ROWS * 128) + r * 128 + (((c ^ r) & 7) << 4);
}
// Bounded wait that polls with the plain test: a slice is mostly there or about to be, and the test that may suspend costs
// more than it saves (64 sequences of 512 .. 16384 tokens: 336 us against 345 us).  The limit is about a second.
__device__ __forceinline__ bool slice_wait(uint32_t bar, uint32_t parity, uint32_t limit = 1u << 25) {
  for (uint32_t it = 0; it < limit; ++it) {
    uint32_t done;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
  }
  return false;
}
// the warps of one slice
template <int RG> __device__ __forceinline__ void slice_sync(int slice) {
  if constexpr (RG == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;\n" ::"r"(2 + slice), "n"(32 * RG) : "memory");
}

}  // namespace

template <typename I, int D, int RG, int NS, int STAGES>
__global__ void __launch_bounds__(128 * RG, RG == 1 && D * sizeof(I) <= 256 ? 2 : 1)
attn_rows_kernel(const PagedArgs a, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  constexpr int SL = 16 * NS, BN = SLICES * SL;
  constexpr int NT = 128 * RG, MT = 16 * RG, RB = D * sizeof(I), CPR = RB / 16, SLB = SL * RB;
  constexpr int BOXES = RB / 128, BW = 128 / sizeof(I);  // boxes of a slice, features of a box
  constexpr int SUMS = 16 * D * 4, PER = 2 * SLB / SUMS < RG ? 2 * SLB / SUMS : RG;  // a warp's sums; of them in a stage
  constexpr int DIST = STAGES - RG / PER;                // slices on their way ahead of the one in use
  constexpr bool F32 = sizeof(I) == 4;
  constexpr int KS = F32 ? D / 8 : D / 16;  // k steps of q . k
  constexpr bool ROOM = F32 && D == 64;     // registers for both parts of the queries and three sets of scores
  static_assert(PER >= 1 && RG % PER == 0, "a warp's sums fit a stage");
  extern __shared__ uint8_t raw[];
  __shared__ Cursor cur, nxt;  // one for the CTA, out of registers
  __shared__ int found, going;  // what the search found; whether there is a next piece
  __shared__ uint64_t full[SLICES][STAGES];
  __shared__ float mass[4 * RG][2][16];  // maxima and masses of the warps' rows
  __shared__ uint32_t where[4 * RG];     // the stages that hold their sums
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint8_t *qsm = smem + SLICES * STAGES * 2 * SLB;  // the query rows, [MT][D]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, qd = lane & 3;
  const int slice = warp & 3, rg = warp >> 2;
  const int cta = blockIdx.x;
  const int P = 1 << a.log2P;
  if (tid < SLICES * STAGES) mbar_init(smem_u32(&full[0][0] + tid), 1);
  if (tid == 0) {
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  pdl_trigger();
  pdl_wait();
  if (a.expire) {  // no copy has been asked for
    if (tid == 0) {
      a.hdr[cta] = make_int4(0, 0, 0, 0);
      a.status[cta] = slice_wait(smem_u32(&full[0][0]), 0, 1024) ? 0 : 4;
    }
    return;
  }
  bool cut = false;  // this CTA's header is written
  int expired = 0;   // a bounded wait ran out
  SeqInfo *seqs = reinterpret_cast<SeqInfo *>(smem);  // the search uses the rings' memory
  cursor_prepare<NT>(a, seqs);
  if (warp == 0) {
    const int x = cursor_begin_one_warp<MT, BN>(a, cur, seqs);
    if (lane == 0) found = x;
  }
  fence_async_smem();
  __syncthreads();
  if (found == 2) {   // a batch too large for one warp
    __syncthreads();  // everyone has read it
    Cursor c;
    const bool some = cursor_begin_any<NT, MT, BN>(a, c, *reinterpret_cast<PlanSmem<NT> *>(smem));
    if (tid == 0) {
      cur = c;
      found = some;
    }
    fence_async_smem();
    __syncthreads();
  }
  bool more = found && cur.works();
  uint8_t *ring = smem + slice * (STAGES * 2 * SLB);
  const uint32_t ring_u = smem_u32(ring), full_u = smem_u32(&full[slice][0]);
  const I *Q = static_cast<const I *>(a.q);
  uint32_t st = 0, ph = 0;  // the ring's next stage to be read and its parity
  auto stage_at = [&](uint32_t k) { return st + k < STAGES ? st + k : st + k - STAGES; };  // k stages on, k < STAGES

  // the blocks [b0, b1) of a piece in which the slice holds a key that some row sees
  auto blocks = [&](const Cursor &c, int &b0, int &b1) {
    bool first, last;
    cursor_piece(c, b0, b1, first, last);
    const int tw = c.w.blk0 * BN + slice * SL;
    if (b0 < b1) {
      if (tw + b0 * BN + SL <= c.w.lo) ++b0;
      if (tw + (b1 - 1) * BN >= c.w.hi) --b1;
    }
    return tw;
  };
  auto page_of = [&](const int *trow, int token) {
    const int j = token >> a.log2P, pg = j < a.max_pages ? trow[j] : -1;
    return (unsigned)pg < (unsigned)a.num_pages ? pg : a.num_pages;
  };
  struct Pages {
    int p[NS];  // of each 16 tokens of a slice
  };
  auto pages_of = [&](const int *trow, int token) {
    Pages pg;
#pragma unroll
    for (int u = 0; u < NS; ++u) pg.p[u] = page_of(trow, token + 16 * u);
    return pg;
  };
  const bool whole = NS > 1 && P >= SL;  // a slice lies in one page, and the boxes have its height
  auto issue = [&](int token, const Pages &pg, int h, uint32_t stage) {
    if (lane == 0 && rg == 0 && !expired) {
      const uint32_t bar = full_u + 8 * stage, dst = ring_u + stage * 2 * SLB;
      mbar_expect_tx(bar, 2 * SLB);
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        if (u > 0 && whole) break;
        const int off = (token + 16 * u) & (P - 1);
#pragma unroll
        for (int i = 0; i < BOXES; ++i) tma_load_4d(dst + (i * SL + 16 * u) * 128, &tk, i * BW, h, off, pg.p[u], bar);
#pragma unroll
        for (int i = 0; i < BOXES; ++i) tma_load_4d(dst + SLB + (i * SL + 16 * u) * 128, &tv, i * BW, h, off, pg.p[u], bar);
      }
    }
  };
  // the pages of the first slices of the piece at c
  struct Ahead {
    int token, h;  // first slice
    int n;         // slices of the piece
    Pages pg[DIST];
  };
  auto look = [&](const Cursor &c) {
    Ahead x;
    int b0, b1;
    x.token = blocks(c, b0, b1) + b0 * BN;
    x.n = b1 - b0;
    x.h = c.h;
    const int *trow = a.table + (long long)c.n * a.table_stride;
#pragma unroll
    for (int s = 0; s < DIST; ++s)
      if (s < x.n) x.pg[s] = pages_of(trow, x.token + s * BN);
    return x;
  };
  // asks for the queries and the first slices of the piece at c
  auto begin_piece = [&](const Cursor &c, const Ahead &x) {
#pragma unroll
    for (int i = 0; i < (MT * CPR + NT - 1) / NT; ++i) {  // the rows, coalesced
      const int y = tid + i * NT, r = y / CPR, ch = y % CPR;
      if (y < MT * CPR) {
        int tok, head;
        row_place(a, c, MT, r < c.w.rows ? r : 0, tok, head);
        cp_async16(qsm + tile_off<MT>(r, ch), Q + tok * a.q_tok + head * a.q_head + ch * (16 / (int)sizeof(I)), r < c.w.rows);
      }
    }
#pragma unroll
    for (int s = 0; s < DIST; ++s)
      if (s < x.n) issue(x.token + s * BN, x.pg[s], x.h, stage_at(s));
  };

  if (more) begin_piece(cur, look(cur));
  while (more) {
    int b0, b1;
    bool first, last;
    const int n = cursor_piece(cur, b0, b1, first, last);
    const int tw = blocks(cur, b0, b1);
    const int lo = cur.w.lo, hi = cur.w.hi, rows = cur.w.rows, pos0 = cur.w.pos0, kvh = cur.h;
    const int *trow = a.table + (long long)cur.n * a.table_stride;
    Pages pg_next = {};
    if (b0 + DIST < b1) pg_next = pages_of(trow, tw + (b0 + DIST) * BN);
    if (tid == NT - 1) {
      Cursor c = cur;
      going = cursor_next<MT, BN>(a, c, n);
      nxt = c;
    }
    cp_async_wait_all();
    __syncthreads();
    more = going;
    Ahead ahead = {};
    if (!F32 && more) ahead = look(nxt);  // its pages are there when this piece ends (fp32 has no registers to keep them in)

    // ---- query fragments: rows g and g + 8 of the warp's 16.  fp32: which feature is which k of a product is free as long
    // as both sides agree, and so 16 bytes of a row serve two k steps: indexes qd and qd + 4 of steps 2 p and 2 p + 1
    // are the four features of 16-byte piece 2 qd + (p & 1) of the 128 bytes p / 2, which a quarter warp reads from all
    // banks (one load for four: 512 new tokens after 3584 with D = 128 take
    // 314 us instead of 403).
    uint32_t qf[KS][4], ql[ROOM ? KS : 1][4];
    int pos[2];
    const int r0 = 16 * rg;
    auto piece = [&](int p) { return 8 * (p >> 1) + 2 * qd + (p & 1); };
    if constexpr (F32) {
#pragma unroll
      for (int p = 0; p < KS / 2; ++p)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint4 v = *reinterpret_cast<const uint4 *>(qsm + tile_off<MT>(r0 + g + 8 * x, piece(p)));
          qf[2 * p][x] = v.x;
          qf[2 * p][x + 2] = v.y;
          qf[2 * p + 1][x] = v.z;
          qf[2 * p + 1][x + 2] = v.w;
        }
      if constexpr (ROOM) {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) split_tf32(__uint_as_float(qf[k][e]), qf[k][e], ql[k][e]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < KS; ++k) ldmatrix_x4(smem_u32(qsm) + tile_off<MT>(r0 + (lane & 15), 2 * k + (lane >> 4)), qf[k]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const unsigned r = (unsigned)cur.t * MT + min(r0 + g + 8 * e, rows - 1);
      pos[e] = cur.s.kv - cur.s.qlen + (int)(r / (unsigned)a.G);
    }
    const bool active = rows > r0;  // the warp's 16 rows are not all past the tile's
    const int pos_last = cur.s.kv - cur.s.qlen + (int)(((unsigned)cur.t * MT + rows - 1) / (unsigned)a.G);

    float acc[D / 8][1][4], m[2], l[2];
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][0][e] = 0.f;

    for (int b = b0; b < b1; ++b) {
      if (!expired && !slice_wait(full_u + 8 * st, ph)) expired = 4;
      slice_sync<RG>(slice);  // every lane of the slice's warps is done with the block before, too
      if (b + DIST < b1) issue(tw + (b + DIST) * BN, pg_next, kvh, stage_at(DIST));
      if (b + DIST + 1 < b1) pg_next = pages_of(trow, tw + (b + DIST + 1) * BN);
      const uint32_t ks = ring_u + st * 2 * SLB, vs = ks + SLB;
      uint8_t *ksp = ring + st * 2 * SLB, *vsp = ksp + SLB;
      if (++st == STAGES) {
        st = 0;
        ph ^= 1;
      }
      const int t0 = tw + b * BN;
      if (t0 < lo || t0 + SL > hi) {
        // value rows that no query sees become zeros: whatever those slots hold, zero weights keep them out (the
        // slice's warps write the same zeros)
        for (int i = lane; i < SLB / 16; i += 32) {
          const int r = (i >> 3) & (SL - 1);
          if (t0 + r < lo || t0 + r >= hi) reinterpret_cast<uint4 *>(vsp)[i] = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();  // the stage is loaded again later
        __syncwarp();
      }
      if (!active) continue;
      // ---- scores: tile j holds tokens 8 j .. 8 j + 7
      constexpr int NA = ROOM ? 3 : 1;
      float s3[2 * NS][NA][4];
#pragma unroll
      for (int j = 0; j < 2 * NS; ++j)
#pragma unroll
        for (int n = 0; n < NA; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s3[j][n][e] = 0.f;
      if constexpr (!F32) {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int u = 0; u < NS; ++u) {
            uint32_t bk[4];
            const uint32_t ad = ks + tile_off<SL>(16 * u + (lane & 7) + 8 * (lane >> 4), 2 * k + ((lane >> 3) & 1));
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                         : "=r"(bk[0]), "=r"(bk[1]), "=r"(bk[2]), "=r"(bk[3]) : "r"(ad) : "memory");
            mma_bf16(s3[2 * u][0], qf[k], bk[0], bk[1]);
            mma_bf16(s3[2 * u + 1][0], qf[k], bk[2], bk[3]);
          }
      } else {
#pragma unroll
        for (int p = 0; p < KS / 2; ++p) {
          float4 bk[2 * NS];
#pragma unroll
          for (int j = 0; j < 2 * NS; ++j) bk[j] = *reinterpret_cast<const float4 *>(ksp + tile_off<SL>(g + 8 * j, piece(p)));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (ROOM) {
                ah[e] = qf[2 * p + x][e];
                al[e] = ql[2 * p + x][e];
              } else {
                split_tf32(__uint_as_float(qf[2 * p + x][e]), ah[e], al[e]);
              }
            }
#pragma unroll
            for (int j = 0; j < 2 * NS; ++j) mma_3tf32(s3[j], ah, al, x ? bk[j].z : bk[j].x, x ? bk[j].w : bk[j].y);
          }
        }
      }
      float s[2 * NS][4];
#pragma unroll
      for (int j = 0; j < 2 * NS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = ROOM ? s3[j][0][e] + s3[j][1 % NA][e] + s3[j][2 % NA][e] : s3[j][0][e];
      // ---- softmax: thread holds rows g, g + 8 (e >> 1), tokens 8 j + 2 qd + (e & 1)
      const bool mask = t0 + SL - 1 > pos0 || (a.window && t0 < pos_last - a.window + 1);
      float mx[2] = {-INFINITY, -INFINITY};
      bool raise = false;
#pragma unroll
      for (int j = 0; j < 2 * NS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float z = s[j][e] * a.scale_log2;
          if (mask) {
            const int key = t0 + 8 * j + 2 * qd + (e & 1), p = pos[e >> 1];
            if (key > p || (a.window && key <= p - a.window)) z = -INFINITY;
          }
          s[j][e] = z;
          mx[e >> 1] = fmaxf(mx[e >> 1], z);
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = quad_max(mx[e]);
        raise |= mx[e] > m[e] + RAISE;
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(m[e], mx[e]);
          const float f = mn == -INFINITY ? 1.f : ex2(m[e] - mn);
          m[e] = mn;
          l[e] *= f;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            acc[j][0][2 * e] *= f;
            acc[j][0][2 * e + 1] *= f;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mm = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
        for (int j = 0; j < 2 * NS; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float p = ex2(s[j][2 * e + x] - mm);
            l[e] += p;
            s[j][2 * e + x] = p;
          }
      }
      // ---- sums += weights x values
      if constexpr (!F32) {
#pragma unroll
        for (int u = 0; u < NS; ++u) {
          uint32_t pa[4];
          pa[0] = pack_bf16(s[2 * u][0], s[2 * u][1]);
          pa[1] = pack_bf16(s[2 * u][2], s[2 * u][3]);
          pa[2] = pack_bf16(s[2 * u + 1][0], s[2 * u + 1][1]);
          pa[3] = pack_bf16(s[2 * u + 1][2], s[2 * u + 1][3]);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t bv[4];
            const uint32_t ad = vs + tile_off<SL>(16 * u + (lane & 7) + 8 * ((lane >> 3) & 1), 2 * j + (lane >> 4));
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                         : "=r"(bv[0]), "=r"(bv[1]), "=r"(bv[2]), "=r"(bv[3]) : "r"(ad) : "memory");
            mma_bf16(acc[2 * j][0], pa, bv[0], bv[1]);
            mma_bf16(acc[2 * j + 1][0], pa, bv[2], bv[3]);
          }
        }
      } else {
        // the 8 tokens of score tile jt are the k of one step: index qd is token 2 qd and qd + 4 is token 2 qd + 1,
        // in the weights (as the scores came out) and in the values alike; column g of the output tiles 4 p + i is
        // feature 4 g + i of the 128 bytes p, so that 16 bytes of a row serve four tiles
#pragma unroll
        for (int jt = 0; jt < 2 * NS; ++jt) {
          uint32_t ph[4], pl[4];
          split_weight(s[jt][0], ph[0], pl[0]);
          split_weight(s[jt][2], ph[1], pl[1]);
          split_weight(s[jt][1], ph[2], pl[2]);
          split_weight(s[jt][3], ph[3], pl[3]);
#pragma unroll
          for (int p = 0; p < D / 32; ++p) {
            const int r = 8 * jt + 2 * qd;
            const float4 v0 = *reinterpret_cast<const float4 *>(vsp + tile_off<SL>(r, 8 * p + g));
            const float4 v1 = *reinterpret_cast<const float4 *>(vsp + tile_off<SL>(r + 1, 8 * p + g));
            mma_3tf32(acc[4 * p], ph, pl, v0.x, v1.x);
            mma_3tf32(acc[4 * p + 1], ph, pl, v0.y, v1.y);
            mma_3tf32(acc[4 * p + 2], ph, pl, v0.z, v1.z);
            mma_3tf32(acc[4 * p + 3], ph, pl, v0.w, v1.w);
          }
        }
      }
    }
    // ---- the slices' sums meet: each warp leaves its own in a stage it has read (16-byte chunks of a row change places
    // by the row's low bits, against bank conflicts)
    {
      const uint32_t at = stage_at(STAGES - 1 - rg / PER) * 2 * SLB + rg % PER * SUMS;
      float *om = reinterpret_cast<float *>(ring + at);
      slice_sync<RG>(slice);  // the other warp of the slice has read it too
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = g + 8 * e;
        const float ls = quad_sum(l[e]);
        if (qd == 0) {
          mass[warp][0][r] = m[e];
          mass[warp][1][r] = ls;
        }
        if constexpr (F32) {
#pragma unroll
          for (int p = 0; p < D / 32; ++p)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              *reinterpret_cast<float4 *>(om + r * D + (((8 * p + 2 * qd + x) ^ (r & 7)) << 2)) =
                  make_float4(acc[4 * p][0][2 * e + x], acc[4 * p + 1][0][2 * e + x], acc[4 * p + 2][0][2 * e + x],
                              acc[4 * p + 3][0][2 * e + x]);
        } else {
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            *reinterpret_cast<float2 *>(om + r * D + (((2 * j + (qd >> 1)) ^ (r & 7)) << 2) + 2 * (qd & 1)) =
                make_float2(acc[j][0][2 * e], acc[j][0][2 * e + 1]);
        }
      }
      if (lane == 0) where[warp] = slice * (STAGES * 2 * SLB) + at;
    }
    __syncthreads();
    if (more) begin_piece(nxt, F32 ? look(nxt) : ahead);
    constexpr int LPR = D / 4;  // lanes of a row
    const int slot = first ? 1 : 0;
    float *rec = a.part + ((long long)cta * 2 + slot) * record_floats(MT, D);
    for (int r = warp * (32 / LPR) + lane / LPR; r < rows; r += 4 * RG * (32 / LPR)) {
      const int c = lane % LPR, w0 = r / 16 * 4, rr = r % 16;  // the row's four warps
      float mw[4], M = -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        mw[x] = mass[w0 + x][0][rr];
        M = fmaxf(M, mw[x]);
      }
      float L = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float f = mw[x] == -INFINITY ? 0.f : ex2(mw[x] - M);
        const float4 v = *reinterpret_cast<const float4 *>(smem + where[w0 + x] + (rr * D + ((c ^ (rr & 7)) << 2)) * 4);
        L += f * mass[w0 + x][1][rr];
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
          *reinterpret_cast<uint2 *>(op) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        }
        if (a.lse && c == 0)
          a.lse[(long long)tok * a.Hq + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      } else {
        *reinterpret_cast<float4 *>(rec + r * D + 4 * c) = o;
        if (c == 0) {
          rec[MT * D + r] = M;
          rec[MT * D + MT + r] = L;
        }
      }
    }
    if (first && !last) {
      cut = true;
      if (tid == 0) a.hdr[cta] = cut_header<MT>(a, cur);
    }
    fence_async_smem();  // the stages with the sums are loaded again
    __syncthreads();
    if (tid == 0) cur = nxt;
    __syncthreads();
  }
  if (tid == 0 && !cut) a.hdr[cta] = make_int4(0, 0, 0, 0);
  if (expired) {  // copies in flight end, if they do, before the shared memory goes
    for (int s = 0; s < STAGES; ++s) mbar_wait(full_u + 8 * s, (uint32_t)s < st ? ph ^ 1 : ph, nullptr, 0, 1u << 16);
  }
  expired = __syncthreads_or(expired);
  if (tid == 0) a.status[cta] = expired ? 4 : 0;
}

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

namespace {
template <typename I, int D, int RG, int NS, int STAGES>
cudaError_t launch_rows(const PagedArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, int ctas, cudaStream_t st) {
  constexpr size_t ring = (size_t)SLICES * STAGES * 2 * 16 * NS * D * sizeof(I);
  static_assert(ring >= sizeof(PlanSmem<128 * RG>) && ring >= WARP_SEQS * sizeof(SeqInfo), "the search uses the rings' memory");
  constexpr size_t smem = 1024 + ring + (size_t)16 * RG * D * sizeof(I);
  auto *k = attn_rows_kernel<I, D, RG, NS, STAGES>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(ctas), dim3(128 * RG), smem, st, a, tk, tv);
}
}  // namespace

// 16 rows a tile where that is enough, and in fp32 with D = 64 always: 96 KB of rings (fp32, D = 128: 192 KB) and then two
// CTAs per SM.  More rows: two row groups and 192 KB of rings, so that a key or value is fetched and, in fp32, split into
// its two parts half as often (fp32: D = 64, 8 sequences of up to 256 new tokens: 44 us with 16 rows, 47 us with 32, the last
// 1024 of 4096 tokens: 313 and 324 us; D = 128, 512 new tokens after 3584: 530 us with 16 rows, 317 us with 32; both sides
// before the guard in split_tf32, which adds 1 to 3 %).
int attn_rows_tile(bool bf, int D, int rows) { return rows <= 16 || (!bf && D == 64) ? 16 : 32; }
int attn_rows_box(bool bf, int MT, int page) { return bf && MT == 32 && page >= 32 ? 32 : 16; }
int attn_rows_per_sm(bool bf, int D, int MT) { return MT == 16 && (bf || D == 64) ? 2 : 1; }
cudaError_t launch_attn_rows(const PagedArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, bool bf, int D, int MT, int ctas,
                             cudaStream_t st) {
  if (!bf) {
    if (D == 64) return launch_rows<float, 64, 1, 1, 3>(a, tk, tv, ctas, st);
    return MT == 16 ? launch_rows<float, 128, 1, 1, 3>(a, tk, tv, ctas, st)
                    : launch_rows<float, 128, 2, 1, 3>(a, tk, tv, ctas, st);
  }
  if (D == 64)
    return MT == 16 ? launch_rows<bf16, 64, 1, 1, 6>(a, tk, tv, ctas, st) : launch_rows<bf16, 64, 2, 2, 6>(a, tk, tv, ctas, st);
  return MT == 16 ? launch_rows<bf16, 128, 1, 1, 3>(a, tk, tv, ctas, st) : launch_rows<bf16, 128, 2, 2, 3>(a, tk, tv, ctas, st);
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
