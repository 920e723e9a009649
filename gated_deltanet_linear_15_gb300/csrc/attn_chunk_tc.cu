// Attention of chunks of new tokens over a paged cache, bf16, on the fifth-generation tensor cores:
//   S = Q K^T,  P = exp2(scale log2(e) S - m),  O += P V,  o = O / sum(P)
// with the running maximum m of a row (softmax layers of a hybrid stack: onedev.kr summary of the FlashQLA talk,
// background paragraph).
//
// Bound by the matrix products (4 D flops per row and key) and, close behind, by one exponential per row and key.  A
// CTA holds 256 query rows as two tiles of 128, so that while the tensor core multiplies for one tile the other tile's
// softmax runs.  Scores and sums live in TMEM (two times 128 columns of S, two times D of O); a softmax warp reads its
// 32 rows of S, one whole row per thread, so a row's maximum and sum need no shuffles, and writes the weights as bf16
// over the scores, from where the second product takes them as its A operand.  O is rescaled in TMEM only when a
// maximum of the warp rises by more than 8 (2^8, which fp32 sums and bf16 weights carry without loss).
//
// Warps: 0-3 and 4-7 the softmax of the two tiles, 8 issues every product, 9 loads.  Keys and values come in 128-token
// tiles through a ring, one TMA box per page and 64 features; a page outside the pool, or outside what the rows see,
// is loaded from an out-of-range coordinate, which fills zeros.  (Warps 10 and 11 only complete the third warpgroup,
// which gives up registers: 168 a thread at launch become 224 for the softmax, which holds a row of S, and 56 here.)  Slots past the last key (or before the first of a
// window) may hold anything, so warp 8 clears their value rows before the product that would multiply them by zero.
// The work split over CTAs is paged.cuh's.  Every wait is bounded; one that expires ends the CTA with a status word.
#include "paged.cuh"
#include "umma.cuh"

namespace gdn {

using namespace umma;

namespace {

constexpr int NTHR = 384, SOFT = 256, MT = 256, BN = 128;
constexpr float RAISE = 8.f;
constexpr uint32_t WAIT_LIMIT = 1u << 22;

__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool b_mn_major, bool neg_a) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((neg_a ? 1u : 0u) << 13) | ((b_mn_major ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <int D> struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int QT = 128 * D * 2;      // bytes of a query tile
  static constexpr int STAGE = BN * D * 2;    // bytes of a key or value tile
  static constexpr int STAGES = D == 128 ? 5 : 8;
  static constexpr int SMEM = 2 * QT + STAGES * STAGE + 1024;
};
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;

struct Bars {
  uint64_t full[8], empty[8], q_full[2], s_full[2], p_full[2], o_full[2], drain;
  uint32_t tmem;
  int dead;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// D[tmem] (+)= A[tmem] * B
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, SDesc b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .b64 db;\n"
      ".reg .pred p;\n"
      "mov.b64 db, {%2, %3};\n"
      "setp.ne.b32 p, %5, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n"
      "}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void tma_load_4d(uint32_t smem_dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n" ::"r"(smem_dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(mbar)
      : "memory");
}
// 32 lanes x 32 columns, not waited for
__device__ __forceinline__ void tmem_ld32_nw(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32_nw(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// packed pairs of fp32
__device__ __forceinline__ uint64_t pk(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void upk(uint64_t r, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// bounded wait; gives up at once when another role of the CTA has
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *dead) {
  const uint32_t b = smem_u32(bar);
  for (uint32_t it = 0; it < WAIT_LIMIT; ++it) {
    uint32_t done;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(done)
        : "r"(b), "r"(parity)
        : "memory");
    if (done) return true;
    if ((it & 63) == 63 && *dead) return false;
  }
  *dead = 1;
  return false;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(NTHR, 1) attn_chunk_kernel(const PagedArgs a, const __grid_constant__ CUtensorMap tk,
                                                             const __grid_constant__ CUtensorMap tv, uint32_t neg) {
  using C = Cfg<D>;
  extern __shared__ uint8_t raw[];
  __shared__ Bars bars;
  __shared__ Cursor start;
  __shared__ int has_work;
  __shared__ long long scan_sh[SOFT / 32];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint8_t *qs = sm, *ring = sm + 2 * C::QT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  volatile int *dead = &bars.dead;

  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(smem_u32(&bars.full[i]), 1);
      mbar_init(smem_u32(&bars.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.q_full[i]), 128);
      mbar_init(smem_u32(&bars.s_full[i]), 1);
      mbar_init(smem_u32(&bars.p_full[i]), 128);
      mbar_init(smem_u32(&bars.o_full[i]), 1);
    }
    mbar_init(smem_u32(&bars.drain), 1);
    bars.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&bars.tmem), TM_COLS);
    tmem_relinquish();
  }
  pdl_trigger();
  pdl_wait();
  if (tid < SOFT) {
    Cursor c;
    const bool more = cursor_begin<SOFT, MT, BN>(a, c, reinterpret_cast<long long(*)[SOFT + 1]>(ring), scan_sh);
    if (tid == 0) {
      start = c;
      has_work = more;
    }
    fence_async_smem();  // the search used the ring's memory
  }
  fence_before();
  __syncthreads();
  fence_after();
  Cursor cur = start;
  bool more = has_work;
  const uint32_t tmem = bars.tmem;
  int used = 0;

  // registers: 128 * (2 * 224 + 56) = 384 * 168, those of the launch
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n");
  if (warp == 9) {
    // ------------------------------------------------------------ loader
    const int P = 1 << a.log2P, box = min(P, BN), pieces = BN / box;
    const int piece = lane / C::HALVES, half = lane % C::HALVES;
    uint32_t st = 0, ph = 0;  // next stage and its parity
    uint32_t issued = 0;      // stages ever filled
    bool ok = true;
    while (more && ok) {
      int b0, b1;
      bool first, last;
      const int n = cursor_piece(cur, b0, b1, first, last);
      const int *trow = a.table + (long long)cur.n * a.table_stride;
      for (int b = b0; b < b1 && ok; ++b) {
        const int t = (cur.w.blk0 + b) * BN + piece * box;
        int page = a.num_pages;  // zeros
        if (piece < pieces && t < cur.w.hi && t + box > cur.w.lo) {
          const int pg = trow[t >> a.log2P];
          if ((unsigned)pg < (unsigned)a.num_pages) page = pg;
        }
        const int off = t & (P - 1);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          ok = ok && wait(&bars.empty[st], ph ^ 1, dead);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(smem_u32(&bars.full[st]), C::STAGE);
          __syncwarp();
          if (piece < pieces)
            tma_load_4d(smem_u32(ring + st * C::STAGE + half * (BN * 128) + piece * box * 128), kv ? &tv : &tk, half * 64, cur.h, off,
                        page, smem_u32(&bars.full[st]));
          ++issued;
          if (++st == C::STAGES) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      more = cursor_next<MT, BN>(a, cur, n);
    }
    // a CTA that gives up waits (bounded) for the copies in flight before its shared memory goes
    if (*dead) {
      const uint32_t k = min(issued, (uint32_t)C::STAGES);
      for (uint32_t i = 0; i < k; ++i) {
        if (st == 0) {
          st = C::STAGES;
          ph ^= 1;
        }
        --st;
        mbar_wait(smem_u32(&bars.full[st]), ph, nullptr, 0, 1u << 20);
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ products
    const uint32_t id_s = idesc_bf16(128, BN, false, neg != 0), id_o = idesc_bf16(128, D, true, false);
    uint32_t st = 0, ph = 0;
    uint32_t pq[2] = {0, 0}, pp[2] = {0, 0};  // parities of the tiles' barriers
    bool ok = true;
    auto next = [&] {
      if (++st == C::STAGES) {
        st = 0;
        ph ^= 1;
      }
    };
    auto scores = [&](int x, uint32_t ks) {  // S[x] = Q[x] K^T
      const SDesc q = sdesc_s(smem_u32(qs + x * C::QT), 16, 1024), k = sdesc_s(ks, 16, 1024);
#pragma unroll 1
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t o = (i >> 2) * (BN * 128) + (i & 3) * 32;
        mma_f16s(tmem + TM_S + x * BN, q + o, k + o, id_s, i > 0);
      }
      mma_commit(smem_u32(&bars.s_full[x]));
    };
    auto sums = [&](int x, uint32_t vs, bool acc) {  // O[x] += P[x] V
      const SDesc v = sdesc_s(vs, BN * 128, 1024);
#pragma unroll 1
      for (int i = 0; i < BN / 16; ++i) mma_ts(tmem + TM_O + x * D, tmem + TM_S + x * BN + 8 * i, v + i * 2048, id_o, acc || i > 0);
    };
    while (more && ok) {
      int b0, b1;
      bool first, last;
      const int n = cursor_piece(cur, b0, b1, first, last);
      const int nx = cur.w.rows > 128 ? 2 : 1;
      if (b0 < b1) {
        for (int x = 0; x < nx; ++x) {
          ok = ok && wait(&bars.q_full[x], pq[x], dead);
          pq[x] ^= 1;
        }
        // keys of the first block
        ok = ok && wait(&bars.full[st], ph, dead);
        if (!ok) break;
        fence_after();
        if (lane == 0) {
          for (int x = 0; x < nx; ++x) scores(x, smem_u32(ring + st * C::STAGE));
          mma_commit(smem_u32(&bars.empty[st]));
        }
        __syncwarp();
        next();
        for (int b = b0; b < b1 && ok; ++b) {
          const uint32_t vstage = st;
          ok = ok && wait(&bars.full[st], ph, dead);
          if (!ok) break;
          // value rows that no query sees become zeros: whatever those slots hold, zero weights keep them out
          const int t0 = (cur.w.blk0 + b) * BN, r_lo = cur.w.lo - t0, r_hi = cur.w.hi - t0;
          if (r_lo > 0 || r_hi < BN) {
            uint8_t *vs = ring + vstage * C::STAGE;
            for (int i = lane; i < BN * 8 * C::HALVES; i += 32) {
              const int r = (i >> 3) & (BN - 1);
              if (r < r_lo || r >= r_hi) reinterpret_cast<uint4 *>(vs)[i] = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            __syncwarp();
          }
          next();
          const bool has_next = b + 1 < b1;
          const uint32_t kstage = st;
          for (int x = 0; x < nx && ok; ++x) {
            ok = wait(&bars.p_full[x], pp[x], dead);
            if (!ok) break;
            pp[x] ^= 1;
            fence_after();
            if (lane == 0) {
              sums(x, smem_u32(ring + vstage * C::STAGE), b > b0);
              if (x == nx - 1) mma_commit(smem_u32(&bars.empty[vstage]));
              if (!has_next) mma_commit(smem_u32(&bars.o_full[x]));
            }
            __syncwarp();
            if (has_next) {
              if (x == 0) ok = wait(&bars.full[kstage], ph, dead);
              if (!ok) break;
              fence_after();
              if (lane == 0) {
                scores(x, smem_u32(ring + kstage * C::STAGE));
                if (x == nx - 1) mma_commit(smem_u32(&bars.empty[kstage]));
              }
              __syncwarp();
            }
          }
          if (has_next) next();
        }
      }
      more = cursor_next<MT, BN>(a, cur, n);
    }
    if (*dead) {  // products in flight end before TMEM goes
      if (lane == 0) mma_commit(smem_u32(&bars.drain));
      __syncwarp();
      mbar_wait(smem_u32(&bars.drain), 0, nullptr, 0, 1u << 20);
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;\n");
    // ------------------------------------------------------------ softmax of tile x
    const int x = warp >> 2, wr = (warp & 3) * 32 + lane;  // row in the tile
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + TM_S + x * BN, to = tmem + lane_base + TM_O + x * D;
    uint32_t ps = 0, po = 0;
    bool ok = true;
    const bf16 *Q = static_cast<const bf16 *>(a.q);
    while (more && ok) {
      int b0, b1;
      bool first, last;
      const int n = cursor_piece(cur, b0, b1, first, last);
      const int rows = cur.w.rows - x * 128;  // of this tile
      if (rows > 0) {
        const int row = x * 128 + wr;
        const bool live = wr < rows;
        int tok, head;
        row_place(a, cur, MT, live ? row : 0, tok, head);
        const int pos = live ? cur.s.kv - cur.s.qlen + tok - cur.s.qbeg : -1;
        float m = -INFINITY, l = 0.f;
        if (b0 < b1) {
          // ---- the warp's 32 query rows, 16 bytes a lane, neighbours in a row
          uint8_t *qt = qs + x * C::QT;
          constexpr int CPR = D / 8;
          for (int i = lane; i < 32 * CPR; i += 32) {
            const int r = (warp & 3) * 32 + i / CPR, c = i % CPR;
            int qt_tok, qt_head;
            const bool there = r < rows;
            row_place(a, cur, MT, x * 128 + (there ? r : 0), qt_tok, qt_head);
            cp_async16(qt + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                       Q + qt_tok * a.q_tok + qt_head * a.q_head + c * 8, there);
          }
          cp_async_wait_all();
          fence_async_smem();
          mbar_arrive(smem_u32(&bars.q_full[x]));

          for (int b = b0; b < b1; ++b) {
            ok = wait(&bars.s_full[x], ps, dead);
            if (!ok) break;
            ps ^= 1;
            fence_after();
            uint32_t s[BN];
#pragma unroll
            for (int i = 0; i < BN / 32; ++i) tmem_ld32_nw(ts + 32 * i, s + 32 * i);
            tmem_wait_ld();
            const int t0 = (cur.w.blk0 + b) * BN;
            const bool cut = t0 + BN - 1 > pos || (a.window && t0 <= pos - a.window);
            if (__any_sync(0xffffffffu, cut)) {
              const int hi = pos - t0, lo = a.window ? pos - a.window - t0 : -1;
#pragma unroll
              for (int i = 0; i < BN; ++i)
                if (i > hi || i <= lo) s[i] = 0xff800000u;
            }
            float mx[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(s[i]);
#pragma unroll
            for (int i = 4; i < BN; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i]));
            const float z = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
            if (__any_sync(0xffffffffu, z > m + RAISE)) {
              const float mn = fmaxf(m, z);
              const float f = mn == -INFINITY ? 1.f : ex2(m - mn);
              m = mn;
              l *= f;
              if (b > b0) {
                // the products that wrote O completed before this tile's scores did, the next ones wait for the weights
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                  uint32_t o[32];
                  tmem_ld32_nw(to + 32 * i, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tmem_st32_nw(to + 32 * i, o);
                }
              }
            }
            const float mm = m == -INFINITY ? 0.f : m;
            const uint64_t sc = pk(a.scale_log2, a.scale_log2), nm = pk(-mm, -mm);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              uint32_t w[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int e = hh * 64 + 2 * i;
                float p0, p1;
                upk(fma2(pk(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc, nm), p0, p1);
                p0 = ex2(p0);
                p1 = ex2(p1);
                sum[i & 1] = add2(sum[i & 1], pk(p0, p1));
                w[i] = pack_bf16(p0, p1);
              }
              tmem_st32_nw(ts + 32 * hh, w);
            }
            float u0, u1;
            upk(add2(sum[0], sum[1]), u0, u1);
            l += u0 + u1;
            tmem_wait_st();
            fence_before();
            mbar_arrive(smem_u32(&bars.p_full[x]));
          }
          if (ok) {
            ok = wait(&bars.o_full[x], po, dead);
            po ^= 1;
            fence_after();
          }
        }
        if (ok) {
          const bool whole = first && last;
          const int slot = first ? 1 : 0;
          float *rec = a.part + ((long long)cta * 2 + slot) * record_floats(MT, D);
          const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
          bf16 *op = static_cast<bf16 *>(a.o) + tok * a.o_tok + head * a.o_head;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            if (b0 < b1) {
              tmem_ld32_nw(to + 32 * i, o);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0;
            }
            if (live) {
              if (whole) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                  uint32_t w[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    w[k] = pack_bf16(__uint_as_float(o[e + 2 * k]) * inv, __uint_as_float(o[e + 2 * k + 1]) * inv);
                  *reinterpret_cast<uint4 *>(op + 32 * i + e) = make_uint4(w[0], w[1], w[2], w[3]);
                }
              } else {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                  *reinterpret_cast<uint4 *>(rec + (size_t)row * D + 32 * i + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
              }
            }
          }
          if (live) {
            if (whole) {
              if (a.lse) a.lse[(long long)tok * a.Hq + head] = m == -INFINITY ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            } else {
              rec[(size_t)MT * D + row] = m;
              rec[(size_t)MT * D + MT + row] = l;
            }
          }
          fence_before();
        }
      }
      if (!(first && last)) {
        used |= 1 << (first ? 1 : 0);
        if (tid == 0) {
          const long long r0 = (long long)cur.t * MT;
          a.hdr[cta * 2 + (first ? 1 : 0)] =
              make_int4(last ? 1 : 2, cur.s.qbeg + (int)(r0 / a.G), cur.h, cur.w.rows << 16 | (int)(r0 % a.G));
        }
      }
      more = cursor_next<MT, BN>(a, cur, n);
    }
    if (tid < 2 && !(used >> tid & 1)) a.hdr[cta * 2 + tid] = make_int4(0, 0, 0, 0);
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (tid == 0) a.status[cta] = bars.dead;
  if (warp == 8) tmem_dealloc(tmem, TM_COLS);
}

cudaError_t launch_attn_chunk_tc(const PagedArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, int D, int ctas, cudaStream_t st) {
  PagedArgs b = a;
  // the sign of the scale goes into the product, so that the largest score is the largest logit; a scale of zero
  // becomes one that leaves every weight at 1 and still sends masked scores to -inf
  const uint32_t neg = a.scale_log2 < 0.f ? 1 : 0;
  b.scale_log2 = fmaxf(fabsf(a.scale_log2), 1e-37f);
  auto *k = D == 128 ? attn_chunk_kernel<128> : attn_chunk_kernel<64>;
  const int smem = D == 128 ? Cfg<128>::SMEM : Cfg<64>::SMEM;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(ctas), dim3(NTHR), (size_t)smem, st, b, tk, tv, neg);
}

}  // namespace gdn
