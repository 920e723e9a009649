// Attention of chunks of new tokens over a paged cache, bf16, on the fifth-generation tensor cores:
//   S = Q K^T,  P = exp2(scale log2(e) S - m),  O += P V,  o = O / sum(P)
// with the running maximum m of a row (softmax layers of a hybrid stack: onedev.kr summary of the FlashQLA talk,
// background paragraph).
//
// Bound by the matrix products (4 D flops per row and key) and, close behind, by one exponential per row and key.  A
// CTA holds 256 query rows as two tiles of 128, so that while the tensor core multiplies for one tile the other tile's
// softmax runs.  Scores and sums live in TMEM (two times 128 columns of S, two times D of O); a softmax warp reads its
// 32 rows of S, one whole row per thread, so a row's maximum and sum need no shuffles, and writes the weights as bf16
// over the scores, from where the second product takes them as its A operand.  A row keeps the maximum of its first
// block as long as the weights of later blocks sum to less than 2^40 against it; O is rescaled in TMEM only when they
// do not, and most blocks look for no maximum at all.
//
// Warps: 0-3 and 4-7 the softmax of the two tiles, 8 issues every product, 9 loads.  Keys and values come in 128-token
// tiles through a ring, one TMA box per page and 64 features; a page outside the pool, or outside what the rows see,
// is loaded from an out-of-range coordinate, which fills zeros.  (The third warpgroup gives up registers: 168 a thread at
// launch become 224 for the softmax, which holds a row of S, and 56 here.)  Slots past the last key (or before the first of
// a window) may hold anything, so their value rows are cleared before the product that would multiply them by zero.
//
// 2048 new tokens after 8192, 32 heads of 128: 187 us alone (1.65 PFLOP/s; tensor pipe 73 % busy, a block of 256 rows by
// 128 keys every 2700 cycles, of which the products need 2050), 201 us in a row of calls, when power holds the clock.
// What is left is the strict order of the two tiles' products and shared memory, whose 256 KB a block take nearly as long.
// The work split over CTAs is paged.cuh's.  Every wait is bounded; one that expires ends the CTA with a status word.
#include "paged.cuh"
#include "umma.cuh"

namespace gdn {

using namespace umma;

namespace {

constexpr int NTHR = 384, SOFT = 256, MT = 256, BN = 128;
constexpr float RAISED = 1099511627776.f;  // 2^40: a block's weights that sum to more have their maximum raised
constexpr uint32_t WAIT_LIMIT = 1u << 18;   // polls of 3.8 us when nothing comes: a second
constexpr uint32_t DRAIN_LIMIT = 1u << 16;  // of each stage or tile after that

template <int D> struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int QT = 128 * D * 2;      // bytes of a query tile
  static constexpr int STAGE = BN * D * 2;    // bytes of a key or value tile
  static constexpr int STAGES = D == 128 ? 5 : 8;
  static constexpr int SMEM = 2 * QT + STAGES * STAGE + 1024;
};
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;

struct Bars {
  uint64_t full[8], empty[8], q_full[2], s_full[2], o_full[2], drain[2];
  uint32_t tmem;
  int dead;
  uint3 stages;  // the loader's next stage and its parity at the end, and how many before it have been filled
};

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
// one lane of the warp, chosen so that the compiler knows it: products issued behind `lane == 0` instead leave the tensor
// core idle between them (350 us against 256 us for 2048 tokens after 8192, 32 heads)
__device__ __forceinline__ bool elect1() {
  uint32_t p;
  asm volatile("{\n.reg .pred P;\nelect.sync _|P, 0xffffffff;\nselp.u32 %0, 1, 0, P;\n}\n" : "=r"(p));
  return p != 0;
}
// 32 bytes of one thread, 32-byte aligned: whole sectors, though the rows of neighbouring threads lie apart
__device__ __forceinline__ void st_global_32b(void *p, const uint32_t *v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
               "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// 16 lanes x 64 columns, not waited for: r[4 i + 2 e], r[4 i + 2 e + 1] = row lane / 4 + 8 e, columns 8 i + 2 (lane % 4), + 1
__device__ __forceinline__ void tmem_ld16x64(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// among the four lanes of a quad: t[i] of lane j becomes t[j] of lane i
__device__ __forceinline__ void quad_transpose(uint32_t (&t)[4][2], int qd) {
#pragma unroll
  for (int b = 1; b <= 2; b <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(i & b)) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bool up = qd & b;
          const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? t[i][k] : t[i | b][k], b);
          t[i][k] = up ? got : t[i][k];
          t[i | b][k] = up ? t[i | b][k] : got;
        }
      }
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

// keeps what is computed from v where it is used, instead of in registers across the loop
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
  asm volatile("" : "+r"(v));
  return v;
}
// cursor_next of a cursor in shared memory: lane 0 moves it for the warp
__device__ __forceinline__ bool cursor_advance(const PagedArgs &a, Cursor &shared, int n) {
  bool more = false;
  if ((threadIdx.x & 31) == 0) {
    Cursor c = shared;
    more = cursor_next<MT, BN>(a, c, n);
    shared = c;
  }
  __syncwarp();
  return __shfl_sync(0xffffffffu, more, 0);
}

// Bounded wait.  The plain test comes first: when the phase is complete already, as it mostly is for the issuing warps, it
// answers sooner than the test that may suspend.  Gives up soon when another role of the CTA has.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *dead, uint32_t limit = WAIT_LIMIT) {
  const uint32_t b = smem_u32(bar);
  uint32_t done;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(done)
      : "r"(b), "r"(parity)
      : "memory");
  if (done) return true;
  for (uint32_t it = 0; it < limit; ++it) {
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
// weights of tile x are in TMEM: four softmax warps and the tile's issuing warp meet.  A hardware barrier, which answers in
// tens of cycles where an mbarrier, in the shared memory that the products read at full rate, takes about 200.  Every warp
// passes it once per block whatever happened to its bounded waits, and both sides wait: a softmax warp that only arrived
// could, once its waits have run out, arrive again in the same generation and leave the others one short for ever.  (It has
// nothing to do before the products that the issuing warp starts here, so waiting costs it nothing.)
__device__ __forceinline__ void weights_ready(int x) { asm volatile("bar.sync %0, 160;\n" ::"r"(2 + x) : "memory"); }
__device__ __forceinline__ void weights_wait(int x) { asm volatile("bar.sync %0, 160;\n" ::"r"(2 + x) : "memory"); }

// The issuing warps of the two tiles take turns, one block's products each, so that one tile's softmax runs under the
// other's products; without turns the tiles fall into step in many CTAs, and both halves of the work wait for each other.
// Handed over by hardware barriers too (a warp that gave its turn waits for the other's before it gives again, so one
// arrival per generation is sure); an issue returns when all but a product or two are done, so the tensor core sees hardly a
// gap.
__device__ __forceinline__ void turn_wait(int x) { asm volatile("bar.sync %0, 64;\n" ::"r"(4 + x) : "memory"); }
__device__ __forceinline__ void turn_give(int x) { asm volatile("bar.arrive %0, 64;\n" ::"r"(4 + x) : "memory"); }

}  // namespace

template <int D>
__global__ void __launch_bounds__(NTHR, 1) attn_chunk_kernel(const PagedArgs a, const __grid_constant__ CUtensorMap tk,
                                                             const __grid_constant__ CUtensorMap tv, uint32_t neg) {
  using C = Cfg<D>;
  extern __shared__ uint8_t raw[];
  __shared__ Bars bars;
  __shared__ Cursor cursors[11], ahead[8];  // every warp walks its own, out of registers; the softmax also looks ahead
  __shared__ int has_work;
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint8_t *qs = sm, *ring = sm + 2 * C::QT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  volatile int *dead = &bars.dead;

  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(smem_u32(&bars.full[i]), 1);
      mbar_init(smem_u32(&bars.empty[i]), 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.q_full[i]), 4);
      mbar_init(smem_u32(&bars.s_full[i]), 1);
      mbar_init(smem_u32(&bars.o_full[i]), 1);
    }
    mbar_init(smem_u32(&bars.drain[0]), 1);
    mbar_init(smem_u32(&bars.drain[1]), 1);
    bars.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (a.expire) {  // before TMEM is taken or any copy asked for
    pdl_trigger();
    pdl_wait();
    if (tid == 0) {
      a.hdr[cta] = make_int4(0, 0, 0, 0);
      wait(&bars.full[0], 0, dead, 1024);
      a.status[cta] = *dead;
    }
    return;
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&bars.tmem), TM_COLS);
    tmem_relinquish();
  }
  pdl_trigger();
  pdl_wait();
  SeqInfo *seqs = reinterpret_cast<SeqInfo *>(ring);  // the search uses the ring's memory
  cursor_prepare<NTHR>(a, seqs);
  if (warp == 0) {
    const int found = cursor_begin_one_warp<MT, BN>(a, cursors[0], seqs);
    if (lane == 0) has_work = found;
  }
  fence_async_smem();
  fence_before();
  __syncthreads();
  fence_after();
  if (const int found = has_work; found == 2) {  // a batch too large for one warp
    __syncthreads();                             // everyone has read it
    if (tid < SOFT) {
      Cursor c;
      const bool some = cursor_begin_any<SOFT, MT, BN>(a, c, *reinterpret_cast<PlanSmem<SOFT> *>(ring));
      if (tid == 0) {
        cursors[0] = c;
        has_work = some;
      }
      fence_async_smem();
    }
    __syncthreads();
  }
  if (warp > 0 && warp < 11 && lane == 0) cursors[warp] = cursors[0];
  if (tid == 0 && !cursors[0].works()) has_work = 0;
  __syncthreads();
  bool more = has_work;
  const uint32_t tmem = bars.tmem;

  // registers: 128 * (2 * 224 + 56) = 384 * 168, those of the launch
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n");
  if (warp == 9) {
    // ------------------------------------------------------------ loader
    Cursor &cur = cursors[9];
    const int P = 1 << a.log2P, box = min(P, BN), pieces = BN / box;
    const int piece = lane / C::HALVES, half = lane % C::HALVES;
    uint32_t st = 0, ph = 0;  // next stage and its parity
    uint32_t issued = 0;      // stages ever filled
    bool ok = true;
    while (more) {
      int b0, b1;
      bool first, last;
      const int n = cursor_piece(cur, b0, b1, first, last);
      const int *trow = a.table + (long long)cur.n * a.table_stride;
      const int lo = cur.w.lo, hi = cur.w.hi, kvh = cur.h;
      int t = (cur.w.blk0 + b0) * BN + piece * box;
      for (int b = b0; b < b1 && ok; ++b, t += BN) {
        int page = a.num_pages;  // zeros
        if (piece < pieces && t < hi && t + box > lo) {
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
            tma_load_4d(smem_u32(ring + st * C::STAGE + half * (BN * 128) + piece * box * 128), kv ? &tv : &tk, half * 64, kvh, off,
                        page, smem_u32(&bars.full[st]));
          ++issued;
          if (++st == C::STAGES) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      __syncwarp();
      more = cursor_advance(a, cur, n);
    }
    if (lane == 0) bars.stages = make_uint3(st, ph, min(issued, (uint32_t)C::STAGES));
  } else if (warp != 11) {
    // ------------------------------------------------------------ products of tile x
    const int x = (warp - 8) >> 1;
    Cursor &cur = cursors[warp];
    const uint32_t id_s = idesc_bf16(128, BN, false, false, neg != 0), id_o = idesc_bf16(128, D, false, true);
    const uint32_t ts = tmem + TM_S + x * BN, to = tmem + TM_O + x * D;
    uint32_t st = 0, ph = 0, pq = 0;  // ring stage and its parity, parity of the tile's query barrier
    bool ok = true;                   // no wait of this warp has expired
    auto next = [&] {
      if (++st == C::STAGES) {
        st = 0;
        ph ^= 1;
      }
    };
    auto scores = [&](uint32_t stage) {  // S = Q K^T
      const SDesc q = sdesc_s(opaque(smem_u32(qs + x * C::QT)), 16, 1024);
      const SDesc k = sdesc_s(opaque(smem_u32(ring + stage * C::STAGE)), 16, 1024);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t o = (i >> 2) * (BN * 128) + (i & 3) * 32;
        mma_f16s(ts, q + o, k + o, id_s, i > 0);
      }
      mma_commit(smem_u32(&bars.s_full[x]));
      mma_commit(smem_u32(&bars.empty[stage]));
    };
    auto sums = [&](uint32_t stage, bool acc) {  // O += P V
      const SDesc v = sdesc_s(opaque(smem_u32(ring + stage * C::STAGE)), BN * 128, 1024);
#pragma unroll
      for (int i = 0; i < BN / 16; ++i) mma_ts(to, ts + 8 * i, v + i * 2048, id_o, acc || i > 0);
    };
    if (x == 1) turn_give(0);  // tile 0 begins
    while (more) {
      int b0, b1;
      bool first, last;
      const int n = cursor_piece(cur, b0, b1, first, last);
      const bool both = cur.w.rows > 128;
      if (b0 < b1 && x * 128 >= cur.w.rows) {  // no such tile here: only hand the stages back
        for (int i = 0; i < 2 * (b1 - b0); ++i) {
          ok = ok && wait(&bars.full[st], ph, dead);
          if (lane == 0) mbar_arrive(smem_u32(&bars.empty[st]));
          next();
        }
      } else if (b0 < b1) {
        ok = ok && wait(&bars.q_full[x], pq, dead);
        pq ^= 1;
        ok = ok && wait(&bars.full[st], ph, dead);  // keys of the first block
        if (both) turn_wait(x);
        fence_after();
        if (ok && elect1()) scores(st);
        __syncwarp();
        if (both) turn_give(x ^ 1);
        next();
        int r_lo = cur.w.lo - (cur.w.blk0 + b0) * BN, r_hi = cur.w.hi - (cur.w.blk0 + b0) * BN;
        for (int b = b0; b < b1; ++b, r_lo -= BN, r_hi -= BN) {
          // values of the block and keys of the next, while the softmax works
          const uint32_t vst = st;
          ok = ok && wait(&bars.full[vst], ph, dead);
          if (r_lo > 0 || r_hi < BN) {
            // value rows that no query sees become zeros: whatever those slots hold, zero weights keep them out (the
            // warps of both tiles write the same zeros)
            uint4 *v = reinterpret_cast<uint4 *>(ring + vst * C::STAGE);
            for (int i = lane; i < BN * 8 * C::HALVES; i += 32) {
              const int r = (i >> 3) & (BN - 1);
              if (r < r_lo || r >= r_hi) v[i] = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            __syncwarp();
          }
          next();
          const bool has_next = b + 1 < b1;
          const uint32_t kst = st;
          if (has_next) {
            ok = ok && wait(&bars.full[kst], ph, dead);
            next();
          }
          weights_wait(x);
          if (both) turn_wait(x);
          fence_after();
          if (ok && elect1()) {
            sums(vst, b > b0);
            if (has_next) scores(kst);
            else mma_commit(smem_u32(&bars.o_full[x]));
          }
          __syncwarp();
          if (both) turn_give(x ^ 1);
          if (ok && elect1()) mma_commit(smem_u32(&bars.empty[vst]));
          __syncwarp();
        }
      }
      __syncwarp();
      more = cursor_advance(a, cur, n);
    }
    if (x == 0) turn_wait(0);  // the turn that was given last
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;\n");
    // ------------------------------------------------------------ softmax of tile x
    Cursor &cur = cursors[warp];
    bool cut = false;  // this CTA's header is written
    const int x = warp >> 2, wr = (warp & 3) * 32 + lane;  // row in the tile
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + TM_S + x * BN, to = tmem + lane_base + TM_O + x * D;
    uint32_t ps = 0, po = 0;
    bool ok = true;
    // The warp's 32 query rows of the piece at cursor c, asked for but not waited for: 16 bytes a lane, neighbours in a
    // row; every lane finds its own row and hands the address on.  False when the piece has no products of this tile.
    auto load_q = [&](const Cursor &c) {
      int b0, b1;
      bool first, last;
      cursor_piece(c, b0, b1, first, last);
      const int rows = c.w.rows - x * 128;
      if (b0 >= b1 || rows <= 0) return false;
      int tok, head;
      row_place(a, c, MT, x * 128 + (wr < rows ? wr : 0), tok, head);
      const unsigned long long mine = reinterpret_cast<unsigned long long>(static_cast<const bf16 *>(a.q) + tok * a.q_tok + head * a.q_head);
      constexpr int CPR = D / 8, RPI = 32 / CPR;  // chunks of a row, rows of one instruction
      uint8_t *qt = qs + x * C::QT;
      const int ch = lane % CPR;
#pragma unroll
      for (int i = 0; i < 32 / RPI; ++i) {
        const int sub = i * RPI + lane / CPR, r = (warp & 3) * 32 + sub;
        const unsigned long long p = __shfl_sync(0xffffffffu, mine, sub);
        cp_async16(qt + (ch >> 3) * (128 * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4),
                   reinterpret_cast<const void *>(p + ch * 16), r < rows);
      }
      return true;
    };
    auto q_arrived = [&](bool pending) {
      if (!pending) return;
      cp_async_wait_all();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.q_full[x]));
    };
    q_arrived(more && load_q(cur));
    while (more) {
      int b0, b1;
      bool first, last;
      const int n = cursor_piece(cur, b0, b1, first, last);
      const int rows = cur.w.rows - x * 128;  // of this tile
      // the next piece, found while this one's first scores are on their way
      if (lane == 0) ahead[warp] = cur;
      __syncwarp();
      const bool more_next = cursor_advance(a, ahead[warp], n);
      auto next_q = [&] { return more_next && load_q(ahead[warp]); };
      if (rows <= 0) q_arrived(next_q());
      if (rows > 0) {
        const int row = x * 128 + wr;
        const bool live = wr < rows;
        int pos = -1;
        if (live) {
          int tok, head;
          row_place(a, cur, MT, row, tok, head);
          pos = cur.s.kv - cur.s.qlen + tok - cur.s.qbeg;
        }
        float m = live ? -INFINITY : 0.f, l = 0.f;
        bool pending = false;
        if (b0 >= b1) pending = next_q();
        if (b0 < b1) {
          int t0 = (cur.w.blk0 + b0) * BN;
          for (int b = b0; b < b1; ++b, t0 += BN) {
            ok = ok && wait(&bars.s_full[x], ps, dead);
            ps ^= 1;
            fence_after();
            // the last scores of the piece are there, so its queries are done with: the next ones come meanwhile
            if (b == b1 - 1) pending = next_q();
            // Weights against the maximum as it stands, without looking for a new one.  Their sum tells whether that
            // will do: below 2^40 so is every weight, and sums and products stay far inside fp32 (bf16 has the same
            // exponents).  Above it, or while a row has no maximum yet, the maximum is taken and the weights are formed
            // anew from the scores, which stay in TMEM until the weights replace them.
            uint32_t s[BN], w[BN / 2];
            float part;
            for (bool raise = __any_sync(0xffffffffu, m == -INFINITY);; raise = true) {
#pragma unroll
              for (int i = 0; i < BN / 32; ++i) tmem_ld32_nw(ts + 32 * i, s + 32 * i);
              tmem_wait_ld();
              if (__any_sync(0xffffffffu, t0 + BN - 1 > pos || (a.window && t0 <= pos - a.window))) {
                const int hi = pos - t0, lo = a.window ? pos - a.window - t0 : -1;
#pragma unroll
                for (int i = 0; i < BN; ++i)
                  if (i > hi || i <= lo) s[i] = 0xff800000u;
              }
              if (raise) {
                float mx[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) mx[k] = __uint_as_float(s[k]);
#pragma unroll
                for (int i = 4; i < BN; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i]));
                const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2);
                const float f = mn == -INFINITY ? 1.f : ex2(m - mn);
                m = mn;
                l *= f;
                if (b > b0) {
                  // the products that wrote O completed before this tile's scores did, the next wait for the weights
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
              uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
              for (int i = 0; i < BN / 2; ++i) {
                float p0, p1;
                upk(fma2(pk(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sc, nm), p0, p1);
                p0 = ex2(p0);
                p1 = ex2(p1);
                sum[i & 3] = add2(sum[i & 3], pk(p0, p1));
                w[i] = pack_bf16(p0, p1);
              }
              float u0, u1;
              upk(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), u0, u1);
              part = u0 + u1;
              if (raise || !__any_sync(0xffffffffu, part > RAISED)) break;
            }
            l += part;
            tmem_st32_nw(ts, w);
            tmem_st32_nw(ts + 32, w + 32);
            tmem_wait_st();
            fence_before();
            weights_ready(x);
          }
          q_arrived(pending);
          pending = false;
          ok = ok && wait(&bars.o_full[x], po, dead);
          po ^= 1;
          fence_after();
        }
        q_arrived(pending);
        {
          const bool whole = first && last;
          int tok, head;
          row_place(a, cur, MT, live ? row : 0, tok, head);
          const int slot = first ? 1 : 0;
          float *rec = a.part + ((long long)cta * 2 + slot) * record_floats(MT, D);
          const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
          const unsigned long long op = reinterpret_cast<unsigned long long>(static_cast<bf16 *>(a.o) + tok * a.o_tok + head * a.o_head);
          // 16 rows by 64 features at a time.  The lane holds two neighbouring features of rows g and g + 8 in each of
          // eight 8-feature groups; a transposition among the four lanes of a row gives each 32 bytes, so that a store
          // of the warp fills whole lines (one row to a thread, 32 lines to a store, took 2 us of a piece).
          const int g = lane >> 2, qd = lane & 3;
#pragma unroll 1
          for (int hb = 0; hb < 2; ++hb) {
#pragma unroll
            for (int cb = 0; cb < D / 64; ++cb) {
              uint32_t o[32];
              if (b0 < b1) {
                tmem_ld16x64(to + ((uint32_t)(16 * hb) << 16) + 64 * cb, o);
                tmem_wait_ld();
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0;
              }
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int sub = 16 * hb + 8 * e + g;  // the row in the warp's 32
                const bool there = (warp & 3) * 32 + sub < rows;
                if (whole) {
                  const float f = __shfl_sync(0xffffffffu, inv, sub);
                  const unsigned long long at = __shfl_sync(0xffffffffu, op, sub) + 2 * (64 * cb + 16 * qd);
                  uint32_t t[4][2], w[8];
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    t[i >> 1][i & 1] = pack_bf16(__uint_as_float(o[4 * i + 2 * e]) * f, __uint_as_float(o[4 * i + 2 * e + 1]) * f);
                  quad_transpose(t, qd);
#pragma unroll
                  for (int i = 0; i < 8; ++i) w[i] = t[i & 3][i >> 2];
                  if (there) {
                    if ((at & 31) == 0) {
                      st_global_32b(reinterpret_cast<void *>(at), w);
                    } else {
                      reinterpret_cast<uint4 *>(at)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                      reinterpret_cast<uint4 *>(at)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                  }
                } else {
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf) {
                    uint32_t t[4][2], w[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      t[i][0] = o[16 * hf + 4 * i + 2 * e];
                      t[i][1] = o[16 * hf + 4 * i + 2 * e + 1];
                    }
                    quad_transpose(t, qd);
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = t[i >> 1][i & 1];
                    if (there) st_global_32b(rec + (size_t)(x * 128 + (warp & 3) * 32 + sub) * D + 64 * cb + 32 * hf + 8 * qd, w);
                  }
                }
              }
            }
          }
          if (live) {
            if (whole) {
              if (a.lse) a.lse[(long long)tok * a.Hq + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            } else {
              rec[(size_t)MT * D + row] = m;
              rec[(size_t)MT * D + MT + row] = l;
            }
          }
          fence_before();
        }
      }
      if (first && !last) {
        cut = true;
        if (tid == 0) a.hdr[cta] = cut_header<MT>(a, cur);
      }
      __syncwarp();
      if (lane == 0) cur = ahead[warp];
      __syncwarp();
      more = more_next;
    }
    if (tid == 0 && !cut) a.hdr[cta] = make_int4(0, 0, 0, 0);
  }
  fence_before();
  __syncthreads();
  fence_after();
  // A CTA in which a wait ran out waits (bounded) for what is in flight before its memory goes, once every role has ended:
  // none starts a copy or a product any more, and all see the same `dead`.
  if (bars.dead) {
    if (warp == 9) {  // the copies of the stages filled last
      uint32_t st = bars.stages.x, ph = bars.stages.y;
      for (uint32_t i = 0; i < bars.stages.z; ++i) {
        if (st == 0) {
          st = C::STAGES;
          ph ^= 1;
        }
        --st;
        mbar_wait(smem_u32(&bars.full[st]), ph, nullptr, 0, DRAIN_LIMIT);
      }
    } else if (warp == 8 || warp == 10) {  // the products of the tile
      const int x = (warp - 8) >> 1;
      if (elect1()) mma_commit(smem_u32(&bars.drain[x]));
      __syncwarp();
      mbar_wait(smem_u32(&bars.drain[x]), 0, nullptr, 0, DRAIN_LIMIT);
    }
    __syncthreads();
  }
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
