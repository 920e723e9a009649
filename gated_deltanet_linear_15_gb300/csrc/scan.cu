// Gated linear recurrence, one state per channel (the elementwise sister of the delta rule, whose gate it shares):
//   h_t = exp(g_t) h_{t-1} + x_t,  y_t = h_t;
// backward, with d_t the gradient that reaches h_t:
//   d_t = dy_t + exp(g_{t+1}) d_{t+1},  dx_t = d_t,  dg_t = exp(g_t) d_t h_{t-1},  dh0 = exp(g_0) d_0.
//
// Bound by bytes: x and g are read once and y is written once; the backward reads dy, x and g and writes dx and dg.
//
// All sequences stand in one line of tokens, cut into segments of SEG = 16 tokens at multiples of 16.  A warp holds a
// segment of CB = 64 channels, two per lane: it runs the recurrence from zero, which gives the segment's map
// c -> A c + H with A = exp(sum of g), and again from the true state once that is known.  The warps of a CTA take
// consecutive segments, so do the CTAs of a cluster (the line is cut among up to eight of them where channels and
// sequences alone leave SMs without work); maps meet in shared memory, within a cluster in that of every CTA, and each warp
// walks through those before its own.  A round is one segment per warp; the state after a round goes to the next in
// registers.  No CTA waits for another outside its cluster.  Taking A from the sum of the log-gates keeps the state's error
// at one rounding per 16 tokens where a channel remembers thousands of them.
//
// Rows come by cp.async into a ring of stages that belongs to the warp, so that loads are in flight during the
// arithmetic and no barrier is needed for them.  A sequence's first token takes its state from h0 (the segment's map
// forgets what came before), its last one writes the final state.
//
// The forward may leave the state before every segment (fp32, 4 bytes for 16 tokens and channel, 1/4 byte a value).  The
// backward runs each segment forward again from there, in registers, and then backward the way the forward goes: what it
// multiplies is the unrounded fp32 state, for as many bytes as reading the rounded y would take.
#include <algorithm>

#include "block.h"
#include "common.cuh"

namespace gdn {

namespace {

constexpr int SEG = SCAN_SEG, CB = 64, STAGES = 3, MAXC = 8;  // MAXC: CTAs of a cluster

// what moves rows: 16-byte pieces, 4-byte pieces, or single bf16 elements
enum Move { M16, M4, M2 };
// a lane's two channels of a block: neighbours, or 32 apart where two neighbours have no common access
template <typename X, int M> struct Lanes {
  static constexpr bool PAIR = M == M16 || (M == M4 && sizeof(X) == 2);
  static __device__ __forceinline__ int first(int lane) { return PAIR ? 2 * lane : lane; }
};

// rows t0 .. t0 + 15, channels c0 .. c0 + 63 of src come to dst [SEG][CB]; zeros outside [lo, hi) x [0, D)
template <typename E, int M>
__device__ __forceinline__ void load_rows(E *dst, const E *src, long long row, int t0, int lo, int hi, int c0, int D) {
  const int lane = threadIdx.x & 31;
  if constexpr (M == M2) {
#pragma unroll
    for (int r = 0; r < SEG; ++r) {
      const bool ok = t0 + r >= lo && t0 + r < hi;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = lane + 32 * k;
        E v = fromf<E>(0.f);
        if (ok && c0 + c < D) v = src[(long long)(t0 + r) * row + c0 + c];
        dst[r * CB + c] = v;
      }
    }
  } else {
    constexpr int B = M == M16 ? 16 : 4, V = B / (int)sizeof(E), PER = CB / V;  // pieces of a row
    constexpr int RPI = PER < 32 ? 32 / PER : 1, CPI = PER < 32 ? PER : 32;       // rows and pieces of one instruction
    const int r0 = lane / CPI;
#pragma unroll
    for (int k = 0; k < PER / CPI; ++k) {
      const int c = (lane % CPI + 32 * k) * V;
      const unsigned span = c0 + c < D ? hi - lo : 0, rel = t0 + r0 - lo;
      const E *s = src + (long long)(t0 + r0) * row + c0 + c;
#pragma unroll
      for (int i = 0; i < SEG / RPI; ++i, s += RPI * row) {
        const bool ok = rel + i * RPI < span;
        E *d = dst + (r0 + i * RPI) * CB + c;
        if constexpr (M == M16) cp_async16(d, ok ? s : src, ok);
        else cp_async4(d, ok ? s : src, ok);
      }
    }
  }
}
// the lane's two values of a row in shared memory
template <typename E, int M> __device__ __forceinline__ uint64_t get2(const E *row, int lane) {
  using L = Lanes<E, M>;
  if constexpr (L::PAIR && sizeof(E) == 2) {
    const uint32_t u = *reinterpret_cast<const uint32_t *>(row + 2 * lane);
    return pk(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  } else if constexpr (L::PAIR) {
    return *reinterpret_cast<const uint64_t *>(row + 2 * lane);
  } else {
    return pk(tof(row[lane]), tof(row[lane + 32]));
  }
}
// Gates of a row.  With bf16 rows the product with log2(e) and ex2.approx, off by 2^-22 of themselves, which a bf16 result does
// not show and which the state carries for 16 tokens at most (its map takes expf of the sum); expf in fp32, where 16 such
// errors would be half of all.
template <bool EXACT> __device__ __forceinline__ uint64_t gates(uint64_t g) {
  float a, b;
  if constexpr (EXACT) {
    upk(g, a, b);
    return pk(expf(a), expf(b));
  } else {
    upk(mul2(g, pk(1.4426950408889634f, 1.4426950408889634f)), a, b);
    asm("ex2.approx.ftz.f32 %0, %0;\n" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;\n" : "+f"(b));
    return pk(a, b);
  }
}
// a row of a block, the lane's channels, of which c is the first; only those below D exist
template <typename E, bool PAIR> __device__ __forceinline__ void put2(E *row, int c, int D, uint64_t p) {
  float u, v;
  upk(p, u, v);
  if constexpr (PAIR) {
    if (c < D) st2(row + c, u, v);
  } else {
    if (c < D) row[c] = fromf<E>(u);
    if (c + 32 < D) row[c + 32] = fromf<E>(v);
  }
}
template <bool PAIR> __device__ __forceinline__ uint64_t take2(const float *row, int c, int D) {
  if constexpr (PAIR) return c < D ? *reinterpret_cast<const uint64_t *>(row + c) : 0;
  else return pk(c < D ? row[c] : 0.f, c + 32 < D ? row[c + 32] : 0.f);
}

// ------------------------------------------------------------------ where sequences begin
// Tokens of the line that a part takes: whole sequences.  Packed sequences go by where they begin, so that parts are of
// about the same size; equal ones by number.
__device__ __forceinline__ int lower_bound(const int *cu, int n, int v) {  // entries of cu[0 .. n) below v
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}
__device__ __forceinline__ int part_begin(const ScanArgs &a, int p, int parts) {
  if (!a.cu) return (int)((long long)a.N * p / parts) * a.T;
  int at = p == 0 ? 0 : (p == parts ? a.N : lower_bound(a.cu, a.N + 1, (int)((long long)a.tokens * p / parts)));
  at = min(at, a.N);
  return min(max(a.cu[at], 0), a.tokens);
}

// The boundaries between sequences around a warp's segment.  With cu, each lane holds one entry of a window that begins at
// entry `base`; it moves with the segments.
struct Bounds {
  int base, e;
  int left;  // windows that may still be looked at: a cu that is not sorted ends the walk, not the kernel
  __device__ __forceinline__ void load(const ScanArgs &a) {
    const int i = base + (threadIdx.x & 31);
    e = i <= a.N ? a.cu[i] : 0x7fffffff;
  }
  __device__ __forceinline__ void init(const ScanArgs &a, int t) {
    left = a.N / 8 + 64;
    base = 0;
    e = 0;
    if (!a.cu) return;
    base = max(lower_bound(a.cu, a.N + 1, t + 1) - 1, 0);
    load(a);
  }
  // moves the window to token t: its first entry is the last one at or before t, or near it
  __device__ __forceinline__ void seek(const ScanArgs &a, int t) {
    if (!a.cu) return;
    for (; left > 0; --left) {
      const unsigned at = __ballot_sync(0xffffffffu, e <= t);
      if (at == 0xffffffffu && base + 31 <= a.N) base += 31;
      else if (!(at & 1) && base > 0) base = max(base - 31, 0);
      else break;
      load(a);
    }
  }
  // bit i (of 17): some sequence begins, or the last one ends, at token t + i.  The window stands at t.
  __device__ __forceinline__ uint32_t mask(const ScanArgs &a, int t) {
    const int lane = threadIdx.x & 31;
    if (!a.cu) return __ballot_sync(0xffffffffu, lane <= SEG && (unsigned)(t + lane) % (unsigned)a.T == 0);
    uint32_t m = 0;
    int b = base, x = e;
    for (int k = 0; k <= a.N / 31 + 1; ++k) {
      const unsigned d = (unsigned)(x - t);
      m |= __reduce_or_sync(0xffffffffu, d <= SEG ? 1u << d : 0u);
      if (__any_sync(0xffffffffu, x > t + SEG) || b + 31 > a.N) break;
      b += 31;
      x = b + lane <= a.N ? a.cu[b + lane] : 0x7fffffff;
    }
    return m;
  }
  // the sequence that holds token t, which is at or behind the window's first entry
  __device__ __forceinline__ int seq(const ScanArgs &a, int t) const {
    if (!a.cu) return (int)((unsigned)t / (unsigned)a.T);
    const int lane = threadIdx.x & 31;
    int b = base, x = e;
    for (int k = 0; k <= a.N / 31 + 1; ++k) {
      const unsigned at = __ballot_sync(0xffffffffu, x <= t);
      if (at != 0xffffffffu || b + 31 > a.N) return min(max(b + __popc(at) - 1, 0), a.N - 1);
      b += 31;
      x = b + lane <= a.N ? a.cu[b + lane] : 0x7fffffff;
    }
    return a.N - 1;
  }
};

// ------------------------------------------------------------------ maps of segments
// c -> A c + H; A < 0 marks one that forgets c (whatever c holds, an infinity among it)
struct Map2 {
  float A[2], H[2];
  __device__ __forceinline__ uint64_t apply(uint64_t p) const {
    float c[2];
    upk(p, c[0], c[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) c[k] = A[k] < 0.f ? H[k] : fmaf(A[k], c[k], H[k]);
    return pk(c[0], c[1]);
  }
  __device__ __forceinline__ void then(const Map2 &n) {  // this one first, then n
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      H[k] = n.A[k] < 0.f ? n.H[k] : fmaf(n.A[k], H[k], n.H[k]);
      A[k] = n.A[k] < 0.f || A[k] < 0.f ? -1.f : A[k] * n.A[k];
    }
  }
};
// of a segment: the sum of its log-gates and its result from zero
__device__ __forceinline__ float4 segment_map(bool fresh, uint64_t sum, uint64_t h) {
  float s0, s1, h0, h1;
  upk(sum, s0, s1);
  upk(h, h0, h1);
  return make_float4(fresh ? -1.f : expf(s0), fresh ? -1.f : expf(s1), h0, h1);
}
template <int W> struct Meet {
  float4 warp[2][W][32];     // by round parity: maps of the CTA's segments
  float4 peer[2][MAXC][32];  // of the cluster's CTAs
};
__device__ __forceinline__ Map2 map_of(const float4 &v) { return {{v.x, v.y}, {v.z, v.w}}; }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
// of a warp that has written nothing that peers read: it need not wait for its own stores
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void store_peer(const float4 *p, int rank, const float4 &v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// A round's exchange: every warp hands in its segment's map, and later gets the state before it; `carry` becomes the state
// after the round.
template <int W> __device__ __forceinline__ void hand_in(Meet<W> &mt, int buf, int cs, int rank, const float4 &mine) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  mt.warp[buf][warp][lane] = mine;
  __syncthreads();
  if (cs == 1) return;
  if (warp == 0) {
    Map2 all = map_of(mt.warp[buf][0][lane]);
#pragma unroll
    for (int j = 1; j < W; ++j) all.then(map_of(mt.warp[buf][j][lane]));
    for (int r = 0; r < cs; ++r) store_peer(&mt.peer[buf][rank][lane], r, make_float4(all.A[0], all.A[1], all.H[0], all.H[1]));
    cluster_arrive();
  } else {
    cluster_arrive_relaxed();
  }
}
template <int W> __device__ __forceinline__ uint64_t get_state(const Meet<W> &mt, int buf, int cs, int rank, uint64_t &carry) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t in = carry;
  if (cs == 1) {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if (j == warp) in = carry;
      carry = map_of(mt.warp[buf][j][lane]).apply(carry);
    }
    return in;
  }
  cluster_wait();
  for (int r = 0; r < cs; ++r) {
    if (r == rank) in = carry;
    carry = map_of(mt.peer[buf][r][lane]).apply(carry);
  }
  for (int j = 0; j < warp; ++j) in = map_of(mt.warp[buf][j][lane]).apply(in);
  return in;
}

template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// the state of sequences without tokens passes through: out[n] = in[n], shared out among a channel block's CTAs
template <bool PAIR, int W>
__device__ __forceinline__ void pass_empty(const ScanArgs &a, const float *in, float *out, int c, int ctas, int cta) {
  if (!a.cu || !out) return;
  for (int n = cta * W + (threadIdx.x >> 5); n < a.N; n += ctas * W) {
    if (a.cu[n + 1] > a.cu[n]) continue;
    put2<float, PAIR>(out + (long long)n * a.D, c, a.D, in ? take2<PAIR>(in + (long long)n * a.D, c, a.D) : 0);
  }
}

// Where a CTA's walk through its part stands.  Segments count in the direction of the walk: number 0 is the part's first
// one, or its last one going backward.
struct Walk {
  int lo, hi;        // tokens of the part
  int rounds, per;   // segments of a round: one for every warp of the cluster
  int first, last;   // the warp's segment of round 0; the line's segment with number 0 going backward
  template <int W> __device__ __forceinline__ void init(const ScanArgs &a, int cs, int rank) {
    lo = part_begin(a, blockIdx.z, gridDim.z);
    hi = part_begin(a, blockIdx.z + 1, gridDim.z);
    const int s0 = lo / SEG, ns = hi > lo ? (hi + SEG - 1) / SEG - s0 : 0;
    per = cs * W;
    rounds = (ns + per - 1) / per;
    first = s0 + rank * W + (threadIdx.x >> 5);
    last = 2 * s0 + ns - 1;
  }
  __device__ __forceinline__ int up(int k) const { return first + k * per; }
  __device__ __forceinline__ int down(int k) const { return last - (first + k * per); }
  __device__ __forceinline__ bool has(int seg) const { return seg * SEG < hi && (seg + 1) * SEG > lo; }
};
// A segment of a round.  One inside a sequence (plain) goes through unrolled code.  One with a boundary, or at a part's end,
// takes loops that look at every row, kept short: code for both in every row was five times as long, and its fetching took
// most of the time (4 x 4096 tokens of 2048 channels: 109 us forward).
struct Piece {
  int seg, t0;
  bool live, plain;
  uint32_t cut;  // boundaries
  Bounds bd;
  __device__ __forceinline__ void look(const ScanArgs &a, const Walk &w, int s) {
    seg = s;
    t0 = s * SEG;
    live = w.has(s);
    cut = 0;
    if (live) {
      bd.seek(a, t0);
      cut = bd.mask(a, t0);
    }
    plain = cut == 0 && t0 >= w.lo && t0 + SEG <= w.hi;
  }
  __device__ __forceinline__ bool inside(const Walk &w, int i) const { return t0 + i >= w.lo && t0 + i < w.hi; }
  __device__ __forceinline__ bool begins(int i) const { return cut >> i & 1; }
  __device__ __forceinline__ bool ends(int i) const { return cut >> (i + 1) & 1; }
};

}  // namespace

// grid: CTAs of a cluster, channel blocks, parts.  Each step hands in the maps of round k + 1 and, while the CTAs of the cluster
// meet, finishes round k, whose states are known.
template <typename X, typename G, int M, int W>
__global__ void __launch_bounds__(32 * W, 2) scan_fwd_kernel(ScanArgs a) {
  constexpr bool PAIR = Lanes<X, M>::PAIR, EXACT = sizeof(X) == 4;
  static_assert(Lanes<X, M>::PAIR == Lanes<G, M>::PAIR, "one layout of channels");
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ Meet<W> mt;
  constexpr int BX = SEG * CB * sizeof(X), ST = BX + SEG * CB * sizeof(G);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = gridDim.x, rank = blockIdx.x, c0 = blockIdx.y * CB, c = c0 + Lanes<X, M>::first(lane);
  uint8_t *ring = raw + warp * (STAGES * ST);
  if (cs > 1) cluster_arrive();  // peers have begun before anything is written to them
  pdl_trigger();
  pdl_wait();
  Walk w = {};
  w.init<W>(a, cs, rank);
  auto load = [&](int k, int slot) {
    if (k < w.rounds && w.has(w.up(k))) {
      uint8_t *st = ring + slot * ST;
      load_rows<X, M>(reinterpret_cast<X *>(st), static_cast<const X *>(a.x), a.x_row, w.up(k) * SEG, w.lo, w.hi, c0, a.D);
      load_rows<G, M>(reinterpret_cast<G *>(st + BX), static_cast<const G *>(a.g), a.g_row, w.up(k) * SEG, w.lo, w.hi, c0, a.D);
    }
    cp_async_commit();
  };
  load(0, 0);
  load(1, 1);
  Piece now = {}, next = {};
  next.bd.init(a, w.up(0) * SEG);
  pass_empty<PAIR, W>(a, a.h0, a.hT, c, cs * gridDim.z, blockIdx.z * cs + rank);
  if (cs > 1) cluster_wait();
  auto x_of = [&](const uint8_t *st, int i) { return get2<X, M>(reinterpret_cast<const X *>(st) + i * CB, lane); };
  auto g_of = [&](const uint8_t *st, int i) { return get2<G, M>(reinterpret_cast<const G *>(st + BX) + i * CB, lane); };
  auto start = [&](const Piece &p, int i) { return a.h0 ? take2<PAIR>(a.h0 + (long long)p.bd.seq(a, p.t0 + i) * a.D, c, a.D) : 0; };
  uint64_t carry = 0, h = 0;
  int slot = STAGES - 1;  // of round k
  for (int k = -1; k < w.rounds; ++k) {
    const int slot1 = slot + 1 == STAGES ? 0 : slot + 1;
    const bool more = k + 1 < w.rounds;
    if (more) {
      next.look(a, w, w.up(k + 1));
      cp_wait<1>();
      __syncwarp();
      const uint8_t *st = ring + slot1 * ST;
      uint64_t sum = 0, z = 0;
      bool fresh = false;
      if (next.plain) {
#pragma unroll
        for (int i = 0; i < SEG; ++i) {
          const uint64_t g = g_of(st, i);
          sum = add2(sum, g);
          z = fma2(gates<EXACT>(g), z, x_of(st, i));
        }
      } else if (next.live) {
#pragma unroll 1
        for (int i = 0; i < SEG; ++i) {
          const uint64_t g = g_of(st, i);
          if (next.begins(i) && next.inside(w, i)) {
            z = start(next, i);
            fresh = true;
          }
          sum = add2(sum, g);
          z = fma2(gates<EXACT>(g), z, x_of(st, i));
        }
      }
      hand_in(mt, k + 1 & 1, cs, rank, segment_map(fresh, sum, z));
    }
    if (k >= 0 && now.live) {
      const uint8_t *st = ring + slot * ST;
      if (a.states && now.t0 >= w.lo) put2<float, PAIR>(a.states + (long long)now.seg * a.D, c, a.D, h);
      X *yr = static_cast<X *>(a.y) + (long long)now.t0 * a.y_row;
      if (now.plain) {
#pragma unroll
        for (int i = 0; i < SEG; ++i, yr += a.y_row) {
          h = fma2(gates<EXACT>(g_of(st, i)), h, x_of(st, i));
          put2<X, PAIR>(yr, c, a.D, h);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < SEG; ++i, yr += a.y_row) {
          if (!now.inside(w, i)) continue;
          if (now.begins(i)) h = start(now, i);
          h = fma2(gates<EXACT>(g_of(st, i)), h, x_of(st, i));
          put2<X, PAIR>(yr, c, a.D, h);
          if (now.ends(i) && a.hT) put2<float, PAIR>(a.hT + (long long)now.bd.seq(a, now.t0 + i) * a.D, c, a.D, h);
        }
      }
    }
    __syncwarp();  // the stage is loaded again
    load(k + STAGES, slot);
    if (more) {
      h = get_state(mt, k + 1 & 1, cs, rank, carry);
      now = next;
    }
    slot = slot1;
  }
  cp_async_wait_all();
}

template <typename X, typename G, int M, int W>
__global__ void __launch_bounds__(32 * W, 2) scan_bwd_kernel(ScanArgs a) {
  constexpr bool PAIR = Lanes<X, M>::PAIR, EXACT = sizeof(X) == 4;
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ Meet<W> mt;
  constexpr int BX = SEG * CB * sizeof(X), ST = 2 * BX + SEG * CB * sizeof(G);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = gridDim.x, rank = blockIdx.x, c0 = blockIdx.y * CB, c = c0 + Lanes<X, M>::first(lane);
  uint8_t *ring = raw + warp * (STAGES * ST);
  if (cs > 1) cluster_arrive();
  pdl_trigger();
  pdl_wait();
  Walk w = {};
  w.init<W>(a, cs, rank);
  auto load = [&](int k, int slot) {
    if (k < w.rounds && w.has(w.down(k))) {
      uint8_t *st = ring + slot * ST;
      const int t = w.down(k) * SEG;
      load_rows<X, M>(reinterpret_cast<X *>(st), static_cast<const X *>(a.x), a.x_row, t, w.lo, w.hi, c0, a.D);
      load_rows<X, M>(reinterpret_cast<X *>(st + BX), static_cast<const X *>(a.dy), a.dy_row, t, w.lo, w.hi, c0, a.D);
      load_rows<G, M>(reinterpret_cast<G *>(st + 2 * BX), static_cast<const G *>(a.g), a.g_row, t, w.lo, w.hi, c0, a.D);
    }
    cp_async_commit();
  };
  load(0, 0);
  load(1, 1);
  Piece now = {}, next = {};
  next.bd.init(a, max(w.down(0) * SEG, 0));
  pass_empty<PAIR, W>(a, a.dhT, a.dh0, c, cs * gridDim.z, blockIdx.z * cs + rank);
  if (cs > 1) cluster_wait();
  auto x_of = [&](const uint8_t *st, int i) { return get2<X, M>(reinterpret_cast<const X *>(st) + i * CB, lane); };
  auto dy_of = [&](const uint8_t *st, int i) { return get2<X, M>(reinterpret_cast<const X *>(st + BX) + i * CB, lane); };
  auto g_of = [&](const uint8_t *st, int i) { return get2<G, M>(reinterpret_cast<const G *>(st + 2 * BX) + i * CB, lane); };
  auto start = [&](const Piece &p, int i) { return a.h0 ? take2<PAIR>(a.h0 + (long long)p.bd.seq(a, p.t0 + i) * a.D, c, a.D) : 0; };
  auto at_end = [&](const Piece &p, int i) { return a.dhT ? take2<PAIR>(a.dhT + (long long)p.bd.seq(a, p.t0 + i) * a.D, c, a.D) : 0; };
  uint64_t carry = 0, d = 0;  // d: what reaches the state from later tokens
  uint64_t h = 0, h1 = 0;     // stored states before the segments of rounds k and k + 1
  int slot = STAGES - 1;
  for (int k = -1; k < w.rounds; ++k) {
    const int slot1 = slot + 1 == STAGES ? 0 : slot + 1;
    const bool more = k + 1 < w.rounds;
    if (more) {
      next.look(a, w, w.down(k + 1));
      h1 = next.live ? take2<PAIR>(a.states + (long long)next.seg * a.D, c, a.D) : 0;
      cp_wait<1>();
      __syncwarp();
      const uint8_t *st = ring + slot1 * ST;
      uint64_t sum = 0, z = 0;
      bool fresh = false;
      if (next.plain) {
#pragma unroll
        for (int i = SEG - 1; i >= 0; --i) {
          const uint64_t g = g_of(st, i);
          sum = add2(sum, g);
          z = mul2(gates<EXACT>(g), add2(dy_of(st, i), z));
        }
      } else if (next.live) {
#pragma unroll 1
        for (int i = SEG - 1; i >= 0; --i) {
          const uint64_t g = g_of(st, i);
          if (next.ends(i) && next.inside(w, i)) {
            z = at_end(next, i);
            fresh = true;
          }
          sum = add2(sum, g);
          z = mul2(gates<EXACT>(g), add2(dy_of(st, i), z));
        }
      }
      hand_in(mt, k + 1 & 1, cs, rank, segment_map(fresh, sum, z));
    }
    if (k >= 0 && now.live) {
      const uint8_t *st = ring + slot * ST;
      X *dxr = static_cast<X *>(a.y) + (long long)(now.t0 + SEG - 1) * a.y_row;
      G *dgr = static_cast<G *>(a.dg) + (long long)(now.t0 + SEG - 1) * a.dg_row;
      if (now.plain) {
        uint64_t al[SEG], hp[SEG];  // gates, and states before the tokens
#pragma unroll
        for (int i = 0; i < SEG; ++i) {
          hp[i] = h;
          al[i] = gates<EXACT>(g_of(st, i));
          h = fma2(al[i], h, x_of(st, i));
        }
#pragma unroll
        for (int i = SEG - 1; i >= 0; --i, dxr -= a.y_row, dgr -= a.dg_row) {
          const uint64_t dx = add2(dy_of(st, i), d);
          d = mul2(al[i], dx);
          put2<X, PAIR>(dxr, c, a.D, dx);
          put2<G, PAIR>(dgr, c, a.D, mul2(d, hp[i]));
        }
      } else {
        uint64_t hp[SEG];  // in local memory
#pragma unroll 1
        for (int i = 0; i < SEG; ++i) {
          if (now.begins(i) && now.inside(w, i)) h = start(now, i);
          hp[i] = h;
          h = fma2(gates<EXACT>(g_of(st, i)), h, x_of(st, i));
        }
#pragma unroll 1
        for (int i = SEG - 1; i >= 0; --i, dxr -= a.y_row, dgr -= a.dg_row) {
          if (!now.inside(w, i)) continue;
          if (now.ends(i)) d = at_end(now, i);
          const uint64_t dx = add2(dy_of(st, i), d);
          d = mul2(gates<EXACT>(g_of(st, i)), dx);
          put2<X, PAIR>(dxr, c, a.D, dx);
          put2<G, PAIR>(dgr, c, a.D, mul2(d, hp[i]));
          if (now.begins(i) && a.dh0) put2<float, PAIR>(a.dh0 + (long long)now.bd.seq(a, now.t0 + i) * a.D, c, a.D, d);
        }
      }
    }
    __syncwarp();
    load(k + STAGES, slot);
    if (more) {
      d = get_state(mt, k + 1 & 1, cs, rank, carry);
      now = next;
      h = h1;
    }
    slot = slot1;
  }
  cp_async_wait_all();
}

// One token of every sequence: state = exp(g) state + x, y = state.  V channels a thread.
template <typename X, typename G, int V> __global__ void __launch_bounds__(256) scan_step_kernel(ScanArgs a) {
  pdl_trigger();
  pdl_wait();
  const int n = blockIdx.y + blockIdx.z * 65535, c = (blockIdx.x * 256 + threadIdx.x) * V;
  if (n >= a.N || c >= a.D) return;
  const X *x = static_cast<const X *>(a.x) + n * a.x_row + c;
  const G *g = static_cast<const G *>(a.g) + n * a.g_row + c;
  float *h = a.hT + n * a.h_row + c;
  X *y = static_cast<X *>(a.y) + n * a.y_row + c;
  if constexpr (V == 4) {
    float xv[4], gv[4];
    auto get4 = [](const auto *p, float (&v)[4]) {
      if constexpr (sizeof(*p) == 2) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        v[0] = __uint_as_float(u.x << 16);
        v[1] = __uint_as_float(u.x & 0xffff0000u);
        v[2] = __uint_as_float(u.y << 16);
        v[3] = __uint_as_float(u.y & 0xffff0000u);
      } else {
        const float4 u = *reinterpret_cast<const float4 *>(p);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
      }
    };
    get4(x, xv);
    get4(g, gv);
    float4 s = *reinterpret_cast<const float4 *>(h);
    s.x = fmaf(expf(gv[0]), s.x, xv[0]);
    s.y = fmaf(expf(gv[1]), s.y, xv[1]);
    s.z = fmaf(expf(gv[2]), s.z, xv[2]);
    s.w = fmaf(expf(gv[3]), s.w, xv[3]);
    *reinterpret_cast<float4 *>(h) = s;
    if constexpr (sizeof(X) == 2) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(s.x, s.y), q = __floats2bfloat162_rn(s.z, s.w);
      *reinterpret_cast<uint2 *>(y) = make_uint2(*reinterpret_cast<const uint32_t *>(&p), *reinterpret_cast<const uint32_t *>(&q));
    } else {
      *reinterpret_cast<float4 *>(y) = s;
    }
  } else {
    const float s = fmaf(expf(tof(g[0])), h[0], tof(x[0]));
    h[0] = s;
    y[0] = fromf<X>(s);
  }
}

namespace {

// The split of a call: parts of whole sequences and CTAs of a cluster, for two CTAs per SM.  Equal sequences go to
// parts first, which exchange nothing; packed ones may be one long sequence and many short ones, so there the line is cut
// within a cluster first.
void split(const ScanArgs &a, int W, int sms, int &parts, int &cs) {
  const int nb = (a.D + CB - 1) / CB, want = std::max(1, 2 * sms / nb);  // CTAs of a channel block
  const auto clustered = [&](int most, long long tokens) {
    return (int)std::max(1ll, std::min({(long long)most, (long long)MAXC, tokens / (W * SEG)}));
  };
  if (!a.cu) {
    parts = std::min(a.N, want);
    cs = clustered(want / parts, a.tokens / parts);
  } else {
    cs = clustered(want, a.tokens);
    parts = std::min(a.N, std::max(1, want / cs));
  }
  parts = std::min(parts, 65535);
}

template <int W, typename... KArgs>
cudaError_t launch_clustered(void (*k)(KArgs...), const ScanArgs &a, int sms, int row_bytes, cudaStream_t st) {
  const size_t smem = (size_t)W * STAGES * SEG * CB * row_bytes;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  int parts, cs;
  split(a, W, sms, parts, cs);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs, (a.D + CB - 1) / CB, parts);
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cs;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, a);
}
template <typename X, typename G, int M> cudaError_t launch_move(const ScanArgs &a, bool bwd, int sms, cudaStream_t st) {
  constexpr int F = sizeof(X) + sizeof(G) == 4 ? 8 : 4, B = sizeof(X) == 2 ? 4 : 2;  // warps, so that two CTAs' stages fit an SM
  if (bwd) return launch_clustered<B>(scan_bwd_kernel<X, G, M, B>, a, sms, 2 * sizeof(X) + sizeof(G), st);
  return launch_clustered<F>(scan_fwd_kernel<X, G, M, F>, a, sms, sizeof(X) + sizeof(G), st);
}
template <typename X, typename G> cudaError_t launch_types(const ScanArgs &a, int move, bool bwd, int sms, cudaStream_t st) {
  if (move == 16) return launch_move<X, G, M16>(a, bwd, sms, st);
  // two bf16 neighbours in 4 bytes and two fp32 ones in 8: one layout of channels for both
  if constexpr (sizeof(X) == sizeof(G)) {
    if (move == 4) return launch_move<X, G, M4>(a, bwd, sms, st);
  }
  if constexpr (sizeof(X) == 2) return launch_move<X, G, M2>(a, bwd, sms, st);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_scan(const ScanArgs &a, bool bf, bool gate_bf, int move, bool bwd, int sms, cudaStream_t st) {
  if (!bf) return launch_types<float, float>(a, move, bwd, sms, st);
  return gate_bf ? launch_types<bf16, bf16>(a, move, bwd, sms, st) : launch_types<bf16, float>(a, move, bwd, sms, st);
}

cudaError_t launch_scan_step(const ScanArgs &a, bool bf, bool gate_bf, bool vec, cudaStream_t st) {
  const int V = vec ? 4 : 1;
  const dim3 grid((unsigned)((a.D + 256 * V - 1) / (256 * V)), (unsigned)std::min(a.N, 65535), (unsigned)((a.N + 65534) / 65535));
  if (!bf)
    return vec ? launch_pdl(scan_step_kernel<float, float, 4>, grid, dim3(256), 0, st, a)
               : launch_pdl(scan_step_kernel<float, float, 1>, grid, dim3(256), 0, st, a);
  if (gate_bf)
    return vec ? launch_pdl(scan_step_kernel<bf16, bf16, 4>, grid, dim3(256), 0, st, a)
               : launch_pdl(scan_step_kernel<bf16, bf16, 1>, grid, dim3(256), 0, st, a);
  return vec ? launch_pdl(scan_step_kernel<bf16, float, 4>, grid, dim3(256), 0, st, a)
             : launch_pdl(scan_step_kernel<bf16, float, 1>, grid, dim3(256), 0, st, a);
}

}  // namespace gdn
