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

constexpr int SEG = SCAN_SEG, CB = 64, W = 8, NTH = 32 * W, MAXC = 8;  // MAXC: CTAs of a cluster

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
#pragma unroll
    for (int i = 0; i < SEG * PER / 32; ++i) {
      const int p = i * 32 + lane, r = p / PER, c = p % PER * V;
      const bool ok = t0 + r >= lo && t0 + r < hi && c0 + c < D;
      const E *s = ok ? src + (long long)(t0 + r) * row + c0 + c : src;
      if constexpr (M == M16) cp_async16(dst + r * CB + c, s, ok);
      else cp_async4(dst + r * CB + c, s, ok);
    }
  }
}
template <typename E, int M> __device__ __forceinline__ void get2(const E *row, int lane, float (&v)[2]) {
  using L = Lanes<E, M>;
  if constexpr (L::PAIR && sizeof(E) == 2) {
    const uint32_t u = *reinterpret_cast<const uint32_t *>(row + 2 * lane);
    v[0] = __uint_as_float(u << 16);
    v[1] = __uint_as_float(u & 0xffff0000u);
  } else if constexpr (L::PAIR) {
    const float2 u = *reinterpret_cast<const float2 *>(row + 2 * lane);
    v[0] = u.x;
    v[1] = u.y;
  } else {
    v[0] = tof(row[lane]);
    v[1] = tof(row[lane + 32]);
  }
}
// a row of a block, the lane's channels, of which c is the first; only those below D exist
template <typename E, bool PAIR> __device__ __forceinline__ void put2(E *row, int c, int D, const float (&v)[2]) {
  if constexpr (PAIR) {
    if (c < D) st2(row + c, v[0], v[1]);
  } else {
    if (c < D) row[c] = fromf<E>(v[0]);
    if (c + 32 < D) row[c + 32] = fromf<E>(v[1]);
  }
}
template <bool PAIR> __device__ __forceinline__ void take2(const float *row, int c, int D, float (&v)[2]) {
  v[0] = v[1] = 0.f;
  if constexpr (PAIR) {
    if (c < D) {
      const float2 u = *reinterpret_cast<const float2 *>(row + c);
      v[0] = u.x;
      v[1] = u.y;
    }
  } else {
    if (c < D) v[0] = row[c];
    if (c + 32 < D) v[1] = row[c + 32];
  }
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
  __device__ __forceinline__ void apply(float (&c)[2]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) c[k] = A[k] < 0.f ? H[k] : fmaf(A[k], c[k], H[k]);
  }
  __device__ __forceinline__ void then(const Map2 &n) {  // this one first, then n
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      H[k] = n.A[k] < 0.f ? n.H[k] : fmaf(n.A[k], H[k], n.H[k]);
      A[k] = n.A[k] < 0.f || A[k] < 0.f ? -1.f : A[k] * n.A[k];
    }
  }
};
struct Meet {
  float4 warp[2][W][32];     // by round parity: maps of the CTA's segments
  float4 peer[2][MAXC][32];  // of the cluster's CTAs
};
__device__ __forceinline__ Map2 map_of(const float4 &v) { return {{v.x, v.y}, {v.z, v.w}}; }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void store_peer(const float4 *p, int rank, const float4 &v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// A round's exchange: every warp hands in its segment's map and gets the state before it; `carry` becomes the state after
// the round.  `between` runs while the cluster's CTAs meet.
template <typename F>
__device__ __forceinline__ void exchange(Meet &mt, int buf, int cs, int rank, const Map2 &mine, float (&carry)[2], float (&in)[2], F between) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  mt.warp[buf][warp][lane] = make_float4(mine.A[0], mine.A[1], mine.H[0], mine.H[1]);
  __syncthreads();
  if (cs == 1) {
    between();
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if (j == warp) {
        in[0] = carry[0];
        in[1] = carry[1];
      }
      map_of(mt.warp[buf][j][lane]).apply(carry);
    }
    return;
  }
  if (warp == 0) {
    Map2 all = map_of(mt.warp[buf][0][lane]);
#pragma unroll
    for (int j = 1; j < W; ++j) all.then(map_of(mt.warp[buf][j][lane]));
    for (int r = 0; r < cs; ++r) store_peer(&mt.peer[buf][rank][lane], r, make_float4(all.A[0], all.A[1], all.H[0], all.H[1]));
  }
  cluster_arrive();
  between();
  cluster_wait();
  for (int r = 0; r < cs; ++r) {
    if (r == rank) {
      in[0] = carry[0];
      in[1] = carry[1];
    }
    map_of(mt.peer[buf][r][lane]).apply(carry);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    if (j < warp) map_of(mt.warp[buf][j][lane]).apply(in);
}

template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// the state of sequences without tokens passes through: out[n] = in[n], shared out among a channel block's CTAs
template <bool PAIR> __device__ __forceinline__ void pass_empty(const ScanArgs &a, const float *in, float *out, int c, int ctas, int cta) {
  if (!a.cu || !out) return;
  for (int n = cta * W + (threadIdx.x >> 5); n < a.N; n += ctas * W) {
    if (a.cu[n + 1] > a.cu[n]) continue;
    float v[2] = {0.f, 0.f};
    if (in) take2<PAIR>(in + (long long)n * a.D, c, a.D, v);
    put2<float, PAIR>(out + (long long)n * a.D, c, a.D, v);
  }
}

}  // namespace

// grid: CTAs of a cluster, channel blocks, parts
template <typename X, typename G, int M, int STAGES>
__global__ void __launch_bounds__(NTH, 2) scan_fwd_kernel(ScanArgs a) {
  constexpr bool PAIR = Lanes<X, M>::PAIR;
  static_assert(Lanes<X, M>::PAIR == Lanes<G, M>::PAIR || M == M4, "one layout of channels");
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ Meet mt;
  constexpr int BX = SEG * CB * sizeof(X), BG = SEG * CB * sizeof(G);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = gridDim.x, rank = blockIdx.x, c0 = blockIdx.y * CB, c = c0 + Lanes<X, M>::first(lane);
  uint8_t *ring = raw + warp * (STAGES * (BX + BG));
  const X *xs = static_cast<const X *>(a.x);
  const G *gs = static_cast<const G *>(a.g);
  X *ys = static_cast<X *>(a.y);
  if (cs > 1) cluster_arrive();  // peers have begun before anything is written to them
  pdl_trigger();
  pdl_wait();
  const int lo = part_begin(a, blockIdx.z, gridDim.z), hi = part_begin(a, blockIdx.z + 1, gridDim.z);
  const int s0 = lo / SEG, ns = hi > lo ? (hi + SEG - 1) / SEG - s0 : 0, per = cs * W, rounds = (ns + per - 1) / per;
  const int s_mine = s0 + rank * W + warp;  // segment of the first round
  auto load = [&](int k) {
    if (k < rounds) {
      uint8_t *st = ring + k % STAGES * (BX + BG);
      const int t = (s_mine + k * per) * SEG;
      if (t < hi) {
        load_rows<X, M>(reinterpret_cast<X *>(st), xs, a.x_row, t, lo, hi, c0, a.D);
        load_rows<G, M>(reinterpret_cast<G *>(st + BX), gs, a.g_row, t, lo, hi, c0, a.D);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) load(k);
  Bounds bd;
  bd.init(a, s_mine * SEG);
  pass_empty<PAIR>(a, a.h0, a.hT, c, cs * gridDim.z, blockIdx.z * cs + rank);
  if (cs > 1) cluster_wait();
  float carry[2] = {0.f, 0.f};
  for (int k = 0; k < rounds; ++k) {
    const int seg = s_mine + k * per, t0 = seg * SEG;
    const bool live = t0 < hi;
    uint32_t cut = 0;  // boundaries
    if (live) {
      bd.seek(a, t0);
      cut = bd.mask(a, t0);
    }
    cp_wait<STAGES - 2>();
    __syncwarp();
    const X *xr = reinterpret_cast<const X *>(ring + k % STAGES * (BX + BG));
    const G *gr = reinterpret_cast<const G *>(ring + k % STAGES * (BX + BG) + BX);
    float al[SEG][2];
    Map2 m = {{1.f, 1.f}, {0.f, 0.f}};
    auto begins = [&](int i) { return (cut >> i & 1) && t0 + i >= lo && t0 + i < hi; };
    auto ends = [&](int i) { return (cut >> (i + 1) & 1) && t0 + i >= lo && t0 + i < hi; };
    auto start = [&](int i, float (&h)[2]) {
      h[0] = h[1] = 0.f;
      if (a.h0) take2<PAIR>(a.h0 + (long long)bd.seq(a, t0 + i) * a.D, c, a.D, h);
    };
    if (live) {
      float sum[2] = {0.f, 0.f};
      bool fresh = false;
#pragma unroll
      for (int i = 0; i < SEG; ++i) {
        float x[2], g[2];
        get2<X, M>(xr + i * CB, lane, x);
        get2<G, M>(gr + i * CB, lane, g);
        if (cut && begins(i)) {
          start(i, m.H);
          fresh = true;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          al[i][e] = expf(g[e]);
          sum[e] += g[e];
          m.H[e] = fmaf(al[i][e], m.H[e], x[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) m.A[e] = fresh ? -1.f : expf(sum[e]);
    }
    float h[2];
    exchange(mt, k & 1, cs, rank, m, carry, h, [&] { load(k + STAGES - 1); });
    if (!live) continue;
    if (a.states && t0 >= lo) put2<float, PAIR>(a.states + (long long)seg * a.D, c, a.D, h);
    X *yr = ys + (long long)t0 * a.y_row;
#pragma unroll
    for (int i = 0; i < SEG; ++i) {
      float x[2];
      get2<X, M>(xr + i * CB, lane, x);
      if (cut && begins(i)) start(i, h);
#pragma unroll
      for (int e = 0; e < 2; ++e) h[e] = fmaf(al[i][e], h[e], x[e]);
      if (t0 + i >= lo && t0 + i < hi) put2<X, PAIR>(yr + i * a.y_row, c, a.D, h);
      if (cut && ends(i) && a.hT) put2<float, PAIR>(a.hT + (long long)bd.seq(a, t0 + i) * a.D, c, a.D, h);
    }
    __syncwarp();  // the stage is loaded again in the next round
  }
  cp_async_wait_all();
}

// The same walk from the line's end; in a part, segment 0 of the walk is the last one.
template <typename X, typename G, int M, int STAGES>
__global__ void __launch_bounds__(NTH, 2) scan_bwd_kernel(ScanArgs a) {
  constexpr bool PAIR = Lanes<X, M>::PAIR;
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ Meet mt;
  constexpr int BX = SEG * CB * sizeof(X), BG = SEG * CB * sizeof(G), ST = 2 * BX + BG;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = gridDim.x, rank = blockIdx.x, c0 = blockIdx.y * CB, c = c0 + Lanes<X, M>::first(lane);
  uint8_t *ring = raw + warp * (STAGES * ST);
  const X *xs = static_cast<const X *>(a.x), *dys = static_cast<const X *>(a.dy);
  const G *gs = static_cast<const G *>(a.g);
  X *dxs = static_cast<X *>(a.y);
  G *dgs = static_cast<G *>(a.dg);
  if (cs > 1) cluster_arrive();
  pdl_trigger();
  pdl_wait();
  const int lo = part_begin(a, blockIdx.z, gridDim.z), hi = part_begin(a, blockIdx.z + 1, gridDim.z);
  const int s0 = lo / SEG, ns = hi > lo ? (hi + SEG - 1) / SEG - s0 : 0, per = cs * W, rounds = (ns + per - 1) / per;
  const int s_mine = s0 + ns - 1 - (rank * W + warp);
  auto load = [&](int k) {
    if (k < rounds) {
      uint8_t *st = ring + k % STAGES * ST;
      const int seg = s_mine - k * per;
      if (seg >= s0) {
        load_rows<X, M>(reinterpret_cast<X *>(st), xs, a.x_row, seg * SEG, lo, hi, c0, a.D);
        load_rows<X, M>(reinterpret_cast<X *>(st + BX), dys, a.dy_row, seg * SEG, lo, hi, c0, a.D);
        load_rows<G, M>(reinterpret_cast<G *>(st + 2 * BX), gs, a.g_row, seg * SEG, lo, hi, c0, a.D);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) load(k);
  Bounds bd;
  bd.init(a, max(s_mine, s0) * SEG);
  pass_empty<PAIR>(a, a.dhT, a.dh0, c, cs * gridDim.z, blockIdx.z * cs + rank);
  if (cs > 1) cluster_wait();
  float carry[2] = {0.f, 0.f};
  for (int k = 0; k < rounds; ++k) {
    const int seg = s_mine - k * per, t0 = seg * SEG;
    const bool live = seg >= s0;
    uint32_t cut = 0;
    float h[2] = {0.f, 0.f};
    if (live) {
      take2<PAIR>(a.states + (long long)seg * a.D, c, a.D, h);
      bd.seek(a, t0);
      cut = bd.mask(a, t0);
    }
    cp_wait<STAGES - 2>();
    __syncwarp();
    const X *xr = reinterpret_cast<const X *>(ring + k % STAGES * ST), *dyr = xr + SEG * CB;
    const G *gr = reinterpret_cast<const G *>(ring + k % STAGES * ST + 2 * BX);
    float al[SEG][2], hp[SEG][2];  // gates, and states before the tokens
    Map2 m = {{1.f, 1.f}, {0.f, 0.f}};
    auto begins = [&](int i) { return (cut >> i & 1) && t0 + i >= lo && t0 + i < hi; };
    auto ends = [&](int i) { return (cut >> (i + 1) & 1) && t0 + i >= lo && t0 + i < hi; };
    auto at_end = [&](int i, float (&d)[2]) {
      d[0] = d[1] = 0.f;
      if (a.dhT) take2<PAIR>(a.dhT + (long long)bd.seq(a, t0 + i) * a.D, c, a.D, d);
    };
    if (live) {
      float sum[2] = {0.f, 0.f};
      bool fresh = false;
#pragma unroll
      for (int i = 0; i < SEG; ++i) {
        float x[2], g[2];
        get2<X, M>(xr + i * CB, lane, x);
        get2<G, M>(gr + i * CB, lane, g);
        if (cut && begins(i)) {
          h[0] = h[1] = 0.f;
          if (a.h0) take2<PAIR>(a.h0 + (long long)bd.seq(a, t0 + i) * a.D, c, a.D, h);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          hp[i][e] = h[e];
          al[i][e] = expf(g[e]);
          sum[e] += g[e];
          h[e] = fmaf(al[i][e], h[e], x[e]);
        }
      }
#pragma unroll
      for (int i = SEG - 1; i >= 0; --i) {
        float dy[2];
        get2<X, M>(dyr + i * CB, lane, dy);
        if (cut && ends(i)) {
          at_end(i, m.H);
          fresh = true;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) m.H[e] = al[i][e] * (dy[e] + m.H[e]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) m.A[e] = fresh ? -1.f : expf(sum[e]);
    }
    float d[2];  // what reaches the state from later tokens
    exchange(mt, k & 1, cs, rank, m, carry, d, [&] { load(k + STAGES - 1); });
    if (!live) continue;
#pragma unroll
    for (int i = SEG - 1; i >= 0; --i) {
      float dy[2], dg[2];
      get2<X, M>(dyr + i * CB, lane, dy);
      if (cut && ends(i)) at_end(i, d);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        dy[e] += d[e];
        d[e] = al[i][e] * dy[e];
        dg[e] = d[e] * hp[i][e];
      }
      if (t0 + i >= lo && t0 + i < hi) {
        put2<X, PAIR>(dxs + (long long)(t0 + i) * a.y_row, c, a.D, dy);
        put2<G, PAIR>(dgs + (long long)(t0 + i) * a.dg_row, c, a.D, dg);
      }
      if (cut && begins(i) && a.dh0) put2<float, PAIR>(a.dh0 + (long long)bd.seq(a, t0 + i) * a.D, c, a.D, d);
    }
    __syncwarp();
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

// The split of a call: parts of whole sequences and CTAs of a cluster, for about two CTAs per SM.  Equal sequences go to
// parts first, which exchange nothing; packed ones may be one long sequence and many short ones, so there the line is cut
// within a cluster first.
void split(const ScanArgs &a, int sms, int &parts, int &cs) {
  const int nb = (a.D + CB - 1) / CB, want = std::max(1, 2 * sms / nb);  // CTAs of a channel block
  const auto clustered = [&](int most, long long tokens) {
    int c = 1;
    while (c < MAXC && 2 * c <= most && tokens > (long long)c * W * SEG) c *= 2;
    return c;
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

template <typename... KArgs>
cudaError_t launch_clustered(void (*k)(KArgs...), const ScanArgs &a, int sms, size_t smem, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  int parts, cs;
  split(a, sms, parts, cs);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs, (a.D + CB - 1) / CB, parts);
  cfg.blockDim = dim3(NTH);
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
  constexpr int F = sizeof(X) + sizeof(G) == 4 ? 3 : 2, B = 2;  // stages
  constexpr size_t row = (size_t)W * SEG * CB;
  if (bwd) return launch_clustered(scan_bwd_kernel<X, G, M, B>, a, sms, row * B * (2 * sizeof(X) + sizeof(G)), st);
  return launch_clustered(scan_fwd_kernel<X, G, M, F>, a, sms, row * F * (sizeof(X) + sizeof(G)), st);
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
