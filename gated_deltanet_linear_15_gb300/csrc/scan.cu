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

constexpr int SEG = SCAN_SEG, MAXC = 8;  // MAXC: CTAs of a cluster

// what moves rows: 16-byte pieces, 4-byte pieces, or single bf16 elements
enum Move { M16, M4, M2 };
// A lane holds NP pairs of a block's 64 NP channels: neighbours, or pairs 64 apart, or single channels 32 apart, as accesses allow.
enum Lay { NEXT, PAIRS, SINGLE };
template <typename X, int M> constexpr int LAY = M == M16 ? NEXT : (M == M4 && sizeof(X) == 2 ? PAIRS : SINGLE);
template <int L, int NP> __device__ __forceinline__ int first_channel(int lane) {
  return L == NEXT ? 2 * NP * lane : (L == PAIRS ? 2 * lane : lane);
}

// a lane's values
template <int NP> struct Vals {
  uint64_t v[NP];
  __device__ __forceinline__ float2 pair(int i) const {
    float2 f;
    upk(v[i], f.x, f.y);
    return f;
  }
};
template <int NP> __device__ __forceinline__ Vals<NP> operator+(Vals<NP> a, const Vals<NP> &b) {
#pragma unroll
  for (int i = 0; i < NP; ++i) a.v[i] = add2(a.v[i], b.v[i]);
  return a;
}
template <int NP> __device__ __forceinline__ Vals<NP> operator*(Vals<NP> a, const Vals<NP> &b) {
#pragma unroll
  for (int i = 0; i < NP; ++i) a.v[i] = mul2(a.v[i], b.v[i]);
  return a;
}
template <int NP> __device__ __forceinline__ Vals<NP> fma(Vals<NP> a, const Vals<NP> &b, const Vals<NP> &c) {
#pragma unroll
  for (int i = 0; i < NP; ++i) a.v[i] = fma2(a.v[i], b.v[i], c.v[i]);
  return a;
}
__device__ __forceinline__ uint64_t wide(uint32_t u) { return pk(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }

// Rows of segments on their way to shared memory, [SEG][CB]: zeros outside [lo, hi) x [0, D).  The lane's place in the row and the
// first of its rows stay the same; `at` moves with the segments.
template <typename E, int M, int CB> struct Loader {
  static constexpr int B = M == M16 ? 16 : (M == M4 ? 4 : 2), V = B / (int)sizeof(E) > 0 ? B / (int)sizeof(E) : 1;
  static constexpr int PER = CB / V, RPI = PER < 32 ? 32 / PER : 1, CPI = PER < 32 ? PER : 32;  // pieces of a row; rows, pieces of an instruction
  const E *src, *at;  // at: of the segment asked for next, the lane's first row
  long long row, step;
  // s: the first segment; per: how far the next one lies
  __device__ __forceinline__ void init(const void *p, long long stride, int c0, long long s, long long per) {
    const int lane = threadIdx.x & 31;
    src = static_cast<const E *>(p);
    row = stride;
    at = src + (s * SEG + lane / CPI) * row + c0 + lane % CPI * V;
    step = per * SEG * row;
  }
  __device__ __forceinline__ void load(E *dst, int t0, int lo, int hi, int c0, int D) {
    const int lane = threadIdx.x & 31, r0 = lane / CPI, c = lane % CPI * V;
    const bool inside = t0 >= lo && t0 + SEG <= hi;
    E *d = dst + r0 * CB + c;
#pragma unroll
    for (int k = 0; k < PER / CPI; ++k) {
      const E *s = at + 32 * k * V;
      const bool there = c0 + c + 32 * k * V < D;
      if constexpr (M == M2) {
#pragma unroll 4
        for (int i = 0; i < SEG; ++i, s += row) {
          E v = fromf<E>(0.f);
          if (there && t0 + i >= lo && t0 + i < hi) v = *s;
          d[i * CB + 32 * k] = v;
        }
      } else {
        auto copy = [](E *d, const E *s, bool ok) {
          if constexpr (M == M16) cp_async16(d, s, ok);
          else cp_async4(d, s, ok);
        };
        if (inside) {
          if (there) {  // what is past D is never looked at
#pragma unroll
            for (int i = 0; i < SEG / RPI; ++i, s += RPI * row) copy(d + i * RPI * CB + 32 * k * V, s, true);
          }
        } else {
          const unsigned span = there ? hi - lo : 0, rel = t0 + r0 - lo;
#pragma unroll 1
          for (int i = 0; i < SEG / RPI; ++i, s += RPI * row) {
            const bool ok = rel + i * RPI < span;
            copy(d + i * RPI * CB + 32 * k * V, ok ? s : src, ok);
          }
        }
      }
    }
    at += step;
  }
};
// the lane's values of a row in shared memory
template <typename E, int L, int NP> __device__ __forceinline__ Vals<NP> get(const E *row, int lane) {
  Vals<NP> x;
  if constexpr (L == NEXT && 2 * NP * sizeof(E) == 8) {
    const uint64_t u = *reinterpret_cast<const uint64_t *>(row + 2 * NP * lane);
    if constexpr (NP == 1) {
      x.v[0] = u;
    } else {
      x.v[0] = wide((uint32_t)u);
      x.v[NP - 1] = wide((uint32_t)(u >> 32));
    }
  } else if constexpr (L == SINGLE) {
#pragma unroll
    for (int i = 0; i < NP; ++i) x.v[i] = pk(tof(row[lane + 64 * i]), tof(row[lane + 64 * i + 32]));
  } else {
    static_assert(sizeof(E) == 2 && (L == PAIRS || NP == 1), "pairs of bf16");
#pragma unroll
    for (int i = 0; i < NP; ++i) x.v[i] = wide(*reinterpret_cast<const uint32_t *>(row + 2 * lane + 64 * i));
  }
  return x;
}
// Gates of a row.  With bf16 rows the product with log2(e) and ex2.approx, off by 2^-22 of themselves, which a bf16 result does
// not show and which the state carries for 16 tokens at most (its map takes expf of the sum); expf in fp32, where 16 such
// errors would be half of all.
template <bool EXACT> __device__ __forceinline__ uint64_t gates2(uint64_t g) {
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
template <bool EXACT, int NP> __device__ __forceinline__ Vals<NP> gates(Vals<NP> g) {
#pragma unroll
  for (int i = 0; i < NP; ++i) g.v[i] = gates2<EXACT>(g.v[i]);
  return g;
}

// a row in global memory: the lane's channels, of which c is the first; only those below D exist
template <typename E, int L, int NP> __device__ __forceinline__ void put(E *row, int c, int D, const Vals<NP> &x) {
  row += c;
  if constexpr (L == NEXT && NP == 2) {
    if (c >= D) return;
    const float2 f = x.pair(0), g = x.pair(1);
    if constexpr (sizeof(E) == 2) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y), q = __floats2bfloat162_rn(g.x, g.y);
      *reinterpret_cast<uint2 *>(row) = make_uint2(*reinterpret_cast<const uint32_t *>(&p), *reinterpret_cast<const uint32_t *>(&q));
    } else {
      *reinterpret_cast<float4 *>(row) = make_float4(f.x, f.y, g.x, g.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float2 f = x.pair(i);
      if constexpr (L == SINGLE) {
        if (c + 64 * i < D) row[64 * i] = fromf<E>(f.x);
        if (c + 64 * i + 32 < D) row[64 * i + 32] = fromf<E>(f.y);
      } else if (c + 64 * i < D) {
        st2(row + 64 * i, f.x, f.y);
      }
    }
  }
}
template <int L, int NP> __device__ __forceinline__ Vals<NP> take(const float *row, int c, int D) {
  Vals<NP> x = {};
  row += c;
  if constexpr (L == NEXT && NP == 2) {
    if (c < D) {
      const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(row);
      x.v[0] = u.x;
      x.v[1] = u.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if constexpr (L == SINGLE) x.v[i] = pk(c + 64 * i < D ? row[64 * i] : 0.f, c + 64 * i + 32 < D ? row[64 * i + 32] : 0.f);
      else if (c + 64 * i < D) x.v[i] = *reinterpret_cast<const uint64_t *>(row + 64 * i);
    }
  }
  return x;
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

// The boundaries between sequences around a warp's segment.  The warp knows the sequence [b0, b1) that its last segment
// began in; most segments lie inside it, and nothing is looked up for them.  With cu, each lane holds one entry of a window
// that begins at entry `base`; it moves with the segments.
struct Bounds {
  int b0, b1;
  int base, e;
  int left;  // windows that may still be looked at: a cu that is not sorted ends the walk, not the kernel
  __device__ __forceinline__ void load(const ScanArgs &a) {
    const int i = base + (threadIdx.x & 31);
    e = i <= a.N ? a.cu[i] : 0x7fffffff;
  }
  __device__ __forceinline__ void init(const ScanArgs &a, int t) {
    b0 = b1 = base = e = 0;
    left = a.N / 8 + 64;
    if (!a.cu) return;
    base = max(lower_bound(a.cu, a.N + 1, t + 1) - 1, 0);
    load(a);
  }
  // bit i (of 17): some sequence begins, or the last one ends, at token t + i.  Moves the window to t: its first entry is
  // the last one at or before t, or near it.
  __device__ __forceinline__ uint32_t mask(const ScanArgs &a, int t) {
    if (t > b0 && t + SEG < b1) return 0;
    const int lane = threadIdx.x & 31;
    if (!a.cu) {
      b0 = (int)((unsigned)t / (unsigned)a.T) * a.T;
      b1 = b0 + a.T;
      return __ballot_sync(0xffffffffu, lane <= SEG && (unsigned)(t + lane - b0) % (unsigned)a.T == 0);
    }
    for (; left > 0; --left) {
      const unsigned at = __ballot_sync(0xffffffffu, e <= t);
      if (at == 0xffffffffu && base + 31 <= a.N) base += 31;
      else if (!(at & 1) && base > 0) base = max(base - 31, 0);
      else break;
      load(a);
    }
    b0 = __reduce_max_sync(0xffffffffu, e <= t ? e : -1);
    b1 = __reduce_min_sync(0xffffffffu, e > t ? e : 0x7fffffff);
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
template <int NP> struct Map {
  float A[2 * NP], H[2 * NP];
  __device__ __forceinline__ void of(float (&c)[2 * NP]) const {
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) c[i] = A[i] < 0.f ? H[i] : fmaf(A[i], c[i], H[i]);
  }
  __device__ __forceinline__ void then(const Map &n) {  // this one first, then n
    n.of(H);
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) A[i] = n.A[i] < 0.f || A[i] < 0.f ? -1.f : A[i] * n.A[i];
  }
};
// of a segment: the sum of its log-gates and its result from zero
template <int NP> __device__ __forceinline__ Map<NP> segment_map(bool fresh, const Vals<NP> &sum, const Vals<NP> &h) {
  Map<NP> m;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const float2 s = sum.pair(i), z = h.pair(i);
    m.A[2 * i] = fresh ? -1.f : expf(s.x);
    m.A[2 * i + 1] = fresh ? -1.f : expf(s.y);
    m.H[2 * i] = z.x;
    m.H[2 * i + 1] = z.y;
  }
  return m;
}
// a map in shared memory: 16-byte pieces of every lane
template <int NP> struct MapSlot {
  float4 p[NP][32];
};
template <int NP> __device__ __forceinline__ float4 piece_of(const Map<NP> &m, int i) {
  return make_float4(m.A[2 * i], m.A[2 * i + 1], m.H[2 * i], m.H[2 * i + 1]);
}
template <int NP> __device__ __forceinline__ Map<NP> map_at(const MapSlot<NP> &s) {
  Map<NP> m;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const float4 v = s.p[i][threadIdx.x & 31];
    m.A[2 * i] = v.x;
    m.A[2 * i + 1] = v.y;
    m.H[2 * i] = v.z;
    m.H[2 * i + 1] = v.w;
  }
  return m;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, int rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"(addr), "r"(rank));
  return at;
}
// 16 bytes into a peer's shared memory, counted by its mbarrier
__device__ __forceinline__ void store_peer(uint32_t at, uint32_t bar, const float4 &v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];\n" ::"r"(at), "f"(v.x),
               "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
// The peers of a cluster run at the same time, so the wait ends; one that did not within about a second gives up.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  for (uint32_t it = 0; it < (1u << 18); ++it) {
    uint32_t done;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
  }
  return false;
}

// A round's exchange: every warp hands in its segment's map, and later gets the state before it; `carry` becomes the state
// after the round.  The CTA's maps meet behind a barrier; every warp joins them and sends the result to some of the cluster's
// CTAs, where an mbarrier counts its bytes.  (A cluster barrier instead makes the warp that releases its maps by it wait
// for its own global stores too.)  Two sets of maps by the round's parity: a CTA sends round r + 2
// only when it has everyone's maps of round r + 1, which come after their reading of round r.
template <int W, int NP> struct Meet {
  typedef MapSlot<NP> Slot;
  Slot *warp, *peer;  // [2][W], [2][cs]
  uint64_t *bar;      // [2]
  int cs, rank;
  __device__ __forceinline__ void init(uint8_t *smem, uint64_t *bars) {
    warp = reinterpret_cast<Slot *>(smem);
    peer = warp + 2 * W;
    bar = bars;
    cs = gridDim.x;
    rank = blockIdx.x;
    if (cs == 1) return;
    if (threadIdx.x < 2) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(smem_u32(bar + threadIdx.x)) : "memory");
      asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    __syncwarp();
    cluster_arrive();  // peers have begun, and their barriers are there, before anything is sent to them
  }
  __device__ __forceinline__ void ready() const {
    if (cs > 1) cluster_wait();
  }
  __device__ __forceinline__ void hand_in(int round, const Map<NP> &mine) const {
    const int me = threadIdx.x >> 5, lane = threadIdx.x & 31, par = round & 1;
    Slot *mw = warp + par * W;
#pragma unroll
    for (int i = 0; i < NP; ++i) mw[me].p[i][lane] = piece_of(mine, i);
    __syncthreads();
    if (cs == 1) return;
    if (threadIdx.x == 0) bar_expect(smem_u32(bar + par), cs * sizeof(Slot));
    if (me >= cs) return;
    Map<NP> all = map_at(mw[0]);
#pragma unroll
    for (int j = 1; j < W; ++j) all.then(map_at(mw[j]));
    const uint32_t at = smem_u32(&peer[par * cs + rank].p[0][lane]), b = smem_u32(bar + par);
#pragma unroll 1
    for (int r = me; r < cs; r += W) {
      const uint32_t ra = peer_addr(at, r), rb = peer_addr(b, r);
#pragma unroll
      for (int i = 0; i < NP; ++i) store_peer(ra + 512 * i, rb, piece_of(all, i));
    }
  }
  __device__ __forceinline__ Vals<NP> state(int round, float (&carry)[2 * NP]) const {
    const int me = threadIdx.x >> 5, par = round & 1;
    const Slot *mw = warp + par * W, *mp = peer + par * cs;
    float in[2 * NP];
    auto keep = [&] {
#pragma unroll
      for (int i = 0; i < 2 * NP; ++i) in[i] = carry[i];
    };
    keep();
    if (cs == 1) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if (j == me) keep();
        map_at(mw[j]).of(carry);
      }
    } else {
      if (!bar_wait(smem_u32(bar + par), round >> 1 & 1)) {
#pragma unroll
        for (int i = 0; i < 2 * NP; ++i) carry[i] = __uint_as_float(0x7fffffffu);  // what follows is not reliable, and shows it
      }
#pragma unroll
      for (int b = 0; b < MAXC; b += 4) {
        if (b >= cs) break;
        Map<NP> m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = map_at(mp[min(b + j, cs - 1)]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (b + j < cs) {
            if (b + j == rank) keep();
            m[j].of(carry);
          }
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        if (j < me) map_at(mw[j]).of(in);
    }
    Vals<NP> h;
#pragma unroll
    for (int i = 0; i < NP; ++i) h.v[i] = pk(in[2 * i], in[2 * i + 1]);
    return h;
  }
};

template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// the state of sequences without tokens passes through: out[n] = in[n], shared out among a channel block's CTAs
template <int L, int NP, int W>
__device__ __forceinline__ void pass_empty(const ScanArgs &a, const float *in, float *out, int c, int ctas, int cta) {
  if (!a.cu || !out) return;
  for (int n = cta * W + (threadIdx.x >> 5); n < a.N; n += ctas * W) {
    if (a.cu[n + 1] > a.cu[n]) continue;
    put<float, L>(out + (long long)n * a.D, c, a.D, in ? take<L, NP>(in + (long long)n * a.D, c, a.D) : Vals<NP>{});
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
    cut = live ? bd.mask(a, t0) : 0;
    plain = cut == 0 && t0 >= w.lo && t0 + SEG <= w.hi;
  }
  __device__ __forceinline__ bool inside(const Walk &w, int i) const { return t0 + i >= w.lo && t0 + i < w.hi; }
  __device__ __forceinline__ bool begins(int i) const { return cut >> i & 1; }
  __device__ __forceinline__ bool ends(int i) const { return cut >> (i + 1) & 1; }
};

}  // namespace

// grid: CTAs of a cluster, channel blocks, parts.  Each step hands in the maps of round k + 1 and, while the CTAs of the cluster
// meet, finishes round k, whose states are known; the stages of round k + 2 are on their way.
template <typename X, typename G, int M, int W, int NP>
__global__ void __launch_bounds__(32 * W, 2) scan_fwd_kernel(ScanArgs a) {
  constexpr int L = LAY<X, M>, CB = 64 * NP;
  typedef Vals<NP> V;
  constexpr bool EXACT = sizeof(X) == 4;
  static_assert(L == LAY<G, M>, "one layout of channels");
  extern __shared__ __align__(16) uint8_t raw[];
  constexpr int BX = SEG * CB * sizeof(X), ST = BX + SEG * CB * sizeof(G);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = gridDim.x, rank = blockIdx.x, c0 = blockIdx.y * CB, c = c0 + first_channel<L, NP>(lane);
  uint8_t *ring = raw + warp * (3 * ST);
  __shared__ uint64_t bars[2];
  Meet<W, NP> mt;
  mt.init(raw + W * 3 * ST, bars);
  pdl_trigger();
  pdl_wait();
  Walk w = {};
  w.init<W>(a, cs, rank);
  Loader<X, M, CB> lx;
  Loader<G, M, CB> lg;
  lx.init(a.x, a.x_row, c0, w.up(0), w.per);
  lg.init(a.g, a.g_row, c0, w.up(0), w.per);
  auto load = [&](int k, int slot) {
    if (k < w.rounds && w.has(w.up(k))) {
      uint8_t *st = ring + slot * ST;
      const int t0 = w.up(k) * SEG;
      lx.load(reinterpret_cast<X *>(st), t0, w.lo, w.hi, c0, a.D);
      lg.load(reinterpret_cast<G *>(st + BX), t0, w.lo, w.hi, c0, a.D);
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int k = 0; k < 2; ++k) load(k, k);
  Piece now = {}, next = {};
  next.bd.init(a, w.up(0) * SEG);
  pass_empty<L, NP, W>(a, a.h0, a.hT, c, cs * gridDim.z, blockIdx.z * cs + rank);
  mt.ready();
  auto x_of = [&](const uint8_t *st, int i) { return get<X, L, NP>(reinterpret_cast<const X *>(st) + i * CB, lane); };
  auto g_of = [&](const uint8_t *st, int i) { return get<G, L, NP>(reinterpret_cast<const G *>(st + BX) + i * CB, lane); };
  auto start = [&](const Piece &p, int i) { return a.h0 ? take<L, NP>(a.h0 + (long long)p.bd.seq(a, p.t0 + i) * a.D, c, a.D) : V{}; };
  float carry[2 * NP] = {};
  V h = {};
  int slot = 2;  // of round k
#pragma unroll 1
  for (int k = -1; k < w.rounds; ++k) {
    const int slot1 = slot == 2 ? 0 : slot + 1;
    const bool more = k + 1 < w.rounds;
    if (more) {
      next.look(a, w, w.up(k + 1));
      cp_wait<1>();
      __syncwarp();
      const uint8_t *st = ring + slot1 * ST;
      V sum = {}, z = {};
      bool fresh = false;
      if (next.plain) {
#pragma unroll
        for (int i = 0; i < SEG; ++i) {
          const V g = g_of(st, i);
          sum = sum + g;
          z = fma(gates<EXACT>(g), z, x_of(st, i));
        }
      } else if (next.live) {
#pragma unroll 1
        for (int i = 0; i < SEG; ++i) {
          const V g = g_of(st, i);
          if (next.begins(i) && next.inside(w, i)) {
            z = start(next, i);
            fresh = true;
          }
          sum = sum + g;
          z = fma(gates<EXACT>(g), z, x_of(st, i));
        }
      }
      mt.hand_in(k + 1, segment_map(fresh, sum, z));
    }
    if (k >= 0 && now.live) {
      const uint8_t *st = ring + slot * ST;
      if (a.states && now.t0 >= w.lo) put<float, L>(a.states + (long long)now.seg * a.D, c, a.D, h);
      X *yr = static_cast<X *>(a.y) + (long long)now.t0 * a.y_row;
      if (now.plain) {
#pragma unroll
        for (int i = 0; i < SEG; ++i, yr += a.y_row) {
          h = fma(gates<EXACT>(g_of(st, i)), h, x_of(st, i));
          put<X, L>(yr, c, a.D, h);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < SEG; ++i, yr += a.y_row) {
          if (!now.inside(w, i)) continue;
          if (now.begins(i)) h = start(now, i);
          h = fma(gates<EXACT>(g_of(st, i)), h, x_of(st, i));
          put<X, L>(yr, c, a.D, h);
          if (now.ends(i) && a.hT) put<float, L>(a.hT + (long long)now.bd.seq(a, now.t0 + i) * a.D, c, a.D, h);
        }
      }
    }
    __syncwarp();  // the stage is loaded again
    load(k + 3, slot);
    if (more) {
      h = mt.state(k + 1, carry);
      now = next;
    }
    slot = slot1;
  }
  cp_async_wait_all();
}

// The same walk from the part's end, a round at a time: with more CTAs to an SM instead of a round ahead it is faster (4 x 4096
// tokens of 2048 channels 80 us instead of 89), since the states before all tokens of a segment take the registers that the
// round ahead needs.  Two stages of dy and g; x is needed after the exchange only, and has one.  LIMIT: CTAs per SM.
template <typename X, typename G, int M, int W, int NP, int LIMIT>
__global__ void __launch_bounds__(32 * W, LIMIT) scan_bwd_kernel(ScanArgs a) {
  constexpr int L = LAY<X, M>, CB = 64 * NP;
  typedef Vals<NP> V;
  constexpr bool EXACT = sizeof(X) == 4;
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ uint64_t bars[2];
  constexpr int BX = SEG * CB * sizeof(X), ST = BX + SEG * CB * sizeof(G);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = gridDim.x, rank = blockIdx.x, c0 = blockIdx.y * CB, c = c0 + first_channel<L, NP>(lane);
  uint8_t *ring = raw + warp * (2 * ST + BX);
  X *sx = reinterpret_cast<X *>(ring + 2 * ST);
  Meet<W, NP> mt;
  mt.init(raw + W * (2 * ST + BX), bars);
  pdl_trigger();
  pdl_wait();
  Walk w = {};
  w.init<W>(a, cs, rank);
  Loader<X, M, CB> lx, ld;
  Loader<G, M, CB> lg;
  lx.init(a.x, a.x_row, c0, w.down(0), -w.per);
  ld.init(a.dy, a.dy_row, c0, w.down(0), -w.per);
  lg.init(a.g, a.g_row, c0, w.down(0), -w.per);
  auto load = [&](int k) {  // dy and g of round k
    if (k < w.rounds && w.has(w.down(k))) {
      uint8_t *st = ring + (k & 1) * ST;
      const int t0 = w.down(k) * SEG;
      ld.load(reinterpret_cast<X *>(st), t0, w.lo, w.hi, c0, a.D);
      lg.load(reinterpret_cast<G *>(st + BX), t0, w.lo, w.hi, c0, a.D);
    }
    cp_async_commit();
  };
  load(0);
  Piece now = {};
  now.bd.init(a, max(w.down(0) * SEG, 0));
  pass_empty<L, NP, W>(a, a.dhT, a.dh0, c, cs * gridDim.z, blockIdx.z * cs + rank);
  mt.ready();
  const uint8_t *st = ring;
  auto x_of = [&](int i) { return get<X, L, NP>(sx + i * CB, lane); };
  auto dy_of = [&](int i) { return get<X, L, NP>(reinterpret_cast<const X *>(st) + i * CB, lane); };
  auto g_of = [&](int i) { return get<G, L, NP>(reinterpret_cast<const G *>(st + BX) + i * CB, lane); };
  auto start = [&](int i) { return a.h0 ? take<L, NP>(a.h0 + (long long)now.bd.seq(a, now.t0 + i) * a.D, c, a.D) : V{}; };
  auto at_end = [&](int i) { return a.dhT ? take<L, NP>(a.dhT + (long long)now.bd.seq(a, now.t0 + i) * a.D, c, a.D) : V{}; };
  float carry[2 * NP] = {};
#pragma unroll 1
  for (int k = 0; k < w.rounds; ++k) {
    st = ring + (k & 1) * ST;
    now.look(a, w, w.down(k));
    if (now.live) lx.load(sx, now.t0, w.lo, w.hi, c0, a.D);
    cp_async_commit();
    load(k + 1);
    V h = now.live ? take<L, NP>(a.states + (long long)now.seg * a.D, c, a.D) : V{};
    cp_wait<2>();
    __syncwarp();
    V sum = {}, d = {};  // d: what reaches the state from later tokens
    bool fresh = false;
    if (now.plain) {
#pragma unroll
      for (int i = SEG - 1; i >= 0; --i) {
        const V g = g_of(i);
        sum = sum + g;
        d = gates<EXACT>(g) * (dy_of(i) + d);
      }
    } else if (now.live) {
#pragma unroll 1
      for (int i = SEG - 1; i >= 0; --i) {
        const V g = g_of(i);
        if (now.ends(i) && now.inside(w, i)) {
          d = at_end(i);
          fresh = true;
        }
        sum = sum + g;
        d = gates<EXACT>(g) * (dy_of(i) + d);
      }
    }
    mt.hand_in(k, segment_map(fresh, sum, d));
    cp_wait<1>();
    __syncwarp();
    X *dxr = static_cast<X *>(a.y) + (long long)(now.t0 + SEG - 1) * a.y_row;
    G *dgr = static_cast<G *>(a.dg) + (long long)(now.t0 + SEG - 1) * a.dg_row;
    if (now.plain) {
      V hp[SEG];  // states before the tokens
#pragma unroll
      for (int i = 0; i < SEG; ++i) {
        hp[i] = h;
        h = fma(gates<EXACT>(g_of(i)), h, x_of(i));
      }
      d = mt.state(k, carry);
#pragma unroll
      for (int i = SEG - 1; i >= 0; --i, dxr -= a.y_row, dgr -= a.dg_row) {
        const V dx = dy_of(i) + d;
        d = gates<EXACT>(g_of(i)) * dx;
        put<X, L>(dxr, c, a.D, dx);
        put<G, L>(dgr, c, a.D, d * hp[i]);
      }
    } else {
      d = mt.state(k, carry);
      if (now.live) {
        V hp[SEG];  // in local memory
#pragma unroll 1
        for (int i = 0; i < SEG; ++i) {
          if (now.begins(i) && now.inside(w, i)) h = start(i);
          hp[i] = h;
          h = fma(gates<EXACT>(g_of(i)), h, x_of(i));
        }
#pragma unroll 1
        for (int i = SEG - 1; i >= 0; --i, dxr -= a.y_row, dgr -= a.dg_row) {
          if (!now.inside(w, i)) continue;
          if (now.ends(i)) d = at_end(i);
          const V dx = dy_of(i) + d;
          d = gates<EXACT>(g_of(i)) * dx;
          put<X, L>(dxr, c, a.D, dx);
          put<G, L>(dgr, c, a.D, d * hp[i]);
          if (now.begins(i) && a.dh0) put<float, L>(a.dh0 + (long long)now.bd.seq(a, now.t0 + i) * a.D, c, a.D, d);
        }
      }
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

// The split of a call: parts of whole sequences and CTAs of a cluster, for `ctas` of them.  Equal sequences go to
// parts first, which exchange nothing; packed ones may be one long sequence and many short ones, so there the line is cut
// within a cluster first.
void split(const ScanArgs &a, int W, int CB, int ctas, int &parts, int &cs) {
  const int nb = (a.D + CB - 1) / CB, want = std::max(1, ctas / nb);  // CTAs of a channel block
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

// ring: bytes of a warp's stages
template <int W, int NP, typename... KArgs>
cudaError_t launch_clustered(void (*k)(KArgs...), const ScanArgs &a, int ctas, int ring, cudaStream_t st) {
  constexpr int SLOT = sizeof(MapSlot<NP>);
  int parts, cs;
  split(a, W, 64 * NP, ctas, parts, cs);
  const int smem = W * ring + 2 * (W + (cs > 1 ? cs : 0)) * SLOT;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, W * ring + 2 * (W + MAXC) * SLOT);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs, (a.D + 64 * NP - 1) / (64 * NP), parts);
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
// What a CTA of W warps takes, and how many of them share an SM.  The forward has as many warps as leave room for two CTAs.
template <typename X, typename G, bool BWD> struct Room {
  static constexpr int row = SEG * 64, SLOT = sizeof(MapSlot<1>), X_ = sizeof(X), G_ = sizeof(G);
  static constexpr int ring = BWD ? 2 * row * (X_ + G_) + row * X_ : 3 * row * (X_ + G_);
  static constexpr int fwd_warps = (227 * 1024 / 2 - 1024 - 8 * SLOT) / (ring + 2 * SLOT);
  static constexpr int fit(int W) { return 227 * 1024 / (W * ring + 2 * (W + MAXC) * SLOT + 1100); }
  static constexpr int regs(int W) { return 512 / (32 * W); }  // at 128 of a thread
  static constexpr int limit(int W) { return std::max(1, std::min(fit(W), regs(W))); }
};
template <typename X, typename G, int M, int W> cudaError_t launch_bwd(const ScanArgs &a, int sms, cudaStream_t st) {
  typedef Room<X, G, true> R;
  return launch_clustered<W, 1>(scan_bwd_kernel<X, G, M, W, 1, R::limit(W)>, a, R::limit(W) * sms, R::ring, st);
}
template <typename X, typename G, int M> cudaError_t launch_move(const ScanArgs &a, bool bwd, int sms, cudaStream_t st) {
  if (!bwd) {
    typedef Room<X, G, false> R;
    return launch_clustered<R::fwd_warps, 1>(scan_fwd_kernel<X, G, M, R::fwd_warps, 1>, a, 2 * sms, R::ring, st);
  }
  // Four warps to a CTA, and several CTAs to an SM; as many as fit one where not even clusters of eight reach two SMs in three
  // (a sequence of 65536 tokens and 64 channels: 8 CTAs).
  const long long most = (long long)((a.D + 63) / 64) * MAXC * (a.cu ? 1 : a.N);
  if (3 * most < 2 * sms) return launch_bwd<X, G, M, sizeof(X) == 2 ? 12 : 8>(a, sms, st);
  return launch_bwd<X, G, M, 4>(a, sms, st);
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
