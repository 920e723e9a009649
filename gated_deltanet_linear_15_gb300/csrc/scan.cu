// Gated linear recurrence, one state per channel (the elementwise sister of the delta rule, whose gate it shares):
//   h_t = exp(g_t) h_{t-1} + x_t,  y_t = h_t;
// backward, with d_t the gradient that reaches h_t:
//   d_t = dy_t + exp(g_{t+1}) d_{t+1},  dx_t = d_t,  dg_t = exp(g_t) d_t h_{t-1},  dh0 = exp(g_0) d_0.
//
// Bound by bytes: x and g are read once and y is written once; the backward reads dy, x and g and writes dx and dg.  What keeps
// it from the rate of a copy is the chain of rounds below: 4 x 4096 tokens of 2048 channels take 47 us forward (4.3 TB/s; a
// kernel that only copies with these accesses 37 us) and 68 us backward (5.0 TB/s) in bf16, 43 and 66 us with half the tokens in
// fp32; one sequence of 65536 tokens and 64 channels, which eight CTAs share, 123 and 145 us (a call among others, inputs from
// memory; alone, under a profiler, 50 and 73 us for the first).
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
#include "pairs.cuh"

namespace gdn {

namespace {

constexpr int SEG = SCAN_SEG, CB = 64, MAXC = 8;  // tokens of a segment, channels of a block, CTAs of a cluster

// What brings rows: 16-byte copies of rows that begin on 16-byte boundaries; 4-byte copies of bf16 pairs; 16-byte copies
// of the aligned pieces that hold a row that begins anywhere (4 x 4096 tokens, 1001 channels: bf16 forward 48 us and backward
// 95, with plain loads of single values 89 and 132; 32749 packed fp32 tokens 134 us, with 4-byte copies 163, parts as they were).  Pairs keep the
// 4-byte copies where they can, for the stores of pairs that go with them (1002 channels: backward 71 us, 1001: 95).
enum Move { M16, M4, ANY };
// Of a block's channels a lane has two neighbours, or two that lie 32 apart where rows begin anywhere.
template <int M> constexpr bool PAIR = M != ANY;
template <bool P> __device__ __forceinline__ int first_channel(int lane) { return P ? 2 * lane : lane; }

// a lane's two values
struct Two {
  uint64_t v;
};
__device__ __forceinline__ Two two(float a, float b) { return {pk(a, b)}; }
__device__ __forceinline__ float2 floats(const Two &x) {
  float2 f;
  upk(x.v, f.x, f.y);
  return f;
}
__device__ __forceinline__ Two operator+(const Two &a, const Two &b) { return {add2(a.v, b.v)}; }
__device__ __forceinline__ Two operator*(const Two &a, const Two &b) { return {mul2(a.v, b.v)}; }
__device__ __forceinline__ Two fma(const Two &a, const Two &b, const Two &c) { return {fma2(a.v, b.v, c.v)}; }

// 16 bytes to shared memory, of which the first n are read and the others are zeros
__device__ __forceinline__ void copy16(void *smem, const void *gmem, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(smem)), "l"(gmem), "r"(n));
}
// A segment's rows in shared memory, [SEG][PITCH].  With ANY, row i begins up to 15 bytes into its place, as far behind a
// 16-byte boundary as in global memory.
template <typename E, int M> struct Tile {
  static constexpr int A = 16 / (int)sizeof(E), PITCH = CB + (M == ANY ? A : 0), BYTES = SEG * PITCH * (int)sizeof(E);
  const E *p;
  unsigned first, row;  // where row 0 begins, how much further the next one does
  __device__ __forceinline__ Two at(int i) const {
    const int lane = threadIdx.x & 31;
    const E *r = p + i * PITCH;
    if constexpr (M == ANY) {
      r += (first + i * row) & (A - 1);
      return two(tof(r[lane]), tof(r[lane + 32]));
    } else if constexpr (sizeof(E) == 2) {
      const uint32_t u = *reinterpret_cast<const uint32_t *>(r + 2 * lane);
      return two(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    } else {
      return {*reinterpret_cast<const uint64_t *>(r + 2 * lane)};
    }
  }
};
// Brings rows of segments, zeros outside [lo, hi).  (What is past D is never looked at.)  The lane's place in a row and the
// first of its rows stay the same; `at` moves with the segments.
template <typename E, int M> struct Loader {
  typedef Tile<E, M> T;
  static constexpr int V = M == M4 ? 2 : T::A, PER = CB / V;  // values of a piece, pieces of a row
  const E *src, *at;  // at: of the segment asked for next, the lane's first piece (ANY: the block's first channel of row 0)
  long long row, step;
  // s: the first segment; per: how far the next one lies
  __device__ __forceinline__ void init(const void *p, long long stride, int c0, long long s, long long per) {
    const int lane = threadIdx.x & 31;
    src = static_cast<const E *>(p);
    row = stride;
    at = src + s * SEG * row + c0 + (M == ANY ? 0 : lane / PER * row + lane % PER * V);
    step = per * SEG * row;
  }
  __device__ __forceinline__ T tile(const void *place, int t0, int c0) const {
    const unsigned base = (unsigned)(reinterpret_cast<uintptr_t>(src) / sizeof(E)) + c0;
    return {static_cast<const E *>(place), base + (unsigned)t0 * (unsigned)row, (unsigned)row};
  }
  __device__ __forceinline__ void load(void *place, int t0, int lo, int hi, int c0, int D) {
    const int lane = threadIdx.x & 31;
    E *dst = static_cast<E *>(place);
    if constexpr (M == ANY) {
      constexpr int C = PER + 1;  // pieces that a row may reach into; none lacks a byte of the row, so none leaves its allocation
      const int bytes = min(CB, D - c0) * (int)sizeof(E);
#pragma unroll
      for (int k = 0; k < (SEG * C + 31) / 32; ++k) {
        const int i = k * 32 + lane, r = i / C, q = i - r * C;
        const uintptr_t b = reinterpret_cast<uintptr_t>(at + r * row);
        const int off = 16 * q - (int)(b & 15);  // the piece's place in the row
        const int n = t0 + r >= lo && t0 + r < hi ? max(min(16, bytes - off), 0) : 0;  // no byte behind the row's last
        if (r < SEG) copy16(dst + r * T::PITCH + q * T::A, reinterpret_cast<const void *>(n ? b + off : reinterpret_cast<uintptr_t>(src) & ~(uintptr_t)15), n);
      }
    } else {
      constexpr int RPI = 32 / PER;  // rows of an instruction
      const int r0 = lane / PER, c = lane % PER * V;
      E *d = dst + r0 * T::PITCH + c;
      const E *s = at;
      auto copy = [](E *d, const E *s, bool ok) {
        if constexpr (M == M16) copy16(d, s, ok ? 16 : 0);
        else cp_async4(d, s, ok);
      };
      if (c0 + c < D) {
        if (t0 >= lo && t0 + SEG <= hi) {
#pragma unroll
          for (int i = 0; i < SEG / RPI; ++i, s += RPI * row) copy(d + i * RPI * T::PITCH, s, true);
        } else {
          const unsigned span = hi - lo, rel = t0 + r0 - lo;
#pragma unroll 1
          for (int i = 0; i < SEG / RPI; ++i, s += RPI * row) {
            const bool ok = rel + i * RPI < span;
            copy(d + i * RPI * T::PITCH, ok ? s : src, ok);
          }
        }
      }
    }
    at += step;
  }
};
// Gates of a row.  With bf16 rows the product with log2(e) and ex2.approx, off by 2^-22 of themselves, which a bf16 result does
// not show and which the state carries for 16 tokens at most (its map takes expf of the sum); expf in fp32, where 16 such
// errors would be half of all.
template <bool EXACT> __device__ __forceinline__ Two gates(const Two &g) {
  float2 f;
  if constexpr (EXACT) {
    f = floats(g);
    return two(expf(f.x), expf(f.y));
  } else {
    f = floats(g * two(1.4426950408889634f, 1.4426950408889634f));
    asm("ex2.approx.ftz.f32 %0, %0;\n" : "+f"(f.x));
    asm("ex2.approx.ftz.f32 %0, %0;\n" : "+f"(f.y));
    return two(f.x, f.y);
  }
}

// a row in global memory: the lane's channels, of which c is the first; only those below D exist
template <bool P, typename E> __device__ __forceinline__ void put(E *row, int c, int D, const Two &x) {
  const float2 f = floats(x);
  if constexpr (P) {
    if (c < D) st2(row + c, f.x, f.y);
  } else {
    if (c < D) row[c] = fromf<E>(f.x);
    if (c + 32 < D) row[c + 32] = fromf<E>(f.y);
  }
}
template <bool P> __device__ __forceinline__ Two take(const float *row, int c, int D) {
  if constexpr (P) return c < D ? Two{*reinterpret_cast<const uint64_t *>(row + c)} : Two{};
  else return two(c < D ? row[c] : 0.f, c + 32 < D ? row[c + 32] : 0.f);
}

// ------------------------------------------------------------------ where sequences begin
// Tokens of the line that a part takes: whole sequences.  Packed sequences go by where they begin, so that parts are of
// about the same size; equal ones by number.
__device__ __forceinline__ int lower_bound(const int *cu, int n, long long v) {  // entries of cu[0 .. n) below v
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}
__device__ __forceinline__ int token_at(const ScanArgs &a, int n) { return min(max(a.cu[n], 0), a.tokens); }
// where part p begins: at the sequence's end that is nearest to an even cut
__device__ __forceinline__ int part_begin(const ScanArgs &a, int p, int parts) {
  if (!a.cu) return (int)((long long)a.N * p / parts) * a.T;
  if (p == 0 || p == parts) return token_at(a, p ? a.N : 0);
  const int want = (int)((long long)a.tokens * p / parts), at = min(lower_bound(a.cu, a.N + 1, want), a.N);
  const int behind = token_at(a, at), before = at > 0 ? token_at(a, at - 1) : behind;
  return want - before < behind - want ? before : behind;
}
// A part of few packed sequences and many rounds (of `round` tokens): the tokens of the largest part set the time, so the warp
// looks for the least number that lets every part take whole sequences up to it, among 32 from the mean to three times that.
// False where there is none, or where the search would take more than it gives.  (16 sequences, 32749 tokens, 1001 channels
// in fp32, four parts: 123 us, 147 with parts by part_begin; with 8 rounds the search, 1 us, only costs.)
constexpr int FEW_PARTS = 8, FEW_SEQS = 16, MANY_ROUNDS = 16;
__device__ __forceinline__ bool even_parts(const ScanArgs &a, int round, int &lo, int &hi) {
  const int parts = gridDim.z;
  if (!a.cu || parts == 1 || parts > FEW_PARTS || a.N > FEW_SEQS * parts) return false;
  if (a.tokens / parts / round < MANY_ROUNDS) return false;
  const long long mean = ((long long)a.tokens + parts - 1) / parts, most = mean + mean * (threadIdx.x & 31) / 16;
  int n = 0, at = token_at(a, 0), end = at, p = 0;  // at: where part p begins, from sequence n
  for (; p < parts && n < a.N; ++p) {
    const int next = min(lower_bound(a.cu, a.N + 1, at + most + 1) - 1, a.N);
    if (next <= n) break;  // a sequence of more than that
    n = next;
    end = token_at(a, n);
    if (p == (int)blockIdx.z) lo = at, hi = end;
    at = end;
  }
  if (p <= (int)blockIdx.z) lo = hi = end;  // nothing is left for this part
  const unsigned ok = __ballot_sync(0xffffffffu, n == a.N);
  if (!ok) return false;
  lo = __shfl_sync(0xffffffffu, lo, __ffs(ok) - 1);
  hi = __shfl_sync(0xffffffffu, hi, __ffs(ok) - 1);
  return true;
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
      const unsigned d = (unsigned)x - (unsigned)t;
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
struct Map {
  float2 A, H;
  static __device__ __forceinline__ float one(float A, float H, float c) { return A < 0.f ? H : fmaf(A, c, H); }
  static __device__ __forceinline__ float both(float A, float B) { return A < 0.f || B < 0.f ? -1.f : A * B; }
  __device__ __forceinline__ float2 of(const float2 &c) const { return make_float2(one(A.x, H.x, c.x), one(A.y, H.y, c.y)); }
  __device__ __forceinline__ void then(const Map &n) {  // this one first, then n
    H = n.of(H);
    A = make_float2(both(A.x, n.A.x), both(A.y, n.A.y));
  }
};
// of a segment: the sum of its log-gates and its result from zero
__device__ __forceinline__ Map segment_map(bool fresh, const Two &sum, const Two &h) {
  const float2 s = floats(sum);
  return {fresh ? make_float2(-1.f, -1.f) : make_float2(expf(s.x), expf(s.y)), floats(h)};
}
// a map in shared memory, 16 bytes of every lane
typedef float4 MapSlot[32];
__device__ __forceinline__ float4 packed(const Map &m) { return make_float4(m.A.x, m.A.y, m.H.x, m.H.y); }
__device__ __forceinline__ Map map_at(const MapSlot &s) {
  const float4 v = s[threadIdx.x & 31];
  return {make_float2(v.x, v.y), make_float2(v.z, v.w)};
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
template <int W> struct Meet {
  MapSlot *warp, *peer;  // [2][W], [2][cs]
  uint64_t *bar;         // [2]
  int cs, rank;
  __device__ __forceinline__ void init(uint8_t *smem, uint64_t *bars) {
    warp = reinterpret_cast<MapSlot *>(smem);
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
  __device__ __forceinline__ void hand_in(int round, const Map &mine) const {
    const int me = threadIdx.x >> 5, lane = threadIdx.x & 31, par = round & 1;
    MapSlot *mw = warp + par * W;
    mw[me][lane] = packed(mine);
    __syncthreads();
    if (cs == 1) return;
    if (threadIdx.x == 0) bar_expect(smem_u32(bar + par), cs * sizeof(MapSlot));
    if (me >= cs) return;
    Map all = map_at(mw[0]);
#pragma unroll
    for (int j = 1; j < W; ++j) all.then(map_at(mw[j]));
    const uint32_t at = smem_u32(&peer[par * cs + rank][lane]), b = smem_u32(bar + par);
#pragma unroll 1
    for (int r = me; r < cs; r += W) store_peer(peer_addr(at, r), peer_addr(b, r), packed(all));
  }
  __device__ __forceinline__ Two state(int round, float2 &carry) const {
    const int me = threadIdx.x >> 5, par = round & 1;
    const MapSlot *mw = warp + par * W, *mp = peer + par * cs;
    float2 in = carry;
    if (cs == 1) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if (j == me) in = carry;
        carry = map_at(mw[j]).of(carry);
      }
    } else {
      if (!bar_wait(smem_u32(bar + par), round >> 1 & 1))  // what follows is not reliable, and shows it
        carry.x = carry.y = __uint_as_float(0x7fffffffu);
#pragma unroll
      for (int b = 0; b < MAXC; b += 4) {
        if (b >= cs) break;
        Map m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = map_at(mp[min(b + j, cs - 1)]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (b + j < cs) {
            if (b + j == rank) in = carry;
            carry = m[j].of(carry);
          }
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        if (j < me) in = map_at(mw[j]).of(in);
    }
    return two(in.x, in.y);
  }
};

template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// the state of sequences without tokens passes through: out[n] = in[n], shared out among a channel block's CTAs
template <bool P, int W>
__device__ __forceinline__ void pass_empty(const ScanArgs &a, const float *in, float *out, int c, int ctas, int cta) {
  if (!a.cu || !out) return;
  for (int n = cta * W + (threadIdx.x >> 5); n < a.N; n += ctas * W) {
    if (a.cu[n + 1] > a.cu[n]) continue;
    put<P>(out + (long long)n * a.D, c, a.D, in ? take<P>(in + (long long)n * a.D, c, a.D) : Two{});
  }
}

// With zero_rest, rows that no sequence names (of y, or of dx and dg) become zeros, shared out in the same way: gradients of a
// padded batch are summed over all its rows.
template <bool P, int W, typename E>
__device__ __forceinline__ void clear_rest(const ScanArgs &a, E *rows, long long stride, int c, int ctas, int cta) {
  if (!a.cu || !a.zero_rest) return;
  const int begin = token_at(a, 0), named = max(token_at(a, a.N) - begin, 0);
  for (long long i = cta * W + (threadIdx.x >> 5); i < a.tokens - named; i += ctas * W)
    put<P>(rows + (i < begin ? i : i + named) * stride, c, a.D, Two{});
}

// Where a CTA's walk through its part stands.  Segments count in the direction of the walk: number 0 is the part's first
// one, or its last one going backward.
struct Walk {
  int lo, hi;        // tokens of the part
  int rounds, per;   // segments of a round: one for every warp of the cluster
  int first, last;   // the warp's segment of round 0; the line's segment with number 0 going backward
  template <int W> __device__ __forceinline__ void init(const ScanArgs &a, int cs, int rank) {
    per = cs * W;
    if (a.cu && a.N <= (int)gridDim.z) {  // a part for every sequence
      lo = token_at(a, min((int)blockIdx.z, a.N));
      hi = token_at(a, min((int)blockIdx.z + 1, a.N));
    } else if (!even_parts(a, per * SEG, lo, hi)) {
      lo = part_begin(a, blockIdx.z, gridDim.z);
      hi = part_begin(a, blockIdx.z + 1, gridDim.z);
    }
    const int s0 = lo / SEG, ns = hi > lo ? (hi + SEG - 1) / SEG - s0 : 0;
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
template <typename X, typename G, int M, int W>
__global__ void __launch_bounds__(32 * W, 2) scan_fwd_kernel(ScanArgs a) {
  constexpr bool P = PAIR<M>, EXACT = sizeof(X) == 4;
  extern __shared__ __align__(16) uint8_t raw[];
  constexpr int BX = Tile<X, M>::BYTES, ST = BX + Tile<G, M>::BYTES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = gridDim.x, rank = blockIdx.x, c0 = blockIdx.y * CB, c = c0 + first_channel<P>(lane);
  uint8_t *ring = raw + warp * (3 * ST);
  __shared__ uint64_t bars[2];
  Meet<W> mt;
  mt.init(raw + W * 3 * ST, bars);
  pdl_trigger();
  pdl_wait();
  Walk w = {};
  w.init<W>(a, cs, rank);
  Loader<X, M> lx;
  Loader<G, M> lg;
  lx.init(a.x, a.x_row, c0, w.up(0), w.per);
  lg.init(a.g, a.g_row, c0, w.up(0), w.per);
  auto load = [&](int k, int slot) {
    if (k < w.rounds && w.has(w.up(k))) {
      uint8_t *st = ring + slot * ST;
      const int t0 = w.up(k) * SEG;
      lx.load(st, t0, w.lo, w.hi, c0, a.D);
      lg.load(st + BX, t0, w.lo, w.hi, c0, a.D);
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int k = 0; k < 2; ++k) load(k, k);
  Piece now = {}, next = {};
  next.bd.init(a, w.up(0) * SEG);
  pass_empty<P, W>(a, a.h0, a.hT, c, cs * gridDim.z, blockIdx.z * cs + rank);
  clear_rest<P, W>(a, static_cast<X *>(a.y), a.y_row, c, cs * gridDim.z, blockIdx.z * cs + rank);
  mt.ready();
  auto start = [&](const Piece &p, int i) { return a.h0 ? take<P>(a.h0 + (long long)p.bd.seq(a, p.t0 + i) * a.D, c, a.D) : Two{}; };
  float2 carry = make_float2(0.f, 0.f);
  Two h = {};
  int slot = 2;  // of round k
#pragma unroll 1
  for (int k = -1; k < w.rounds; ++k) {
    const int slot1 = slot == 2 ? 0 : slot + 1;
    const bool more = k + 1 < w.rounds;
    if (more) {
      next.look(a, w, w.up(k + 1));
      cp_wait<1>();
      __syncwarp();
      const Tile<X, M> x = lx.tile(ring + slot1 * ST, next.t0, c0);
      const Tile<G, M> g = lg.tile(ring + slot1 * ST + BX, next.t0, c0);
      Two sum = {}, z = {};
      bool fresh = false;
      if (next.plain) {
#pragma unroll
        for (int i = 0; i < SEG; ++i) {
          const Two gi = g.at(i);
          sum = sum + gi;
          z = fma(gates<EXACT>(gi), z, x.at(i));
        }
      } else if (next.live) {
#pragma unroll 1
        for (int i = 0; i < SEG; ++i) {
          const Two gi = g.at(i);
          if (next.begins(i) && next.inside(w, i)) {
            z = start(next, i);
            fresh = true;
          }
          sum = sum + gi;
          z = fma(gates<EXACT>(gi), z, x.at(i));
        }
      }
      mt.hand_in(k + 1, segment_map(fresh, sum, z));
    }
    if (k >= 0 && now.live) {
      const Tile<X, M> x = lx.tile(ring + slot * ST, now.t0, c0);
      const Tile<G, M> g = lg.tile(ring + slot * ST + BX, now.t0, c0);
      if (a.states && now.t0 >= w.lo) put<P>(a.states + (long long)now.seg * a.D, c, a.D, h);
      X *yr = static_cast<X *>(a.y) + (long long)now.t0 * a.y_row;
      if (now.plain) {
#pragma unroll
        for (int i = 0; i < SEG; ++i, yr += a.y_row) {
          h = fma(gates<EXACT>(g.at(i)), h, x.at(i));
          put<P>(yr, c, a.D, h);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < SEG; ++i, yr += a.y_row) {
          if (!now.inside(w, i)) continue;
          if (now.begins(i)) h = start(now, i);
          h = fma(gates<EXACT>(g.at(i)), h, x.at(i));
          put<P>(yr, c, a.D, h);
          if (now.ends(i) && a.hT) put<P>(a.hT + (long long)now.bd.seq(a, now.t0 + i) * a.D, c, a.D, h);
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
template <typename X, typename G, int M, int W, int LIMIT>
__global__ void __launch_bounds__(32 * W, LIMIT) scan_bwd_kernel(ScanArgs a) {
  constexpr bool P = PAIR<M>, EXACT = sizeof(X) == 4;
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ uint64_t bars[2];
  constexpr int BX = Tile<X, M>::BYTES, ST = BX + Tile<G, M>::BYTES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = gridDim.x, rank = blockIdx.x, c0 = blockIdx.y * CB, c = c0 + first_channel<P>(lane);
  uint8_t *ring = raw + warp * (2 * ST + BX);
  uint8_t *sx = ring + 2 * ST;
  Meet<W> mt;
  mt.init(raw + W * (2 * ST + BX), bars);
  pdl_trigger();
  pdl_wait();
  Walk w = {};
  w.init<W>(a, cs, rank);
  Loader<X, M> lx, ld;
  Loader<G, M> lg;
  lx.init(a.x, a.x_row, c0, w.down(0), -w.per);
  ld.init(a.dy, a.dy_row, c0, w.down(0), -w.per);
  lg.init(a.g, a.g_row, c0, w.down(0), -w.per);
  auto load = [&](int k) {  // dy and g of round k
    if (k < w.rounds && w.has(w.down(k))) {
      uint8_t *st = ring + (k & 1) * ST;
      const int t0 = w.down(k) * SEG;
      ld.load(st, t0, w.lo, w.hi, c0, a.D);
      lg.load(st + BX, t0, w.lo, w.hi, c0, a.D);
    }
    cp_async_commit();
  };
  load(0);
  Piece now = {};
  now.bd.init(a, max(w.down(0) * SEG, 0));
  pass_empty<P, W>(a, a.dhT, a.dh0, c, cs * gridDim.z, blockIdx.z * cs + rank);
  clear_rest<P, W>(a, static_cast<X *>(a.y), a.y_row, c, cs * gridDim.z, blockIdx.z * cs + rank);
  clear_rest<P, W>(a, static_cast<G *>(a.dg), a.dg_row, c, cs * gridDim.z, blockIdx.z * cs + rank);
  mt.ready();
  auto start = [&](int i) { return a.h0 ? take<P>(a.h0 + (long long)now.bd.seq(a, now.t0 + i) * a.D, c, a.D) : Two{}; };
  auto at_end = [&](int i) { return a.dhT ? take<P>(a.dhT + (long long)now.bd.seq(a, now.t0 + i) * a.D, c, a.D) : Two{}; };
  float2 carry = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int k = 0; k < w.rounds; ++k) {
    now.look(a, w, w.down(k));
    const uint8_t *st = ring + (k & 1) * ST;
    const Tile<X, M> x = lx.tile(sx, now.t0, c0), dy = ld.tile(st, now.t0, c0);
    const Tile<G, M> g = lg.tile(st + BX, now.t0, c0);
    if (now.live) lx.load(sx, now.t0, w.lo, w.hi, c0, a.D);
    cp_async_commit();
    load(k + 1);
    Two h = now.live ? take<P>(a.states + (long long)now.seg * a.D, c, a.D) : Two{};
    cp_wait<2>();
    __syncwarp();
    Two sum = {}, d = {};  // d: what reaches the state from later tokens
    bool fresh = false;
    if (now.plain) {
#pragma unroll
      for (int i = SEG - 1; i >= 0; --i) {
        const Two gi = g.at(i);
        sum = sum + gi;
        d = gates<EXACT>(gi) * (dy.at(i) + d);
      }
    } else if (now.live) {
#pragma unroll 1
      for (int i = SEG - 1; i >= 0; --i) {
        const Two gi = g.at(i);
        if (now.ends(i) && now.inside(w, i)) {
          d = at_end(i);
          fresh = true;
        }
        sum = sum + gi;
        d = gates<EXACT>(gi) * (dy.at(i) + d);
      }
    }
    mt.hand_in(k, segment_map(fresh, sum, d));
    cp_wait<1>();
    __syncwarp();
    X *dxr = static_cast<X *>(a.y) + (long long)(now.t0 + SEG - 1) * a.y_row;
    G *dgr = static_cast<G *>(a.dg) + (long long)(now.t0 + SEG - 1) * a.dg_row;
    if (now.plain) {
      Two hp[SEG];  // states before the tokens
#pragma unroll
      for (int i = 0; i < SEG; ++i) {
        hp[i] = h;
        h = fma(gates<EXACT>(g.at(i)), h, x.at(i));
      }
      d = mt.state(k, carry);
#pragma unroll
      for (int i = SEG - 1; i >= 0; --i, dxr -= a.y_row, dgr -= a.dg_row) {
        const Two dx = dy.at(i) + d;
        d = gates<EXACT>(g.at(i)) * dx;
        put<P>(dxr, c, a.D, dx);
        put<P>(dgr, c, a.D, d * hp[i]);
      }
    } else {
      d = mt.state(k, carry);
      if (now.live) {
        Two hp[SEG];  // in local memory
#pragma unroll 1
        for (int i = 0; i < SEG; ++i) {
          if (now.begins(i) && now.inside(w, i)) h = start(i);
          hp[i] = h;
          h = fma(gates<EXACT>(g.at(i)), h, x.at(i));
        }
#pragma unroll 1
        for (int i = SEG - 1; i >= 0; --i, dxr -= a.y_row, dgr -= a.dg_row) {
          if (!now.inside(w, i)) continue;
          if (now.ends(i)) d = at_end(i);
          const Two dx = dy.at(i) + d;
          d = gates<EXACT>(g.at(i)) * dx;
          put<P>(dxr, c, a.D, dx);
          put<P>(dgr, c, a.D, d * hp[i]);
          if (now.begins(i) && a.dh0) put<P>(a.dh0 + (long long)now.bd.seq(a, now.t0 + i) * a.D, c, a.D, d);
        }
      }
    }
    __syncwarp();
  }
  cp_async_wait_all();
}

// One token of every sequence: state = exp(g) state + x, y = state.  V channels a thread: four where rows allow it, or one.
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
// within a cluster first.  peers: CTAs of a cluster at most.
void split(const ScanArgs &a, int W, int ctas, int peers, int &parts, int &cs) {
  const int nb = (a.D + CB - 1) / CB, want = std::max(1, ctas / nb);  // CTAs of a channel block
  const auto clustered = [&](int most, long long tokens) {
    return (int)std::max(1ll, std::min({(long long)most, (long long)peers, tokens / (W * SEG)}));
  };
  if (!a.cu) {
    parts = std::min(a.N, want);
    cs = clustered(want / parts, a.tokens / parts);
  } else {
    cs = clustered(want, a.tokens);
    parts = std::min(a.N, std::max(1, want / cs));
    if (a.N < 2 * parts) parts = a.N;  // (12 sequences of up to 4000 tokens, 512 channels, backward: 2.5 TB/s, 2.3 in 9 parts)
  }
  parts = std::min(parts, 65535);
}

// ring: bytes of a warp's stages
template <int W, typename... KArgs>
cudaError_t launch_clustered(void (*k)(KArgs...), const ScanArgs &a, int ctas, int ring, int peers, cudaStream_t st) {
  constexpr int SLOT = sizeof(MapSlot);
  int parts, cs;
  split(a, W, ctas, peers, parts, cs);
  const int smem = W * ring + 2 * (W + (cs > 1 ? cs : 0)) * SLOT;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, W * ring + 2 * (W + MAXC) * SLOT);
  if (e != cudaSuccess) return e;
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
constexpr int HALF_SM = 227 * 1024 / 2 - 1024;  // shared memory of one of two CTAs
// What a CTA of W warps takes, and how many of them share an SM.  The forward has as many warps as leave
// room for two CTAs, with eight peers or at least four (fp32 rows that begin anywhere: 16 packed sequences of up to 4000
// tokens, 1001 channels: 3.2 TB/s with four warps and four peers, 2.7 with three and eight, 2.6 with four and six).
template <typename X, typename G, int M, bool BWD> struct Room {
  static constexpr int SLOT = sizeof(MapSlot), BX = Tile<X, M>::BYTES, BG = Tile<G, M>::BYTES;
  static constexpr int ring = BWD ? 2 * (BX + BG) + BX : 3 * (BX + BG);
  static constexpr int fwd_warps() { return (HALF_SM - 4 * 2 * SLOT) / (ring + 2 * SLOT); }
  static constexpr int fwd_peers() { return HALF_SM - fwd_warps() * (ring + 2 * SLOT) >= MAXC * 2 * SLOT ? MAXC : 4; }
  static constexpr int fit(int W) { return 227 * 1024 / (W * ring + 2 * (W + MAXC) * SLOT + 1100); }
  static constexpr int regs(int W) { return 512 / (32 * W); }  // at 128 of a thread
  static constexpr int limit(int W) { return std::max(1, std::min(fit(W), regs(W))); }
};
template <typename X, typename G, int M, int W> cudaError_t launch_bwd(const ScanArgs &a, int sms, cudaStream_t st) {
  typedef Room<X, G, M, true> R;
  return launch_clustered<W>(scan_bwd_kernel<X, G, M, W, R::limit(W)>, a, R::limit(W) * sms, R::ring, MAXC, st);
}
template <typename X, typename G, int M> cudaError_t launch_move(const ScanArgs &a, bool bwd, int sms, cudaStream_t st) {
  if (!bwd) {
    typedef Room<X, G, M, false> R;
    return launch_clustered<R::fwd_warps()>(scan_fwd_kernel<X, G, M, R::fwd_warps()>, a, 2 * sms, R::ring, R::fwd_peers(), st);
  }
  // Four warps to a CTA, and several CTAs to an SM; as many as fit one where not even clusters of eight reach two SMs in three
  // (a sequence of 65536 tokens and 64 channels: 8 CTAs; but 24 packed ones of up to 2900 tokens and 512 channels take 2.7 TB/s with
  // four warps and 1.2 with twelve).
  const long long most = (long long)((a.D + CB - 1) / CB) * MAXC * a.N;
  if (3 * most < 2 * sms) return launch_bwd<X, G, M, sizeof(X) == 2 ? 12 : 8>(a, sms, st);
  return launch_bwd<X, G, M, 4>(a, sms, st);
}
template <typename X, typename G> cudaError_t launch_types(const ScanArgs &a, int move, bool bwd, int sms, cudaStream_t st) {
  if (move == 16) return launch_move<X, G, M16>(a, bwd, sms, st);
  if constexpr (sizeof(X) + sizeof(G) == 4) {
    if (move == 4) return launch_move<X, G, M4>(a, bwd, sms, st);
  }
  return launch_move<X, G, ANY>(a, bwd, sms, st);
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
