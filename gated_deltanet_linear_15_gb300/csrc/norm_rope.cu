// Root-mean-square norm of each head of q and k, and its turn to the token's position, in one pass:
//   r = (mean(x^2) + eps)^(-1/2),  y = R(p) (r x (w + off)),
// R(p) the turn of the feature pairs by position p (rope.cu).  Backward, with u = R(p)^T dy and xhat = r x:
//   dx = r (u (w + off) - xhat mean(u (w + off) xhat)),  dw = sum over tokens and heads of u xhat.
// No power of r stands alone: with a small eps those of a head of zeros leave fp32, and what they multiply is 0.
// With a paged cache the keys and values of new tokens go to their slots in the same pass.
//
// Bound by bytes: every element is read once and written once (backward: x and dy read, dx written).  A thread's unit is
// that of rope.cu, 32 bytes of a head that hold whole pairs; the D sizeof(I) / 32 threads of a head are neighbours in a
// warp, so a head's sums take a few shuffles, and the data stay in registers between the sum and the turn.  Units come by
// cp.async to places of the thread's own, a few ahead of the one in work.  (Loaded to registers instead, as in rope.cu,
// the sums' latencies left too few bytes in flight: 8192 tokens of 32 + 8 + 8 heads 50 us.)  Arithmetic is in packed
// pairs of fp32.  8192 tokens of 32 + 8 + 8 heads of 128, bf16, appended: 36.8 us on the GPU, 5.6 TB/s (rope.cu without the
// norm: 34.3); the backward of 16384 tokens of 16 + 4 heads: 44 us, 5.8 TB/s, and 4 us for the weights' sums.
//
// The backward's CTAs stay and walk over tokens, some of them over the heads of q and the others over those of k, since a
// thread's place in the head does not change: it keeps its sums of dw in registers.  Each CTA leaves one partial row, and a
// second kernel adds these in order.
//
// Heads whose size, strides or alignment do not allow 16-byte units: a warp to a head.
#include <algorithm>

#include "rope.cuh"
#include "pairs.cuh"

namespace gdn {

namespace {

constexpr int UNF = 3, UNB = 2;  // units of a thread on their way, forward and backward
constexpr int NTB = 256, MAXD = NORM_ROPE_MAX_DIM;  // threads of the backward, features of a head

// sum over the neighbouring lanes (UPH, or n where that is 0: a power of two) that hold a head
template <int UPH> __device__ __forceinline__ float head_sum(float x, int n) {
  const int m = UPH ? UPH : n;
  const unsigned mask = m == 32 ? 0xffffffffu : ((1u << m) - 1) << (threadIdx.x & 31 & ~(m - 1));
  if constexpr (UPH > 0) {
#pragma unroll
    for (int o = UPH / 2; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
  } else {
    for (int o = m >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
  }
  return x;
}
// 16 bytes to shared memory.  Where a unit's pieces are neighbours, each of its two copies takes half a sector, and they go by
// way of L1, so that L2 is asked once (with this and the stores below 16384 tokens of 16 + 4 interleaved heads go backward in
// 44 us instead of 66; pieces that are not neighbours are 2 us faster past L1, 8192 tokens of 48 heads appended).  A place is
// asked for again right after it was read: the copies are "memory" to the compiler, which may not move that read behind them.
__device__ __forceinline__ void copy16(void *smem, const void *gmem, bool neighbours) {
  if (neighbours) asm volatile("cp.async.ca.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(smem)), "l"(gmem) : "memory");
  else asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(smem)), "l"(gmem) : "memory");
}
// both pieces of a unit to global memory, in one store where they are neighbours on a 32-byte boundary (two of half a
// sector each otherwise)
template <typename I> __device__ __forceinline__ void store_unit(I *p, int gap, const uint4 &a, const uint4 &b) {
  if (gap * sizeof(I) == 16 && (reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x),
                 "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    *reinterpret_cast<uint4 *>(p) = a;
    *reinterpret_cast<uint4 *>(p + gap) = b;
  }
}
// A unit's features as packed pairs: piece 0 in v[0 .. PV), piece 1 in v[PV .. 2 PV).
template <typename I> struct Unit {
  static constexpr int V = 16 / sizeof(I), PV = V / 2;
  uint64_t v[2 * PV];
  __device__ __forceinline__ void widen(const uint4 &a, const uint4 &b) {
    if constexpr (sizeof(I) == 2) {
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
      v[0] = pk(__uint_as_float(a.x), __uint_as_float(a.y));
      v[1] = pk(__uint_as_float(a.z), __uint_as_float(a.w));
      v[2] = pk(__uint_as_float(b.x), __uint_as_float(b.y));
      v[3] = pk(__uint_as_float(b.z), __uint_as_float(b.w));
    }
  }
  __device__ __forceinline__ void pack(uint4 &a, uint4 &b) const {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 2 * PV; ++i) {
      float x, y;
      upk(v[i], x, y);
      if constexpr (sizeof(I) == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      } else {
        w[2 * i] = __float_as_uint(x);
        w[2 * i + 1] = __float_as_uint(y);
      }
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
  }
  // four values every `step` places
  __device__ __forceinline__ void read(const float4 *p, int step) {
#pragma unroll
    for (int i = 0; i < PV; ++i) {
      const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(p + i * step);
      v[2 * i] = a.x;
      v[2 * i + 1] = a.y;
    }
  }
  __device__ __forceinline__ float dot(const Unit &o) const {
    uint64_t s0 = mul2(v[0], o.v[0]), s1 = mul2(v[PV], o.v[PV]);
#pragma unroll
    for (int i = 1; i < PV; ++i) {
      s0 = fma2(v[i], o.v[i], s0);
      s1 = fma2(v[PV + i], o.v[PV + i], s1);
    }
    float x, y;
    upk(add2(s0, s1), x, y);
    return x + y;
  }
  __device__ __forceinline__ Unit operator*(const Unit &o) const {
    Unit r;
#pragma unroll
    for (int i = 0; i < 2 * PV; ++i) r.v[i] = mul2(v[i], o.v[i]);
    return r;
  }
  __device__ __forceinline__ Unit operator*(float f) const {
    const uint64_t ff = pk(f, f);
    Unit r;
#pragma unroll
    for (int i = 0; i < 2 * PV; ++i) r.v[i] = mul2(v[i], ff);
    return r;
  }
  __device__ __forceinline__ Unit plus(const Unit &o, float f) const {  // this + o f
    const uint64_t ff = pk(f, f);
    Unit r;
#pragma unroll
    for (int i = 0; i < 2 * PV; ++i) r.v[i] = fma2(o.v[i], ff, v[i]);
    return r;
  }
};
// A unit's angles: halves (IL false): pairs of feature i of both pieces, c, s and -s of two neighbours in a word; interleaved:
// pairs of neighbours, (c, c) and (-s, s).
template <typename I, bool IL> struct Angles {
  static constexpr int V = Unit<I>::V, PV = V / 2, N = IL ? V : PV;
  uint64_t c[N], s[N], m[IL ? 1 : N];
  // from the table's floats of the pairs u V .., four every `step` places
  __device__ __forceinline__ void read(const float4 *cs, int step, bool inverse) {
#pragma unroll
    for (int i = 0; i < PV; ++i) {
      float4 w = cs[i * step];
      if (inverse) {
        w.y = -w.y;
        w.w = -w.w;
      }
      if constexpr (IL) {
        c[2 * i] = pk(w.x, w.x);
        c[2 * i + 1] = pk(w.z, w.z);
        s[2 * i] = pk(-w.y, w.y);
        s[2 * i + 1] = pk(-w.w, w.w);
      } else {
        c[i] = pk(w.x, w.z);
        s[i] = pk(w.y, w.w);
        m[i] = pk(-w.y, -w.w);
      }
    }
  }
  __device__ __forceinline__ void turn(Unit<I> &x) const {
    if constexpr (IL) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float p, q;
        upk(x.v[i], p, q);
        x.v[i] = fma2(pk(q, p), s[i], mul2(x.v[i], c[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < PV; ++i) {
        const uint64_t p = x.v[i], q = x.v[PV + i];
        x.v[i] = fma2(q, m[i], mul2(p, c[i]));
        x.v[PV + i] = fma2(p, s[i], mul2(q, c[i]));
      }
    }
  }
};
// where a position's angles of the unit's pairs u V .. lie
template <int V> __device__ __forceinline__ const float4 *angles_at(const RopeArgs &a, int pos, int u) {
  return reinterpret_cast<const float4 *>(a.table + ((long long)pos * (a.rot / 2) + u * V) * 2);
}
// Weights in shared memory in the units' order: the k-th four of unit u at [k * uph + u], so that neighbouring lanes
// read neighbouring places (in the features' order four lanes at a time met in the same banks: a quarter of the backward's time).
template <int V, bool IL, int NT> __device__ __forceinline__ void stage_weights(float4 *dst, const float *w, float off, const RopeArgs &a, int uph) {
  for (int i = threadIdx.x; i < uph * (V / 2); i += NT) {
    const int u = i % uph, k = i / uph;
    const bool halves = u * 2 * V < a.rot && !IL;
    const int f0 = halves ? u * V : u * 2 * V, gap = halves ? a.rot / 2 : V, f = k < V / 4 ? f0 + 4 * k : f0 + gap + 4 * (k - V / 4);
    dst[i] = make_float4(w[f] + off, w[f + 1] + off, w[f + 2] + off, w[f + 3] + off);
  }
}
struct HeadOf {
  int group, head;
};
__device__ __forceinline__ HeadOf head_of(const RopeArgs &a, int h) {
  const int h1 = a.grp[0].heads, h2 = h1 + (a.ngrp > 1 ? a.grp[1].heads : 0), g = (h >= h1) + (h >= h2);
  return {g, h - (g == 0 ? 0 : (g == 1 ? h1 : h2))};
}

}  // namespace

// The next UN units of a thread are on their way to its own places in shared memory at any time: what is in flight takes no
// registers, and only the thread itself reads it.
template <typename I, int UN, bool IL, int UPH, bool PAGED>
__global__ void __launch_bounds__(NTR, 7) norm_rope_kernel(const __grid_constant__ NormRopeArgs n, int units, int slots) {
  constexpr int V = 16 / sizeof(I);
  const RopeArgs &a = n.r;
  const int uph = UPH ? UPH : units;
  __shared__ uint4 ring[UN][2][NTR];
  __shared__ float4 w[2][(UPH ? UPH * 2 * V : MAXD) / 4];
  pdl_trigger();
  pdl_wait();
  const int tpt = uph * slots, tpb = NTR / tpt;
  const int tl = threadIdx.x / tpt, in = threadIdx.x - tl * tpt, hs = in / uph, u = in - hs * uph;
  const long long t = (long long)blockIdx.x * tpb + tl;
  const bool there = tl < tpb && t < a.tokens;
  const bool turned = u * 2 * V < a.rot, halves = turned && !IL;
  const int f0 = halves ? u * V : u * 2 * V, gap = halves ? a.rot / 2 : V;  // the unit's pieces
  // asking: the thread's heads of one group after another
  int gi = -1, left = 0, slot = 0;  // heads of group gi still to be asked for; the place of the next one
  const I *src = nullptr;
  long long s_step = 0;
  auto ask = [&] {
    while (left <= 0 && gi + 1 < a.ngrp) {
      const RopeGroup &g = a.grp[++gi];
      left = g.heads - hs;
      s_step = slots * g.s_head;
      src = static_cast<const I *>(g.src) + t * g.s_tok + hs * g.s_head + f0;
    }
    if (left > 0) {
      copy16(&ring[slot][0][threadIdx.x], src, gap == V);
      copy16(&ring[slot][1][threadIdx.x], src + gap, gap == V);
      src += s_step;
      left -= slots;
    }
    cp_async_commit();
    slot = slot + 1 == UN ? 0 : slot + 1;
  };
  if (there) {
#pragma unroll 1
    for (int j = 0; j < UN; ++j) ask();
  }
  stage_weights<V, IL, NTR>(w[0], n.w[0], n.off, a, uph);
  if (n.w[1]) stage_weights<V, IL, NTR>(w[1], n.w[1], n.off, a, uph);
  __syncthreads();
  if (!there) return;
  const float inv_d = 1.f / (float)a.D;
  const TokPlace pl = place_of(a, (int)t);
  const bool turns = turned && pl.pos >= 0;
  Angles<I, IL> an;
  if (turns) an.read(angles_at<V>(a, pl.pos, u), 1, false);
  int at = 0;  // the place of the next unit to be worked on
  // the thread's heads of one group: `norm` and `page` at compile time, so that nothing is asked in the loop
  auto walk = [&](const RopeGroup &g, const float4 *weight, auto norm, auto page) {
    const long long d_step = slots * g.d_head;
    I *dst = static_cast<I *>(g.dst) + hs * g.d_head + f0;
    if constexpr (decltype(page)::value) dst += pl.page * g.d_page + pl.off * g.d_tok;
    else dst += t * g.d_tok;
#pragma unroll 1
    for (int h = hs; h < g.heads; h += slots) {
      asm volatile("cp.async.wait_group %0;\n" ::"n"(UN - 1) : "memory");
      uint4 x0 = ring[at][0][threadIdx.x], x1 = ring[at][1][threadIdx.x];
      at = at + 1 == UN ? 0 : at + 1;
      if constexpr (decltype(norm)::value) {
        Unit<I> x, wt;
        x.widen(x0, x1);
        const float r = rsqrtf(fmaf(head_sum<UPH>(x.dot(x), uph), inv_d, n.eps));
        wt.read(weight + u, uph);
        x = x * wt;
        if (turns) an.turn(x);
        (x * r).pack(x0, x1);
      }
      store_unit(dst, gap, x0, x1);
      dst += d_step;
      ask();
    }
  };
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  walk(a.grp[0], w[0], yes, no);
  if constexpr (PAGED) {
    if (pl.page >= 0) {
      walk(a.grp[1], w[1], yes, yes);
      walk(a.grp[2], w[1], no, yes);
    }
  } else {
    if (a.ngrp > 1) walk(a.grp[1], w[1], yes, no);
  }
  cp_async_wait_all();
}

// any head of up to MAXD features: a warp to a head, its lanes over pairs (past rot: over features)
template <typename I> __global__ void __launch_bounds__(NTR) norm_rope_any_kernel(NormRopeArgs n) {
  const RopeArgs &a = n.r;
  pdl_trigger();
  pdl_wait();
  const int half = a.rot / 2, per = half + a.D - a.rot, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long all = (long long)a.tokens * a.heads;
  for (long long i = (long long)blockIdx.x * (NTR / 32) + warp; i < all; i += (long long)gridDim.x * (NTR / 32)) {
    const int t = (int)(i / a.heads);
    const HeadOf ho = head_of(a, (int)(i - (long long)t * a.heads));
    const RopeGroup &g = a.grp[ho.group];
    const TokPlace pl = place_of(a, t);
    if (g.d_page && pl.page < 0) continue;
    const I *src = static_cast<const I *>(g.src) + (long long)t * g.s_tok + ho.head * g.s_head;
    I *dst = static_cast<I *>(g.dst) + ho.head * g.d_head + (g.d_page ? pl.page * g.d_page + pl.off * g.d_tok : (long long)t * g.d_tok);
    if (!g.turn) {
      for (int f = lane; f < a.D; f += 32) dst[f] = src[f];
      continue;
    }
    float sum = 0.f;
    for (int f = lane; f < a.D; f += 32) {
      const float x = tof(src[f]);
      sum += x * x;
    }
    const float r = rsqrtf(warp_sum(sum) / (float)a.D + n.eps);
    const float *w = n.w[ho.group];
    for (int k = lane; k < per; k += 32) {
      if (k >= half) {
        const int f = k - half + a.rot;
        dst[f] = fromf<I>(tof(src[f]) * (r * (w[f] + n.off)));
        continue;
      }
      const int f0 = a.interleaved ? 2 * k : k, f1 = a.interleaved ? 2 * k + 1 : k + half;
      float x = tof(src[f0]) * (r * (w[f0] + n.off)), y = tof(src[f1]) * (r * (w[f1] + n.off));
      if (pl.pos >= 0) {
        const float *cs = a.table + ((long long)pl.pos * half + k) * 2;
        const float c = cs[0], s = cs[1], z = x * c - y * s;
        y = y * c + x * s;
        x = z;
      }
      dst[f0] = fromf<I>(x);
      dst[f1] = fromf<I>(y);
    }
  }
}

// Backward: group g's src is x, its dst dx; dy beside them.  The first `split` CTAs take the heads of group 0, the others those
// of group 1.  part: [gridDim.x][D].  A thread's items are its heads of one token after another, the next UN of them on their
// way to shared memory as in the forward, a token's angles with its first head.
template <typename I, int UN, bool IL, int UPH, int gi>
__device__ __forceinline__ void norm_rope_bwd_group(const NormRopeArgs &n, int units, int slots, int cta, int ctas) {
  constexpr int V = 16 / sizeof(I), PV = V / 2;
  const RopeArgs &a = n.r;
  const int uph = UPH ? UPH : units;
  __shared__ float4 w[(UPH ? UPH * 2 * V : MAXD) / 4];
  extern __shared__ uint4 ring_mem[];
  uint4(*ring)[4 + PV][NTB] = reinterpret_cast<uint4(*)[4 + PV][NTB]>(ring_mem);  // [UN]: x, dy, angles
  static_assert(UN * 4 * 16 >= (2 * V + 1) * 4, "the sums fit the rings");
  const RopeGroup &g = a.grp[gi];
  pdl_trigger();
  pdl_wait();
  stage_weights<V, IL, NTB>(w, n.w[gi], n.off, a, uph);
  __syncthreads();
  const int tpt = uph * slots, tpb = NTB / tpt;
  const int tl = threadIdx.x / tpt, in = threadIdx.x - tl * tpt, hs = in / uph, u = in - hs * uph;
  const bool turned = u * 2 * V < a.rot, halves = turned && !IL;
  const int f0 = halves ? u * V : u * 2 * V, f1 = halves ? u * V + a.rot / 2 : u * 2 * V + V;
  const int step = ctas * tpb;
  const float inv_d = 1.f / (float)a.D;
  Unit<I> dw = {};
  // of a token: its position, -1 where it does not turn
  auto position = [&](long long t) {
    const int pos = turned && t < a.tokens ? a.positions[t] : -1;
    return pos < a.rows ? pos : -1;
  };
  long long t = (long long)cta * tpb + tl;
  if (tl < tpb && t < a.tokens && hs < g.heads) {
    const int gap = f1 - f0;
    // asking: the thread's heads of one token after another, with the first of a token its angles
    long long ta = t;
    int ha = hs, slot = 0, at = 0, pos = position(t), pos1 = position(t + step);
    unsigned turning = 0;  // which places hold the first head of a token that turns
    const I *src = static_cast<const I *>(g.src) + t * g.s_tok + hs * g.s_head + f0;
    const I *dy = static_cast<const I *>(n.dy[gi]) + t * n.dy_tok[gi] + hs * n.dy_head[gi] + f0;
    auto ask = [&] {
      if (ta < a.tokens) {
        copy16(&ring[slot][0][threadIdx.x], src, gap == V);
        copy16(&ring[slot][1][threadIdx.x], src + gap, gap == V);
        copy16(&ring[slot][2][threadIdx.x], dy, gap == V);
        copy16(&ring[slot][3][threadIdx.x], dy + gap, gap == V);
        if (ha == hs) {
          turning &= ~(1u << slot);
          if (pos >= 0) {
            turning |= 1u << slot;
            const float4 *cs = angles_at<V>(a, pos, u);
#pragma unroll
            for (int i = 0; i < PV; ++i) copy16(&ring[slot][4 + i][threadIdx.x], cs + i, true);
          }
          pos = pos1;
          pos1 = position(ta + 2ll * step);
        }
        ha += slots;
        if (ha < g.heads) {
          src += slots * g.s_head;
          dy += slots * n.dy_head[gi];
        } else {
          src += step * g.s_tok - (ha - slots - hs) * g.s_head;
          dy += step * n.dy_tok[gi] - (ha - slots - hs) * n.dy_head[gi];
          ha = hs;
          ta += step;
        }
      }
      cp_async_commit();
      slot = slot + 1 == UN ? 0 : slot + 1;
    };
#pragma unroll 1
    for (int j = 0; j < UN; ++j) ask();
    I *dst = static_cast<I *>(g.dst) + t * g.d_tok + hs * g.d_head + f0;
    for (; t < a.tokens; t += step, dst += step * g.d_tok) {
      Angles<I, IL> an;
      bool turns = false;
      I *out = dst;
#pragma unroll 1
      for (int h = hs; h < g.heads; h += slots, out += slots * g.d_head) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(UN - 1) : "memory");
        if (h == hs) {
          turns = turning >> at & 1;
          if (turns) an.read(reinterpret_cast<const float4 *>(&ring[at][4][threadIdx.x]), NTB, true);
        }
        Unit<I> x, y, wt;
        x.widen(ring[at][0][threadIdx.x], ring[at][1][threadIdx.x]);
        y.widen(ring[at][2][threadIdx.x], ring[at][3][threadIdx.x]);
        at = at + 1 == UN ? 0 : at + 1;
        if (turns) an.turn(y);
        wt.read(w + u, uph);
        wt = wt * y;  // u (w + off)
        const float sum = head_sum<UPH>(x.dot(x), uph), dot = head_sum<UPH>(x.dot(wt), uph);
        const float r = rsqrtf(fmaf(sum, inv_d, n.eps));
        y = y * r;
#pragma unroll
        for (int i = 0; i < 2 * PV; ++i) dw.v[i] = fma2(y.v[i], x.v[i], dw.v[i]);
        uint4 o0, o1;
        (wt.plus(x, -(r * (r * (dot * inv_d)))) * r).pack(o0, o1);
        store_unit(out, gap, o0, o1);
        ask();
      }
    }
    cp_async_wait_all();
  }
  __syncthreads();  // the rings' memory holds the sums now
  float(&sums)[NTB][2 * V + 1] = *reinterpret_cast<float(*)[NTB][2 * V + 1]>(ring);
  // the threads of one place in the head, in order
#pragma unroll
  for (int i = 0; i < 2 * PV; ++i) upk(dw.v[i], sums[threadIdx.x][2 * i], sums[threadIdx.x][2 * i + 1]);
  __syncthreads();
  for (int f = threadIdx.x; f < a.D; f += NTB) {
    const int fu = f / (2 * V), i = f - fu * 2 * V;
    float z = 0.f;
    for (int k = fu; k < tpb * tpt; k += uph) z += sums[k][i];
    const bool fh = fu * 2 * V < a.rot && !IL;
    const int at = fh ? (i < V ? fu * V + i : fu * V + a.rot / 2 + i - V) : f;
    n.part[(long long)blockIdx.x * a.D + at] = z;
  }
}

template <typename I, int UN, bool IL, int UPH>
__global__ void __launch_bounds__(NTB, 2) norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs n, int units, int slots0, int slots1, int split) {
  // the group at compile time, so that its strides are constants and no loads in the loop
  if ((int)blockIdx.x < split) norm_rope_bwd_group<I, UN, IL, UPH, 0>(n, units, slots0, blockIdx.x, split);
  else norm_rope_bwd_group<I, UN, IL, UPH, 1>(n, units, slots1, blockIdx.x - split, gridDim.x - split);
}

// a warp to a head, which keeps its sums of dw in shared memory; the CTA's warps add up in order at the end
template <typename I> __global__ void __launch_bounds__(NTR) norm_rope_bwd_any_kernel(NormRopeArgs n, int split) {
  const RopeArgs &a = n.r;
  extern __shared__ float acc[];  // [warps][D]
  const int gi = (int)blockIdx.x >= split, cta = blockIdx.x - (gi ? split : 0), ctas = gi ? gridDim.x - split : split;
  const RopeGroup g = a.grp[gi];
  pdl_trigger();
  pdl_wait();
  const int half = a.rot / 2, per = half + a.D - a.rot, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < NTR / 32 * a.D; i += NTR) acc[i] = 0.f;
  __syncthreads();
  const long long all = (long long)a.tokens * g.heads;
  for (long long i = (long long)cta * (NTR / 32) + warp; i < all; i += (long long)ctas * (NTR / 32)) {
    const int t = (int)(i / g.heads), h = (int)(i - (long long)t * g.heads);
    const TokPlace pl = place_of(a, t);
    const I *x = static_cast<const I *>(g.src) + (long long)t * g.s_tok + h * g.s_head;
    const I *dy = static_cast<const I *>(n.dy[gi]) + (long long)t * n.dy_tok[gi] + h * n.dy_head[gi];
    I *dx = static_cast<I *>(g.dst) + (long long)t * g.d_tok + h * g.d_head;
    const float *w = n.w[gi];
    float *dw = acc + warp * a.D;
    // u of the lane's k-th pair or feature
    auto back = [&](int k, int &f0, int &f1, float &u0, float &u1) {
      f0 = f1 = k - half + a.rot;
      u1 = 0.f;
      if (k >= half) {
        u0 = tof(dy[f0]);
        return;
      }
      f0 = a.interleaved ? 2 * k : k;
      f1 = a.interleaved ? 2 * k + 1 : k + half;
      u0 = tof(dy[f0]);
      u1 = tof(dy[f1]);
      if (pl.pos >= 0) {
        const float *cs = a.table + ((long long)pl.pos * half + k) * 2;
        const float c = cs[0], s = cs[1], z = u0 * c + u1 * s;
        u1 = u1 * c - u0 * s;
        u0 = z;
      }
    };
    float sum = 0.f, dot = 0.f;
    for (int k = lane; k < per; k += 32) {
      int f0, f1;
      float u0, u1;
      back(k, f0, f1, u0, u1);
      const float x0 = tof(x[f0]), x1 = k < half ? tof(x[f1]) : 0.f;
      sum += x0 * x0 + x1 * x1;
      dot += x0 * (u0 * (w[f0] + n.off)) + x1 * (u1 * (w[f1] + n.off));
    }
    sum = warp_sum(sum);
    dot = warp_sum(dot);
    const float r = rsqrtf(sum / (float)a.D + n.eps), m = r * (r * (dot / (float)a.D));
    for (int k = lane; k < per; k += 32) {
      int f0, f1;
      float u0, u1;
      back(k, f0, f1, u0, u1);
      const float x0 = tof(x[f0]), x1 = k < half ? tof(x[f1]) : 0.f;
      dx[f0] = fromf<I>(r * (u0 * (w[f0] + n.off) - x0 * m));
      dw[f0] += u0 * (x0 * r);
      if (k < half) {
        dx[f1] = fromf<I>(r * (u1 * (w[f1] + n.off) - x1 * m));
        dw[f1] += u1 * (x1 * r);
      }
    }
  }
  __syncthreads();
  for (int f = threadIdx.x; f < a.D; f += NTR) {
    float z = 0.f;
    for (int k = 0; k < NTR / 32; ++k) z += acc[k * a.D + f];
    n.part[(long long)blockIdx.x * a.D + f] = z;
  }
}

// dw of each group: its CTAs' partial rows in order, 32 features by 32 shares of the rows to a block
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float *part, int rows, int split, int D, float *dw0, float *dw1) {
  __shared__ float sh[32][32];
  pdl_trigger();
  pdl_wait();
  const int f = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5, g = blockIdx.y;
  const int begin = g ? split : 0, count = g ? rows - split : split;
  float z = 0.f;
  if (f < D) {
    const int r0 = begin + count * y / 32, r1 = begin + count * (y + 1) / 32;
#pragma unroll 8
    for (int r = r0; r < r1; ++r) z += part[(long long)r * D + f];
  }
  sh[y][threadIdx.x & 31] = z;
  __syncthreads();
  if (y != 0 || f >= D) return;
  z = 0.f;
#pragma unroll
  for (int k = 0; k < 32; ++k) z += sh[k][threadIdx.x];
  (g ? dw1 : dw0)[f] = z;
}

// the kernels' variants by type, pairing and the units of a head (0: any)
namespace {
template <typename I, int UN, bool IL, bool PAGED> auto forward_kernel(int uph) {
  switch (uph) {
    case 4: return norm_rope_kernel<I, UN, IL, 4, PAGED>;
    case 8: return norm_rope_kernel<I, UN, IL, 8, PAGED>;
    case 16: return norm_rope_kernel<I, UN, IL, 16, PAGED>;
    default: return norm_rope_kernel<I, UN, IL, 0, PAGED>;
  }
}
template <typename I, int UN> auto forward_kernel(const RopeArgs &a, int uph) {
  if (a.positions) return a.interleaved ? forward_kernel<I, UN, true, false>(uph) : forward_kernel<I, UN, false, false>(uph);
  return a.interleaved ? forward_kernel<I, UN, true, true>(uph) : forward_kernel<I, UN, false, true>(uph);
}
template <typename I, bool IL> auto backward_kernel(int uph) {
  switch (uph) {
    case 4: return norm_rope_bwd_kernel<I, UNB, IL, 4>;
    case 8: return norm_rope_bwd_kernel<I, UNB, IL, 8>;
    case 16: return norm_rope_bwd_kernel<I, UNB, IL, 16>;
    default: return norm_rope_bwd_kernel<I, UNB, IL, 0>;
  }
}
}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &n, bool bf, bool vec, cudaStream_t st) {
  const RopeArgs &a = n.r;
  if (!vec) {
    const dim3 grid((unsigned)std::min((long long)a.tokens * a.heads / (NTR / 32) + 1, 152ll * 64));
    return bf ? launch_pdl(norm_rope_any_kernel<bf16>, grid, dim3(NTR), 0, st, n)
              : launch_pdl(norm_rope_any_kernel<float>, grid, dim3(NTR), 0, st, n);
  }
  // 64 threads a token (each walks over a few heads), more while that leaves SMs without work
  const int uph = a.D * (bf ? 2 : 4) / 32;
  int slots = 64 / uph > 0 ? 64 / uph : 1;
  while (slots < a.heads && 2 * slots * uph <= NTR && (long long)a.tokens * slots * uph < 152ll * 4 * NTR) slots *= 2;
  const int tpb = NTR / (slots * uph);
  const dim3 grid(((unsigned)a.tokens + tpb - 1) / tpb);
  auto *k = bf ? forward_kernel<bf16, UNF>(a, uph) : forward_kernel<float, UNF>(a, uph);
  return launch_pdl(k, grid, dim3(NTR), 0, st, n, uph, slots);
}

int norm_rope_bwd_ctas(int tokens, int heads, int sms) {
  return (int)std::max(2ll, std::min((long long)tokens * heads / 16 + 1, 2ll * sms));
}

cudaError_t launch_norm_rope_bwd(const NormRopeArgs &n, bool bf, bool vec, int ctas, float *dw0, float *dw1, cudaStream_t st) {
  const RopeArgs &a = n.r;
  // CTAs of either group, by their heads
  const int split = a.ngrp == 1 ? ctas : std::min(ctas - 1, std::max(1, (int)((long long)ctas * a.grp[0].heads / a.heads)));
  cudaError_t e;
  if (!vec) {
    const int smem = NTR / 32 * a.D * (int)sizeof(float);
    e = bf ? launch_pdl(norm_rope_bwd_any_kernel<bf16>, dim3(ctas), dim3(NTR), smem, st, n, split)
           : launch_pdl(norm_rope_bwd_any_kernel<float>, dim3(ctas), dim3(NTR), smem, st, n, split);
  } else {
    // heads that a token's threads begin with: what gives the longest thread the least to do, a token's angles counted as half
    // an item
    const int uph = a.D * (bf ? 2 : 4) / 32;
    int slots[2] = {1, 1};
    for (int g = 0; g < a.ngrp; ++g) {
      long long best = 0;
      for (int s = 1; s * uph <= NTB; s *= 2) {
        const long long step = (long long)(g ? ctas - split : split) * (NTB / (s * uph)), tokens = (a.tokens + step - 1) / step;
        const long long cost = tokens * (2 * ((a.grp[g].heads + s - 1) / s) + 1);
        if (!best || cost < best) {
          best = cost;
          slots[g] = s;
        }
      }
    }
    auto *k = bf ? (a.interleaved ? backward_kernel<bf16, true>(uph) : backward_kernel<bf16, false>(uph))
                 : (a.interleaved ? backward_kernel<float, true>(uph) : backward_kernel<float, false>(uph));
    const int smem = UNB * (4 + (bf ? 4 : 2)) * 16 * NTB;
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k, dim3(ctas), dim3(NTB), smem, st, n, uph, slots[0], slots[1], split);
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_rope_dw_kernel, dim3((a.D + 31) / 32, a.ngrp), dim3(1024), 0, st, (const float *)n.part, ctas, split, a.D, dw0, dw1);
}

}  // namespace gdn
