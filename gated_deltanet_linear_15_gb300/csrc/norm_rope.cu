// Root-mean-square norm of each head of q and k, and its turn to the token's position, in one pass:
//   r = (mean(x^2) + eps)^(-1/2),  y = R(p) (r x (w + off)),
// R(p) the turn of the feature pairs by position p (rope.cu).  Backward, with u = R(p)^T dy and xhat = r x:
//   dx = r (u (w + off) - xhat mean(u (w + off) xhat)),  dw = sum over tokens and heads of u xhat.
// With a paged cache the keys and values of new tokens go to their slots in the same pass.
//
// Bound by bytes: every element is read once and written once (backward: x and dy read, dx written).  A thread's unit is
// that of rope.cu, 32 bytes of a head that hold whole pairs; the D sizeof(I) / 32 threads of a head are neighbours in a
// warp, so a head's sums take a few shuffles, and the data stay in registers between the sum and the turn.  Weights come
// from shared memory: in registers, those of q and k take 32 and cost a third of the loads in flight.
//
// The backward's CTAs stay and walk over tokens, some of them over the heads of q and the others over those of k, since a
// thread's place in the head does not change: it keeps its sums of dw in registers.  Each CTA leaves one partial row, and a
// second kernel adds these in order.
//
// Heads whose size, strides or alignment do not allow 16-byte units: a warp to a head.
#include <algorithm>

#include "rope.cuh"

namespace gdn {

namespace {

constexpr int NTB = 256, MAXD = NORM_ROPE_MAX_DIM;  // threads of the backward, features of a head

// sum over the `n` neighbouring lanes (a power of two) that hold a head
__device__ __forceinline__ float head_sum(float x, int n) {
  const unsigned mask = n == 32 ? 0xffffffffu : ((1u << n) - 1) << (threadIdx.x & 31 & ~(n - 1));
  for (int o = n >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
  return x;
}
template <int V> __device__ __forceinline__ void read_weights(const float *w, int f0, int f1, float (&p)[V], float (&q)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const float4 a = *reinterpret_cast<const float4 *>(w + f0 + i), b = *reinterpret_cast<const float4 *>(w + f1 + i);
    p[i] = a.x; p[i + 1] = a.y; p[i + 2] = a.z; p[i + 3] = a.w;
    q[i] = b.x; q[i + 1] = b.y; q[i + 2] = b.z; q[i + 3] = b.w;
  }
}
// the angles of the unit's pairs u V .. at position pos
template <int V> __device__ __forceinline__ void read_angles(const RopeArgs &a, int pos, int u, float (&c)[V], float (&s)[V]) {
  const float2 *cs = reinterpret_cast<const float2 *>(a.table) + (long long)pos * (a.rot / 2) + u * V;
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    const float4 w = *reinterpret_cast<const float4 *>(cs + i);
    c[i] = w.x;
    c[i + 1] = w.z;
    s[i] = a.inverse ? -w.y : w.y;
    s[i + 1] = a.inverse ? -w.w : w.w;
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

template <typename I, int UN>
__global__ void __launch_bounds__(NTR, 6) norm_rope_kernel(NormRopeArgs n, int uph, int slots) {
  constexpr int V = 16 / sizeof(I);
  const RopeArgs &a = n.r;
  __shared__ __align__(16) float w[2][MAXD];
  pdl_trigger();
  pdl_wait();
  for (int i = threadIdx.x; i < 2 * a.D; i += NTR) {
    const int g = i >= a.D, f = i - g * a.D;
    w[g][f] = n.w[g] ? n.w[g][f] + n.off : 0.f;
  }
  __syncthreads();
  const int tpt = uph * slots, tpb = NTR / tpt;
  const int tl = threadIdx.x / tpt, in = threadIdx.x - tl * tpt, hs = in / uph, u = in - hs * uph;
  const long long t = (long long)blockIdx.x * tpb + tl;
  if (tl >= tpb || t >= a.tokens) return;
  const bool turned = u * 2 * V < a.rot, halves = turned && !a.interleaved;
  const int f0 = halves ? u * V : u * 2 * V, f1 = halves ? u * V + a.rot / 2 : u * 2 * V + V;
  TokPlace pl;
  float c[V], s[V];
  bool placed = false;
  for (int h0 = hs; h0 < a.heads; h0 += slots * UN) {
    uint4 x0[UN], x1[UN];
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      const int h = h0 + j * slots;
      if (h < a.heads) {
        const HeadOf ho = head_of(a, h);
        const RopeGroup &g = a.grp[ho.group];
        const I *src = static_cast<const I *>(g.src) + t * g.s_tok + ho.head * g.s_head;
        x0[j] = *reinterpret_cast<const uint4 *>(src + f0);
        x1[j] = *reinterpret_cast<const uint4 *>(src + f1);
      }
    }
    if (!placed) {
      placed = true;
      pl = place_of(a, (int)t);
      if (turned && pl.pos >= 0) read_angles<V>(a, pl.pos, u, c, s);
    }
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      const int h = h0 + j * slots;
      if (h >= a.heads) break;
      const HeadOf ho = head_of(a, h);
      const RopeGroup &g = a.grp[ho.group];
      if (g.turn) {  // not a value head
        float p[V], q[V], wp[V], wq[V];
        unpack<I>(x0[j], p);
        unpack<I>(x1[j], q);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum += p[i] * p[i] + q[i] * q[i];
        const float r = rsqrtf(head_sum(sum, uph) / (float)a.D + n.eps);
        read_weights<V>(w[ho.group], f0, f1, wp, wq);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          p[i] *= r * wp[i];
          q[i] *= r * wq[i];
        }
        if (turned && pl.pos >= 0) turn_unit<V>(p, q, c, s, a.interleaved);
        x0[j] = repack<I>(p);
        x1[j] = repack<I>(q);
      }
      I *dst = static_cast<I *>(g.dst) + ho.head * g.d_head;
      if (g.d_page) {
        if (pl.page < 0) continue;
        dst += pl.page * g.d_page + pl.off * g.d_tok;
      } else {
        dst += t * g.d_tok;
      }
      *reinterpret_cast<uint4 *>(dst + f0) = x0[j];
      *reinterpret_cast<uint4 *>(dst + f1) = x1[j];
    }
  }
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
// of group 1.  part: [gridDim.x][D].  A thread's items are its heads of one token after another; the next item's data, and
// the next token's angles where it begins one, are asked for before the current item is worked on.
template <typename I>
__global__ void __launch_bounds__(NTB, 2) norm_rope_bwd_kernel(NormRopeArgs n, int uph, int slots, int split) {
  constexpr int V = 16 / sizeof(I);
  const RopeArgs &a = n.r;
  __shared__ __align__(16) float w[MAXD];
  __shared__ float sums[NTB][2 * V + 1];
  const int gi = (int)blockIdx.x >= split, cta = blockIdx.x - (gi ? split : 0), ctas = gi ? gridDim.x - split : split;
  const RopeGroup g = a.grp[gi];
  pdl_trigger();
  pdl_wait();
  for (int f = threadIdx.x; f < a.D; f += NTB) w[f] = n.w[gi][f] + n.off;
  __syncthreads();
  const int tpt = uph * slots, tpb = NTB / tpt;
  const int tl = threadIdx.x / tpt, in = threadIdx.x - tl * tpt, hs = in / uph, u = in - hs * uph;
  const bool turned = u * 2 * V < a.rot, halves = turned && !a.interleaved;
  const int f0 = halves ? u * V : u * 2 * V, f1 = halves ? u * V + a.rot / 2 : u * 2 * V + V;
  const int step = ctas * tpb;
  float dw[2 * V] = {};
  struct Item {
    uint4 x0, x1, d0, d1;
  };
  auto read = [&](long long t, int h) {
    Item i;
    const I *src = static_cast<const I *>(g.src) + t * g.s_tok + h * g.s_head + f0;
    const I *dy = static_cast<const I *>(n.dy[gi]) + t * n.dy_tok[gi] + h * n.dy_head[gi] + f0;
    i.x0 = *reinterpret_cast<const uint4 *>(src);
    i.x1 = *reinterpret_cast<const uint4 *>(src + f1 - f0);
    i.d0 = *reinterpret_cast<const uint4 *>(dy);
    i.d1 = *reinterpret_cast<const uint4 *>(dy + f1 - f0);
    return i;
  };
  // of a token: its position, -1 where it does not turn
  auto position = [&](long long t) {
    const int pos = t < a.tokens ? a.positions[t] : -1;
    return turned && pos >= 0 && pos < a.rows ? pos : -1;
  };
  long long t = (long long)cta * tpb + tl;
  int h = hs;
  if (tl < tpb && t < a.tokens && h < g.heads) {
    Item now = read(t, h);
    int pos = position(t), pos1 = position(t + step);
    float c[V], s[V];
    if (pos >= 0) read_angles<V>(a, pos, u, c, s);  // a.inverse is set
    for (;;) {
      long long t1 = t;
      int h1 = h + slots;
      if (h1 >= g.heads) {
        h1 = hs;
        t1 += step;
      }
      const bool more = t1 < a.tokens;
      Item next = {};
      float c1[V], s1[V];
      if (more) {
        next = read(t1, h1);
        if (t1 != t && pos1 >= 0) read_angles<V>(a, pos1, u, c1, s1);
      }
      float p[V], q[V], y[V], z[V], wp[V], wq[V];
      unpack<I>(now.x0, p);
      unpack<I>(now.x1, q);
      unpack<I>(now.d0, y);
      unpack<I>(now.d1, z);
      if (pos >= 0) turn_unit<V>(y, z, c, s, a.interleaved);
      read_weights<V>(w, f0, f1, wp, wq);
      float sum = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sum += p[i] * p[i] + q[i] * q[i];
        dot += p[i] * (y[i] * wp[i]) + q[i] * (z[i] * wq[i]);
      }
      sum = head_sum(sum, uph);
      dot = head_sum(dot, uph);
      const float r = rsqrtf(sum / (float)a.D + n.eps), m = r * r * (dot / (float)a.D);  // xhat mean(..) = x m
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dw[i] += y[i] * (p[i] * r);
        dw[V + i] += z[i] * (q[i] * r);
        p[i] = r * (y[i] * wp[i] - p[i] * m);
        q[i] = r * (z[i] * wq[i] - q[i] * m);
      }
      I *dst = static_cast<I *>(g.dst) + t * g.d_tok + h * g.d_head + f0;
      *reinterpret_cast<uint4 *>(dst) = repack<I>(p);
      *reinterpret_cast<uint4 *>(dst + f1 - f0) = repack<I>(q);
      if (!more) break;
      if (t1 != t) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          c[i] = c1[i];
          s[i] = s1[i];
        }
        pos = pos1;
        pos1 = position(t1 + step);
      }
      t = t1;
      h = h1;
      now = next;
    }
  }
  // the threads of one place in the head, in order
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) sums[threadIdx.x][i] = dw[i];
  __syncthreads();
  for (int f = threadIdx.x; f < a.D; f += NTB) {
    const int fu = f / (2 * V), i = f - fu * 2 * V;
    float z = 0.f;
    for (int k = fu; k < tpb * tpt; k += uph) z += sums[k][i];
    const bool fh = fu * 2 * V < a.rot && !a.interleaved;
    const int at = fh ? (i < V ? fu * V + i : fu * V + a.rot / 2 + i - V) : f;
    n.part[(long long)blockIdx.x * a.D + at] = z;
  }
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
    const float r = rsqrtf(sum / (float)a.D + n.eps), m = r * r * (dot / (float)a.D);
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
  return bf ? launch_pdl(norm_rope_kernel<bf16, 3>, grid, dim3(NTR), 0, st, n, uph, slots)
            : launch_pdl(norm_rope_kernel<float, 2>, grid, dim3(NTR), 0, st, n, uph, slots);
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
    // heads that a token's threads begin with: what gives the longest thread the fewest items, the fewest heads among equals
    // (angles are read once for all heads of a thread)
    const int uph = a.D * (bf ? 2 : 4) / 32;
    int slots = 1;
    long long best = 0;
    for (int s = 1; s * uph <= NTB; s *= 2) {
      const int tpb = NTB / (s * uph);
      long long items = 0;
      for (int g = 0; g < a.ngrp; ++g) {
        const long long step = (long long)(a.ngrp == 1 ? ctas : (g ? ctas - split : split)) * tpb;
        items = std::max(items, (a.tokens + step - 1) / step * ((a.grp[g].heads + s - 1) / s));
      }
      if (!best || items < best) {
        best = items;
        slots = s;
      }
    }
    e = bf ? launch_pdl(norm_rope_bwd_kernel<bf16>, dim3(ctas), dim3(NTB), 0, st, n, uph, slots, split)
           : launch_pdl(norm_rope_bwd_kernel<float>, dim3(ctas), dim3(NTB), 0, st, n, uph, slots, split);
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_rope_dw_kernel, dim3((a.D + 31) / 32, a.ngrp), dim3(1024), 0, st, (const float *)n.part, ctas, split, a.D, dw0, dw1);
}

}  // namespace gdn
