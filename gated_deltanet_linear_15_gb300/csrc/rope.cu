// Rotary positions: the feature pair (a, b) of a head at position p turns by the pair's angle,
//   (a, b) -> (a cos - b sin, b cos + a sin),
// over the first `rot` features; its gradient is the turn back.  With a paged cache, the keys and values of new
// tokens go to their slots in the same pass (softmax layers of a hybrid stack: onedev.kr summary of the FlashQLA talk,
// background paragraph).
//
// Bound by bytes: every element is read and written once, the table adds rot * 4 bytes per token for all its heads.
// A thread's unit is 32 bytes of a head as two 16-byte pieces that turn into each other: pieces i and i + rot/2 in
// the half layout, two neighbours when interleaved, so one unit holds whole pairs and every access is 16 bytes.  A thread
// keeps one unit's place in the head and one token, and walks over heads, `slots` apart: it reads the unit's cos and sin
// once for all of them, asks for the data of UN heads before it turns any, and finds the token's position and cache slot
// while the first of them are on their way.  (A line of units with one head per thread reads the table, 64 bytes for 32 of
// data, for every head: 41 us for the append of 8192 tokens of 32 + 8 + 8 heads, bf16, instead of 37.  CTAs of 128 threads,
// seven to an SM, leave a shorter last wave than three of 256: 34.6 us, 5.9 TB/s.  16384 tokens of 16 + 16 heads in fp32:
// 80.7 us, 6.7 TB/s.)
#include <math.h>

#include "rope.cuh"

namespace gdn {

// 16-byte path: D and rot multiples of two pieces' features, every pointer and stride a multiple of 16 bytes.  uph: units
// of a head; slots: heads that a token's threads begin with.
template <typename I, int UN>
__global__ void __launch_bounds__(NTR, 7) rope_kernel(RopeArgs a, int uph, int slots) {
  constexpr int V = 16 / sizeof(I);  // features of a piece
  pdl_trigger();
  pdl_wait();
  const int tpt = uph * slots, tpb = NTR / tpt;  // threads of a token, tokens of a CTA
  const int tl = threadIdx.x / tpt, in = threadIdx.x - tl * tpt, hs = in / uph, u = in - hs * uph;
  const long long t = (long long)blockIdx.x * tpb + tl;
  if (tl >= tpb || t >= a.tokens) return;
  const bool turned = u * 2 * V < a.rot, halves = turned && !a.interleaved;
  const int f0 = halves ? u * V : u * 2 * V, f1 = halves ? u * V + a.rot / 2 : u * 2 * V + V;
  const int h1 = a.grp[0].heads, h2 = h1 + (a.ngrp > 1 ? a.grp[1].heads : 0);
  TokPlace pl;
  float c[V], s[V];
  bool placed = false;
  for (int h0 = hs; h0 < a.heads; h0 += slots * UN) {
    uint4 x0[UN], x1[UN];
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      const int h = h0 + j * slots;
      if (h < a.heads) {
        const int gi = (h >= h1) + (h >= h2), hh = h - (gi == 0 ? 0 : (gi == 1 ? h1 : h2));
        const RopeGroup &g = a.grp[gi];
        const I *src = static_cast<const I *>(g.src) + t * g.s_tok + hh * g.s_head;
        x0[j] = *reinterpret_cast<const uint4 *>(src + f0);
        x1[j] = *reinterpret_cast<const uint4 *>(src + f1);
      }
    }
    if (!placed) {
      placed = true;
      pl = place_of(a, (int)t);
      if (turned && pl.pos >= 0) {  // the unit's pairs u V ..
        const float2 *cs = reinterpret_cast<const float2 *>(a.table) + (long long)pl.pos * (a.rot / 2) + u * V;
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float4 w = *reinterpret_cast<const float4 *>(cs + i);
          c[i] = w.x;
          c[i + 1] = w.z;
          s[i] = a.inverse ? -w.y : w.y;
          s[i + 1] = a.inverse ? -w.w : w.w;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      const int h = h0 + j * slots;
      if (h >= a.heads) break;
      const int gi = (h >= h1) + (h >= h2), hh = h - (gi == 0 ? 0 : (gi == 1 ? h1 : h2));
      const RopeGroup &g = a.grp[gi];
      I *dst = static_cast<I *>(g.dst) + hh * g.d_head;
      if (g.d_page) {
        if (pl.page < 0) continue;
        dst += pl.page * g.d_page + pl.off * g.d_tok;
      } else {
        dst += t * g.d_tok;
      }
      if (turned && g.turn && pl.pos >= 0) {
        float p[V], q[V];
        unpack<I>(x0[j], p);
        unpack<I>(x1[j], q);
        turn_unit<V>(p, q, c, s, a.interleaved);
        x0[j] = repack<I>(p);
        x1[j] = repack<I>(q);
      }
      *reinterpret_cast<uint4 *>(dst + f0) = x0[j];
      *reinterpret_cast<uint4 *>(dst + f1) = x1[j];
    }
  }
}

// any even rot, any D, strides and alignment: one feature pair (or, past rot, one feature) per step
template <typename I>
__global__ void __launch_bounds__(NTR) rope_any_kernel(RopeArgs a) {
  pdl_trigger();
  pdl_wait();
  const int half = a.rot / 2, per = half + a.D - a.rot;
  const long long per_tok = (long long)a.heads * per;
  for (int t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const TokPlace pl = place_of(a, t);
    for (long long in = threadIdx.x + (long long)blockIdx.y * NTR; in < per_tok; in += (long long)NTR * gridDim.y) {
      int head = (int)(in / per), gi = 0;
      const int i = (int)(in - (long long)head * per);
      while (gi < a.ngrp - 1 && head >= a.grp[gi].heads) head -= a.grp[gi++].heads;
      const RopeGroup &g = a.grp[gi];
      const I *s = static_cast<const I *>(g.src) + (long long)t * g.s_tok + head * g.s_head;
      I *d;
      if (g.d_page) {
        if (pl.page < 0) continue;
        d = static_cast<I *>(g.dst) + pl.page * g.d_page + pl.off * g.d_tok + head * g.d_head;
      } else {
        d = static_cast<I *>(g.dst) + (long long)t * g.d_tok + head * g.d_head;
      }
      if (i >= half) {
        d[i - half + a.rot] = s[i - half + a.rot];
        continue;
      }
      const int f0 = a.interleaved ? 2 * i : i, f1 = a.interleaved ? 2 * i + 1 : i + half;
      if (!g.turn || pl.pos < 0) {
        const I x = s[f0], y = s[f1];
        d[f0] = x;
        d[f1] = y;
        continue;
      }
      const float *cs = a.table + ((long long)pl.pos * half + i) * 2;
      const float c = cs[0], sn = a.inverse ? -cs[1] : cs[1];
      const float x = tof(s[f0]), y = tof(s[f1]);
      d[f0] = fromf<I>(x * c - y * sn);
      d[f1] = fromf<I>(y * c + x * sn);
    }
  }
}

__global__ void __launch_bounds__(256) rope_table_kernel(const double *freq, int pairs, long long n, double amp, float2 *out) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  double s, c;
  sincos((double)(i / pairs) * freq[i % pairs], &s, &c);
  out[i] = make_float2((float)(amp * c), (float)(amp * s));
}

cudaError_t launch_rope_table(const double *freq, int pairs, int rows, double amp, float *table, cudaStream_t st) {
  const long long n = (long long)rows * pairs;
  rope_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(freq, pairs, n, amp, reinterpret_cast<float2 *>(table));
  return cudaGetLastError();
}

cudaError_t launch_rope(const RopeArgs &a, bool bf, bool vec, cudaStream_t st) {
  if (!vec) {
    const long long per_tok = (long long)a.heads * (a.D - a.rot / 2);
    const dim3 grid((unsigned)(a.tokens < 65535 ? a.tokens : 65535), (unsigned)(per_tok > 4 * NTR ? 4 : 1));
    return bf ? launch_pdl(rope_any_kernel<bf16>, grid, dim3(NTR), 0, st, a)
              : launch_pdl(rope_any_kernel<float>, grid, dim3(NTR), 0, st, a);
  }
  // 64 threads a token (each walks over a few heads), more while that leaves SMs without work
  const int uph = a.D * (bf ? 2 : 4) / 32;
  int slots = 64 / uph > 0 ? 64 / uph : 1;
  while (slots < a.heads && 2 * slots * uph <= NTR && (long long)a.tokens * slots * uph < 152ll * 4 * NTR) slots *= 2;
  const int tpb = NTR / (slots * uph);
  const dim3 grid(((unsigned)a.tokens + tpb - 1) / tpb);
  return bf ? launch_pdl(rope_kernel<bf16, 3>, grid, dim3(NTR), 0, st, a, uph, slots)
            : launch_pdl(rope_kernel<float, 2>, grid, dim3(NTR), 0, st, a, uph, slots);
}

}  // namespace gdn
