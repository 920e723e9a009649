// What the kernels of rotary positions share: where a token goes, and 16-byte pieces as fp32 values.
#pragma once
#include "block.h"
#include "common.cuh"

namespace gdn {

namespace {

constexpr int NTR = ROPE_THREADS;

// position and cache slot of a token: slot -1 when it has none, position -1 when it is outside the table
struct TokPlace {
  int pos;
  int page, off;
};
__device__ __forceinline__ TokPlace place_of(const RopeArgs &a, int t) {
  TokPlace p;
  p.page = -1;
  p.off = 0;
  if (a.positions) {
    p.pos = a.positions[t];
  } else {
    int n, last;
    if (a.cu_q) {  // the last sequence that begins at or before t (empty ones share their begin with the next)
      int lo = 0, hi = a.N;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_q[mid] <= t) lo = mid;
        else hi = mid;
      }
      n = lo;
      last = a.cu_q[n + 1];
      if (t < a.cu_q[n] || t >= last) {
        p.pos = -1;
        return p;
      }
    } else {
      n = t / a.per_seq;
      last = (n + 1) * a.per_seq;
    }
    p.pos = a.kv_lens[n] - last + t;
    if (p.pos >= 0 && (p.pos >> a.log2P) < a.max_pages) {
      const int pg = a.pages[n * a.table_stride + (p.pos >> a.log2P)];
      if ((unsigned)pg < (unsigned)a.num_pages) {
        p.page = pg;
        p.off = p.pos & ((1 << a.log2P) - 1);
      }
    }
  }
  if (p.pos < 0 || p.pos >= a.rows) p.pos = -1;
  return p;
}

template <typename I> __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[16 / sizeof(I)]);
template <> __device__ __forceinline__ void unpack<bf16>(const uint4 &u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <> __device__ __forceinline__ void unpack<float>(const uint4 &u, float (&x)[4]) {
  x[0] = __uint_as_float(u.x);
  x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z);
  x[3] = __uint_as_float(u.w);
}
template <typename I> __device__ __forceinline__ uint4 repack(const float (&x)[16 / sizeof(I)]);
template <> __device__ __forceinline__ uint4 repack<bf16>(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ uint4 repack<float>(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// a unit's pairs turn by the angles (c, s): the unit holds pieces p and q of V features, whose pairs are (p[i], q[i]), or
// neighbours when interleaved
template <int V>
__device__ __forceinline__ void turn_unit(float (&p)[V], float (&q)[V], const float (&c)[V], const float (&s)[V], bool interleaved) {
  if (interleaved) {  // the unit's 2 V features are pairs 0 .. V - 1
    float y[2 * V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float u0 = 2 * i < V ? p[(2 * i) % V] : q[(2 * i) % V], u1 = 2 * i < V ? p[(2 * i + 1) % V] : q[(2 * i + 1) % V];
      y[2 * i] = u0 * c[i] - u1 * s[i];
      y[2 * i + 1] = u1 * c[i] + u0 * s[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = y[i];
      q[i] = y[V + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float u0 = p[i], u1 = q[i];
      p[i] = u0 * c[i] - u1 * s[i];
      q[i] = u1 * c[i] + u0 * s[i];
    }
  }
}

}  // namespace

}  // namespace gdn
