// Root-mean-square norm of the residual stream, forward and backward:
//   h = x + residual,  rstd = (mean(h^2) + eps)^(-1/2),  y = h rstd w,
//   fp8: per row or per 128 features  scale = amax |y| / 448,  y8 = e4m3(y * (448 / amax |y|));
//   dx = rstd w dy - h rstd^3 <w dy, h> / D + dh,  dw = sum over rows of dy h rstd.
// (The norm in front of the projections of every layer of the stacks that onedev.kr's summary of the FlashQLA talk
// describes, background paragraph.)
//
// Bound by bytes: a row is read once into registers (16-byte pieces, neighbours in neighbouring threads), reduced, and
// written once; the fp8 scales come from the same registers.  TPR threads hold a row, two pieces each where that works
// out, so that a CTA of 256 threads works on several short rows at once; rows of at most 32 pieces need no barrier at all.
// CTAs stay and walk over rows, with the weight in registers, and ask for the next row before they reduce the one they
// have.  The backward keeps its share of dw in registers too; each CTA leaves one partial row, and a second kernel adds
// these in order.  8192 rows of 4096 to fp8: 37.6 us, 6.3 TB/s; 64 rows: 2.6 us on the GPU; backward of 16384 rows of 2048:
// 48.3 us, 5.5 TB/s, 45 us of it the first kernel.  fp8 multiplies by the reciprocal scale: two roundings of 2^-24 against
// the definition, as the scale and a division by it have, which takes the 8192 rows from 37.4 to 46.0 us.  Sums are fp32;
// rows of which dim, stride or alignment does not allow 16-byte pieces go one feature at a time.
#include <cuda_fp8.h>

#include <algorithm>

#include "block.h"
#include "common.cuh"

namespace gdn {

namespace {

constexpr float E4M3_MAX = 448.f, AMAX_FLOOR = 1e-30f;

template <typename I> struct Vec { static constexpr int N = 16 / sizeof(I); };
template <typename I> __device__ __forceinline__ void widen(const uint4 &u, float *x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(I) == 2) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      x[i] = __uint_as_float(w[i]);
    }
  }
}
template <typename I> __device__ __forceinline__ uint4 narrow(const float *x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(I) == 2) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    } else {
      w[i] = __float_as_uint(x[i]);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint32_t fp8x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
__device__ __forceinline__ uint8_t fp8x1(float a) { return __nv_cvt_float_to_fp8(a, __NV_SATFINITE, __NV_E4M3); }

// reduction over the TPR threads of a row; sh: this row group's 2 x (TPR / 32) floats, halves used in turn so that
// one barrier per reduction is enough.  Every thread of the CTA takes part.
template <int TPR, bool MAX> __device__ __forceinline__ float row_reduce(float x, float *sh, int &turn) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, x, o);
    x = MAX ? fmaxf(x, y) : x + y;
  }
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    float *b = sh + turn * W;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) b[(threadIdx.x % TPR) >> 5] = x;
    __syncthreads();
    x = b[0];
#pragma unroll
    for (int i = 1; i < W; ++i) x = MAX ? fmaxf(x, b[i]) : x + b[i];
  }
  return x;
}

}  // namespace

template <typename I, int NTH, int TPR, int NV>
__global__ void __launch_bounds__(NTH) norm_fwd_kernel(NormArgs a) {
  constexpr int V = Vec<I>::N, RPC = NTH / TPR;
  constexpr bool AHEAD = NV <= 2;  // registers for the next row
  __shared__ float sh[RPC][TPR > 32 ? 2 * (TPR / 32) : 1];
  pdl_trigger();
  pdl_wait();
  const int tr = threadIdx.x % TPR, grp = threadIdx.x / TPR, pieces = a.D / V;
  int turn = 0;
  float w[NV][V];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = tr + k * TPR;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 t = c < pieces ? *reinterpret_cast<const float4 *>(a.weight + c * V + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      w[k][i] = t.x + a.off;
      w[k][i + 1] = t.y + a.off;
      w[k][i + 2] = t.z + a.off;
      w[k][i + 3] = t.w + a.off;
    }
  }
  const float invD = 1.f / a.D;
  const long long step = (long long)gridDim.x * RPC;
  uint4 xr[NV], rr[NV];  // the row that comes next
  auto load = [&](long long r) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = tr + k * TPR;
      xr[k] = rr[k] = make_uint4(0, 0, 0, 0);
      if (r < a.T && c < pieces) {
        xr[k] = *reinterpret_cast<const uint4 *>(static_cast<const I *>(a.x) + r * a.x_row + c * V);
        if (a.res) rr[k] = *reinterpret_cast<const uint4 *>(static_cast<const I *>(a.res) + r * a.r_row + c * V);
      }
    }
  };
  long long r = (long long)blockIdx.x * RPC + grp;
  if (AHEAD) load(r);
  for (long long r0 = (long long)blockIdx.x * RPC; r0 < a.T; r0 += step, r += step) {
    const bool live = r < a.T;
    if (!AHEAD) load(r);
    float h[NV][V];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float t[V];
      widen<I>(xr[k], h[k]);
      widen<I>(rr[k], t);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (a.res) h[k][i] += t[i];
        ss += h[k][i] * h[k][i];
      }
    }
    if (AHEAD) load(r + step);
    if (a.h_out) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = tr + k * TPR;
        if (live && c < pieces) *reinterpret_cast<uint4 *>(static_cast<I *>(a.h_out) + r * a.h_row + c * V) = narrow<I>(h[k]);
      }
    }
    const float rstd = rsqrtf(row_reduce<TPR, false>(ss, sh[grp], turn) * invD + a.eps);
    if (a.rstd && live && tr == 0) a.rstd[r] = rstd;
    if (!a.fp8) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = tr + k * TPR;
#pragma unroll
        for (int i = 0; i < V; ++i) h[k][i] = h[k][i] * rstd * w[k][i];
        if (live && c < pieces) *reinterpret_cast<uint4 *>(static_cast<I *>(a.y) + r * a.y_row + c * V) = narrow<I>(h[k]);
      }
      continue;
    }
    float amax = 0.f, gm[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      gm[k] = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        h[k][i] = h[k][i] * rstd * w[k][i];
        gm[k] = fmaxf(gm[k], fabsf(h[k][i]));
      }
      amax = fmaxf(amax, gm[k]);
    }
    if (a.group == 0) {
      amax = row_reduce<TPR, true>(amax, sh[grp], turn);
      if (live && tr == 0) a.scale[r] = fmaxf(amax, AMAX_FLOOR) / E4M3_MAX;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = tr + k * TPR;
      float m = amax;
      if (a.group) {  // 128 features: 16 (bf16) or 32 (fp32) neighbouring threads
        m = gm[k];
#pragma unroll
        for (int o = 64 / V; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (live && c < pieces && c % (128 / V) == 0) a.scale[r * (a.D / 128) + c / (128 / V)] = fmaxf(m, AMAX_FLOOR) / E4M3_MAX;
      }
      const float inv = E4M3_MAX / fmaxf(m, AMAX_FLOOR);
      if (live && c < pieces) {
        uint8_t *y = static_cast<uint8_t *>(a.y) + r * a.y_row + c * V;
        const uint32_t lo = fp8x4(h[k][0] * inv, h[k][1] * inv, h[k][2] * inv, h[k][3] * inv);
        if constexpr (V == 8) {
          *reinterpret_cast<uint2 *>(y) = make_uint2(lo, fp8x4(h[k][4] * inv, h[k][5] * inv, h[k][6] * inv, h[k][7] * inv));
        } else {
          *reinterpret_cast<uint32_t *>(y) = lo;
        }
      }
    }
  }
}

// one feature at a time, a CTA per row
template <typename I> __global__ void __launch_bounds__(256) norm_fwd_any_kernel(NormArgs a) {
  __shared__ float sh[2 * 8];
  pdl_trigger();
  pdl_wait();
  int turn = 0;
  for (long long r = blockIdx.x; r < a.T; r += gridDim.x) {
    const I *x = static_cast<const I *>(a.x) + r * a.x_row;
    const I *q = a.res ? static_cast<const I *>(a.res) + r * a.r_row : nullptr;
    float ss = 0.f;
    for (int i = threadIdx.x; i < a.D; i += 256) {
      const float h = tof(x[i]) + (q ? tof(q[i]) : 0.f);
      ss += h * h;
    }
    const float rstd = rsqrtf(row_reduce<256, false>(ss, sh, turn) / a.D + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
    auto y_at = [&](int i) { return (tof(x[i]) + (q ? tof(q[i]) : 0.f)) * rstd * (a.weight[i] + a.off); };
    const int gsz = a.group ? a.group : a.D;
    float inv = 0.f;
    for (int g0 = 0; a.fp8 && g0 < a.D; g0 += gsz) {
      float m = 0.f;
      for (int i = g0 + threadIdx.x; i < g0 + gsz; i += 256) m = fmaxf(m, fabsf(y_at(i)));
      m = fmaxf(row_reduce<256, true>(m, sh, turn), AMAX_FLOOR);
      if (threadIdx.x == 0) a.scale[r * (a.D / gsz) + g0 / gsz] = m / E4M3_MAX;
      inv = E4M3_MAX / m;
      if (a.group)
        for (int i = g0 + threadIdx.x; i < g0 + gsz; i += 256) static_cast<uint8_t *>(a.y)[r * a.y_row + i] = fp8x1(y_at(i) * inv);
    }
    // h_out may take an input's place: without groups a feature is read and written by one thread, but the last group's
    // reads are those of other threads
    if (a.group && a.h_out) __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += 256) {
      const float h = tof(x[i]) + (q ? tof(q[i]) : 0.f), y = h * rstd * (a.weight[i] + a.off);
      if (a.h_out) static_cast<I *>(a.h_out)[r * a.h_row + i] = fromf<I>(h);
      if (!a.fp8) static_cast<I *>(a.y)[r * a.y_row + i] = fromf<I>(y);
      else if (!a.group) static_cast<uint8_t *>(a.y)[r * a.y_row + i] = fp8x1(y * inv);
    }
  }
}

template <typename I, int NTH, int TPR, int NV>
__global__ void __launch_bounds__(NTH) norm_bwd_kernel(NormArgs a) {
  constexpr int V = Vec<I>::N, RPC = NTH / TPR;
  constexpr bool AHEAD = TPR <= 256;  // registers for the next row; with 512 threads a row two CTAs per SM do better without
  __shared__ float sh[RPC][TPR > 32 ? 2 * (TPR / 32) : 1];
  extern __shared__ float dsh[];  // [D], when several row groups share a CTA
  pdl_trigger();
  pdl_wait();
  const int tr = threadIdx.x % TPR, grp = threadIdx.x / TPR, pieces = a.D / V;
  int turn = 0;
  float w[NV][V], dw[NV][V];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = tr + k * TPR;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[k][i] = c < pieces ? a.weight[c * V + i] + a.off : 0.f;
      dw[k][i] = 0.f;
    }
  }
  const float invD = 1.f / a.D;
  const long long step = (long long)gridDim.x * RPC;
  uint4 hn[NV], gn[NV], en[NV];  // the row that comes next
  float rn = 0.f;
  auto load = [&](long long r) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = tr + k * TPR;
      hn[k] = gn[k] = en[k] = make_uint4(0, 0, 0, 0);
      if (r < a.T && c < pieces) {
        hn[k] = *reinterpret_cast<const uint4 *>(static_cast<const I *>(a.h) + r * a.x_row + c * V);
        gn[k] = *reinterpret_cast<const uint4 *>(static_cast<const I *>(a.x) + r * a.y_row + c * V);
        if (a.res) en[k] = *reinterpret_cast<const uint4 *>(static_cast<const I *>(a.res) + r * a.r_row + c * V);
      }
    }
    rn = r < a.T ? a.rstd_in[r] : 0.f;
  };
  long long r = (long long)blockIdx.x * RPC + grp;
  if (AHEAD) load(r);
  for (long long r0 = (long long)blockIdx.x * RPC; r0 < a.T; r0 += step, r += step) {
    const bool live = r < a.T;
    if (!AHEAD) load(r);
    uint4 hr[NV], gr[NV], er[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      hr[k] = hn[k];
      gr[k] = gn[k];
      er[k] = en[k];
    }
    const float rstd = rn;
    if (AHEAD) load(r + step);
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float h[V], g[V];
      widen<I>(hr[k], h);
      widen<I>(gr[k], g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dot += g[i] * w[k][i] * h[i];
        dw[k][i] += g[i] * (h[i] * rstd);
      }
    }
    const float s = row_reduce<TPR, false>(dot, sh[grp], turn) * invD * rstd * rstd * rstd;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = tr + k * TPR;
      float h[V], g[V], e[V];
      widen<I>(hr[k], h);
      widen<I>(gr[k], g);
      widen<I>(er[k], e);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = rstd * w[k][i] * g[i] - s * h[i];
        e[i] = a.res ? d + e[i] : d;
      }
      if (live && c < pieces) *reinterpret_cast<uint4 *>(static_cast<I *>(a.y) + r * a.h_row + c * V) = narrow<I>(e);
    }
  }
  // this CTA's share of dw: the row groups one after another, then to its row of the partials
  if constexpr (RPC > 1) {
    for (int x = 0; x < RPC; ++x) {
      if (grp == x) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int c = tr + k * TPR;
          if (c < pieces) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
              if (x == 0) dsh[c * V + i] = dw[k][i];
              else dsh[c * V + i] += dw[k][i];
            }
          }
        }
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < a.D; i += NTH) a.part[(long long)blockIdx.x * a.D + i] = dsh[i];
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = tr + k * TPR;
      if (c < pieces) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
          *reinterpret_cast<float4 *>(a.part + (long long)blockIdx.x * a.D + c * V + i) =
              make_float4(dw[k][i], dw[k][i + 1], dw[k][i + 2], dw[k][i + 3]);
      }
    }
  }
}

template <typename I> __global__ void __launch_bounds__(256) norm_bwd_any_kernel(NormArgs a) {
  __shared__ float sh[2 * 8];
  pdl_trigger();
  pdl_wait();
  int turn = 0;
  float *part = a.part + (long long)blockIdx.x * a.D;  // thread t owns columns t, t + 256, ...
  for (int i = threadIdx.x; i < a.D; i += 256) part[i] = 0.f;
  for (long long r = blockIdx.x; r < a.T; r += gridDim.x) {
    const I *g = static_cast<const I *>(a.x) + r * a.y_row, *h = static_cast<const I *>(a.h) + r * a.x_row;
    const I *e = a.res ? static_cast<const I *>(a.res) + r * a.r_row : nullptr;
    const float rstd = a.rstd_in[r];
    float dot = 0.f;
    for (int i = threadIdx.x; i < a.D; i += 256) dot += tof(g[i]) * (a.weight[i] + a.off) * tof(h[i]);
    const float s = row_reduce<256, false>(dot, sh, turn) / a.D * rstd * rstd * rstd;
    for (int i = threadIdx.x; i < a.D; i += 256) {
      const float gi = tof(g[i]), hi = tof(h[i]);
      part[i] += gi * (hi * rstd);
      const float d = rstd * (a.weight[i] + a.off) * gi - s * hi;
      static_cast<I *>(a.y)[r * a.h_row + i] = fromf<I>(e ? d + tof(e[i]) : d);
    }
  }
}

// dw = the partial rows, added in order: 32 warps take every 32nd row of 32 columns, then join
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *part, int rows, int D, float *dw) {
  __shared__ float sh[32][33];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < D) {
#pragma unroll 10
    for (int r = y; r < rows; r += 32) s += part[(long long)r * D + c];
  }
  sh[y][lane] = s;
  __syncthreads();
  s = sh[lane][y];  // column y of the 32, its 32 partial sums over the lanes
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && blockIdx.x * 32 + y < D) dw[blockIdx.x * 32 + y] = s;
}

namespace {

template <typename I, int NTH, int TPR, int NV> cudaError_t fwd(const NormArgs &a, int sms, cudaStream_t st) {
  static const int per_sm = [] {  // resident CTAs of this kernel, the same on every GB300
    int n = 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, norm_fwd_kernel<I, NTH, TPR, NV>, NTH, 0) == cudaSuccess && n > 0 ? n : 1;
  }();
  const long long want = (a.T + NTH / TPR - 1) / (NTH / TPR), cap = (long long)sms * per_sm;
  return launch_pdl(norm_fwd_kernel<I, NTH, TPR, NV>, dim3((unsigned)(want < cap ? want : cap)), dim3(NTH), 0, st, a);
}
// Threads of a row and pieces of each: two pieces, up to 512 threads, then four; one piece each where a row needs no
// second, or where there are fewer rows than SMs and a call is as long as its slowest row.
struct RowShape {
  int tpr, nv;  // tpr 0: the row does not fit
};
RowShape row_shape(const NormArgs &a, int V, int sms) {
  const int p = a.D / V;
  if (p <= 16) return {16, 1};
  if (p <= 32) return {32, 1};
  if (a.T < sms && p > 128 && p <= 512) return {512, 1};
  for (int t = 32; t <= 512; t *= 2)
    if (p <= 2 * t) return {t, 2};
  return p <= 512 * 4 ? RowShape{512, 4} : RowShape{0, 0};
}
template <typename I> cudaError_t fwd_shape(const NormArgs &a, int sms, cudaStream_t st) {
  const RowShape s = row_shape(a, Vec<I>::N, sms);
  switch (s.tpr * 8 + s.nv) {
    case 16 * 8 + 1: return fwd<I, 256, 16, 1>(a, sms, st);
    case 32 * 8 + 1: return fwd<I, 256, 32, 1>(a, sms, st);
    case 32 * 8 + 2: return fwd<I, 256, 32, 2>(a, sms, st);
    case 64 * 8 + 2: return fwd<I, 256, 64, 2>(a, sms, st);
    case 128 * 8 + 2: return fwd<I, 256, 128, 2>(a, sms, st);
    case 256 * 8 + 2: return fwd<I, 256, 256, 2>(a, sms, st);
    case 512 * 8 + 1: return fwd<I, 512, 512, 1>(a, sms, st);
    case 512 * 8 + 2: return fwd<I, 512, 512, 2>(a, sms, st);
    case 512 * 8 + 4: return fwd<I, 512, 512, 4>(a, sms, st);
  }
  return cudaErrorInvalidValue;
}

template <typename I, int NTH, int TPR, int NV> cudaError_t bwd(const NormArgs &a, int ctas, cudaStream_t st) {
  const size_t smem = NTH > TPR ? (size_t)a.D * 4 : 0;
  return launch_pdl(norm_bwd_kernel<I, NTH, TPR, NV>, dim3(ctas), dim3(NTH), smem, st, a);
}
template <typename I> cudaError_t bwd_shape(const NormArgs &a, int sms, int ctas, cudaStream_t st) {
  const RowShape s = row_shape(a, Vec<I>::N, sms);
  switch (s.tpr * 8 + s.nv) {
    case 16 * 8 + 1: return bwd<I, 256, 16, 1>(a, ctas, st);
    case 32 * 8 + 1: return bwd<I, 256, 32, 1>(a, ctas, st);
    case 32 * 8 + 2: return bwd<I, 256, 32, 2>(a, ctas, st);
    case 64 * 8 + 2: return bwd<I, 256, 64, 2>(a, ctas, st);
    case 128 * 8 + 2: return bwd<I, 256, 128, 2>(a, ctas, st);
    case 256 * 8 + 2: return bwd<I, 256, 256, 2>(a, ctas, st);
    case 512 * 8 + 1: return bwd<I, 512, 512, 1>(a, ctas, st);
    case 512 * 8 + 2: return bwd<I, 512, 512, 2>(a, ctas, st);
    case 512 * 8 + 4: return bwd<I, 512, 512, 4>(a, ctas, st);
  }
  return cudaErrorInvalidValue;
}

bool in_registers(const NormArgs &a, bool bf, bool vec, int sms) { return vec && row_shape(a, bf ? 8 : 4, sms).tpr > 0; }

}  // namespace

// CTAs of the backward: what the registers of a thread let an SM hold, three with one piece per thread, two otherwise
int norm_bwd_ctas(const NormArgs &a, bool bf, bool vec, int sms) {
  const long long cap = (long long)sms * (row_shape(a, bf ? 8 : 4, sms).nv == 1 ? 3 : 2);
  long long rows = 1;
  if (in_registers(a, bf, vec, sms)) rows = std::max(1, 256 / row_shape(a, bf ? 8 : 4, sms).tpr);
  const long long want = (a.T + rows - 1) / rows;
  return (int)(want < cap ? (want > 0 ? want : 1) : cap);
}

cudaError_t launch_norm_fwd(const NormArgs &a, bool bf, bool vec, int sms, cudaStream_t st) {
  if (in_registers(a, bf, vec, sms)) return bf ? fwd_shape<bf16>(a, sms, st) : fwd_shape<float>(a, sms, st);
  const unsigned grid = (unsigned)(a.T < 8ll * sms ? a.T : 8ll * sms);
  return bf ? launch_pdl(norm_fwd_any_kernel<bf16>, dim3(grid), dim3(256), 0, st, a)
            : launch_pdl(norm_fwd_any_kernel<float>, dim3(grid), dim3(256), 0, st, a);
}

cudaError_t launch_norm_bwd(const NormArgs &a, bool bf, bool vec, int sms, cudaStream_t st) {
  const int ctas = norm_bwd_ctas(a, bf, vec, sms);
  cudaError_t e;
  if (in_registers(a, bf, vec, sms)) {
    e = bf ? bwd_shape<bf16>(a, sms, ctas, st) : bwd_shape<float>(a, sms, ctas, st);
  } else {
    e = bf ? launch_pdl(norm_bwd_any_kernel<bf16>, dim3(ctas), dim3(256), 0, st, a)
           : launch_pdl(norm_bwd_any_kernel<float>, dim3(ctas), dim3(256), 0, st, a);
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_dw_kernel, dim3((a.D + 31) / 32), dim3(1024), 0, st, (const float *)a.part, ctas, a.D, a.dw);
}

}  // namespace gdn
