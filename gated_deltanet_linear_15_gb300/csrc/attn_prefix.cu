// Attention of groups of sequences that share a prefix, around the kernels that compute it in two parts: HEAD, the shared keys,
// once for all the group's new tokens, and TAIL, every sequence's own keys behind them.  With the sums, maxima and masses
// of the pieces i of both parts,
//   m = max m_i,  o = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i,  lse = ln 2 (m + log2 sum 2^(m_i - m) l_i).
//
// The plan looks at the lengths, which only the device knows: a group's prefix is cut to what all its sequences with new tokens
// had cached before them, so that every new token sees all of it, whatever the caller says; and a group with one such sequence
// has none.  The prefix is read from the table row of the first of them, which therefore holds all of it: a sequence without new
// tokens may have ended, with a row that names no pages.  It is one block, a warp to a group, and a few more that clear the
// rows' notes.
//
// The parts run at the same time, each on some of the SMs, where one of them at least is the row kernel, which waits for memory
// most of the time while the other one computes: launches, searches and ends of the two overlap too.  The plan shares
// the SMs out by the parts' blocks, and the CTAs behind a part's share leave at once.  64 sequences of up to 1024 tokens of their
// own behind 8192 shared ones, 8 key heads of 128, one new token each: 55 us; one part after the other 72; as sequences
// that share nothing 228.  Two chunk kernels only take from one another (8 groups of 8 with 5 new tokens each, in a row of
// calls: 79 us at the same time, 63 one after the other).
//
// The join takes a warp to a row.  The rows' notes say where its pieces are: a head that 152 CTAs share has as many, and a row
// reads no more of them than D sums and two numbers each, all from L2.  Bound by latency: a batch of pieces is asked for at once.
#include "paged.cuh"

namespace gdn {

namespace {

constexpr int NTP = 1024, JOIN_WARPS = 4, BATCH = 8;
constexpr int NONE = -2;  // a row's note: no pieces

}  // namespace

// The SMs are shared out so that both parts end at about the same time.  (The sums are of whole numbers, so their order does
// not matter.  Calls whose parts do not share the SMs have a plan without this code, which costs 3 us even where it is jumped
// over.)
__device__ __forceinline__ void share_out(const PagedArgs &a, const PrefixPlan &p) {
  __syncthreads();  // all is planned
  long long work[2] = {0, 0};  // blocks of a key head's items, with their setup
  auto add = [&](int part, int rows, int keys) {
    const PrefixPlan::Share &s = p.share[part];
    if (rows > 0) work[part] += (long long)((rows + s.MT - 1) / s.MT) * ((keys + s.BN - 1) / s.BN + s.setup);
  };
  for (int g = threadIdx.x; g < p.groups; g += NTP) {
    const int4 v = p.head[g];
    if (v.z > 0) add(0, v.y * a.G, v.z);
  }
  for (int n = threadIdx.x; n < a.N; n += NTP) {
    const int4 v = p.tail[n];
    add(1, v.y * a.G, v.z - v.w);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (work[i]) atomicAdd(p.blocks + i, (unsigned long long)work[i]);
  }
  __syncthreads();
  if (threadIdx.x > 0) return;
  float w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = (float)__ldcg(p.blocks + i) * (float)a.Hkv;
  int sms = 0;  // of HEAD
  if (w[0] > 0.f) {
    const float late = p.share[0].start - p.share[1].start, h = w[0] * p.share[0].cost, t = w[1] * p.share[1].cost;
    // no CTA without a block, and no less than a quarter for the tails, whose work is known least
    int hi = max(1, (int)fminf(0.75f * (float)p.sms, ceilf(w[0] / (float)p.share[0].per_sm)));
    for (sms = 1; sms < hi;) {
      const int mid = (sms + hi) >> 1;
      if (late + h / (float)mid <= t / (float)(p.sms - mid)) hi = mid;
      else sms = mid + 1;
    }
  }
  p.ctas[0] = sms * p.share[0].per_sm;
  asm volatile("st.release.gpu.global.b32 [%0], %1;\n" ::"l"(p.ctas + 1), "r"((p.sms - sms) * p.share[1].per_sm) : "memory");
}

template <bool TOGETHER> __global__ void __launch_bounds__(NTP) prefix_plan_kernel(PagedArgs a, PrefixPlan p, int2 *head_loc, int2 *tail_loc) {
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x > 0) {
    const long long rows = (long long)a.total_q * a.Hq;
    for (long long i = (long long)(blockIdx.x - 1) * NTP + threadIdx.x; i < rows; i += (long long)(gridDim.x - 1) * NTP) {
      head_loc[i] = make_int2(NONE, 0);
      tail_loc[i] = make_int2(NONE, 0);
    }
    return;
  }
  if (TOGETHER && threadIdx.x < 2) p.blocks[threadIdx.x] = 0;
  for (int n = threadIdx.x; n < a.N; n += NTP) {  // sequences that no group names have no prefix
    const SeqInfo s = seq_info(a, n);
    p.tail[n] = make_int4(s.qbeg, s.qlen, s.kv, 0);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int g = threadIdx.x >> 5; g < p.groups; g += NTP / 32) {
    int n0, n1;
    if (p.cu_seqs) {
      n0 = min(max(p.cu_seqs[g], 0), a.N);
      n1 = min(max(p.cu_seqs[g + 1], n0), a.N);
    } else {
      const int per = a.N / p.groups;
      n0 = g * per;
      n1 = n0 + per;
    }
    int cached = 0x7fffffff, beg = 0x7fffffff, end = 0, first = 0x7fffffff, last = -1;
    for (int n = n0 + lane; n < n1; n += 32) {
      const SeqInfo s = seq_info(a, n);
      if (s.qlen == 0) continue;  // sees nothing, and limits nothing
      first = min(first, n);
      last = n;
      cached = min(cached, s.kv - s.qlen);
      beg = min(beg, s.qbeg);
      end = max(end, s.qbeg + s.qlen);
    }
    cached = __reduce_min_sync(0xffffffffu, cached);
    beg = __reduce_min_sync(0xffffffffu, beg);
    end = __reduce_max_sync(0xffffffffu, end);
    first = __reduce_min_sync(0xffffffffu, first);
    last = __reduce_max_sync(0xffffffffu, last);
    const int prefix = last > first ? max(0, min(p.prefix_lens[g], cached)) : 0;
    // The group's rows are those from the first token to the last: its sequences follow one another.
    if (lane == 0) p.head[g] = prefix > 0 ? make_int4(beg, end - beg, prefix, first) : make_int4(0, 0, 0, 0);
    for (int n = n0 + lane; n < n1; n += 32) p.tail[n].w = min(prefix, p.tail[n].z);
  }
  if constexpr (TOGETHER) share_out(a, p);
}

template <typename I, int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS) prefix_join_kernel(PagedArgs head, PagedArgs tail, int head_MT, int tail_MT, int head_ctas,
                                                                      int tail_ctas) {
  constexpr int E = D / 32;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)tail.total_q * tail.Hq;
  for (long long row = (long long)blockIdx.x * JOIN_WARPS + (threadIdx.x >> 5); row < rows; row += (long long)gridDim.x * JOIN_WARPS) {
    const int2 at[2] = {head.loc[row], tail.loc[row]};
    if (at[0].x == NONE && at[1].x == NONE) continue;  // no sequence names the token
    float M = -INFINITY, L = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const PagedArgs &a = part ? tail : head;
      const int MT = part ? tail_MT : head_MT, ctas = part ? tail_ctas : head_ctas, c = at[part].x, r = at[part].y;
      if (c == NONE) continue;
      const bool whole = c < 0;
      int np = 1;
      if (!whole) {
        if (c >= ctas || (unsigned)r >= (unsigned)MT) continue;
        np = min(a.hdr[c].x, ctas - c);
      }
      const long long rf = (long long)record_floats(MT, D);
      // piece 0 is slot 1 of CTA c, piece i slot 0 of CTA c + i
      const float *p0 = whole ? a.sums + row * D : a.part + ((long long)c * 2 + 1) * rf + (long long)r * D;
      const float *p1 = a.part + (long long)c * 2 * rf + (long long)r * D;
      for (int b = 0; b < np; b += BATCH) {
        float m[BATCH], l[BATCH], v[BATCH][E];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          m[i] = -INFINITY;
          l[i] = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) v[i][e] = 0.f;
          if (b + i < np) {
            const float *p = b + i == 0 ? p0 : p1 + (b + i) * 2 * rf;
            if (whole) {
              const float2 x = a.mass[row];
              m[i] = x.x;
              l[i] = x.y;
            } else {  // maxima and masses of the record, behind its sums
              const float *q = p - (long long)r * D + MT * D + r;
              m[i] = q[0];
              l[i] = q[MT];
            }
            if constexpr (E == 4) {
              const float4 t = *reinterpret_cast<const float4 *>(p + 4 * lane);
              v[i][0] = t.x; v[i][1] = t.y; v[i][2] = t.z; v[i][3] = t.w;
            } else {
              const float2 t = *reinterpret_cast<const float2 *>(p + 2 * lane);
              v[i][0] = t.x; v[i][1] = t.y;
            }
          }
        }
        float mn = M;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) mn = fmaxf(mn, m[i]);
        const float ref = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every factor below is 0
        float f = exp2f(M - ref);
        L *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          f = exp2f(m[i] - ref);
          L += f * l[i];
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] += f * v[i][e];
        }
        M = mn;
      }
    }
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // nothing seen: zeros; a NaN stays
    const long long tok = row / tail.Hq;
    const int h = (int)(row - tok * tail.Hq);
    I *op = static_cast<I *>(tail.o) + tok * tail.o_tok + h * tail.o_head + E * lane;
#pragma unroll
    for (int e = 0; e < E; e += 2) st2(op + e, o[e] * inv, o[e + 1] * inv);
    if (tail.lse && lane == 0) tail.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
}

cudaError_t launch_prefix_plan(const PagedArgs &a, const PrefixPlan &p, int2 *head_loc, int2 *tail_loc, cudaStream_t st) {
  const long long rows = (long long)a.total_q * a.Hq;
  const unsigned clear = (unsigned)((rows + 4 * NTP - 1) / (4 * NTP) < 152 ? (rows + 4 * NTP - 1) / (4 * NTP) : 152);
  return launch_pdl(p.together ? prefix_plan_kernel<true> : prefix_plan_kernel<false>, dim3(1 + clear), dim3(NTP), 0, st, a, p, head_loc, tail_loc);
}

cudaError_t launch_prefix_join(const PagedArgs &head, const PagedArgs &tail, bool bf, int D, int head_MT, int tail_MT, int head_ctas,
                               int tail_ctas, cudaStream_t st) {
  const long long rows = (long long)tail.total_q * tail.Hq, blocks = (rows + JOIN_WARPS - 1) / JOIN_WARPS;
  const dim3 grid((unsigned)(blocks < 152 * 16 ? blocks : 152 * 16));
  auto *k = bf ? (D == 64 ? prefix_join_kernel<bf16, 64> : prefix_join_kernel<bf16, 128>)
               : (D == 64 ? prefix_join_kernel<float, 64> : prefix_join_kernel<float, 128>);
  return launch_pdl(k, grid, dim3(32 * JOIN_WARPS), 0, st, head, tail, head_MT, tail_MT, head_ctas, tail_ctas);
}

}  // namespace gdn
