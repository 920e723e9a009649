// Upkeep of a paged cache: growing, branching, ending and compacting sequences, and copying pages or per-sequence
// states (the caches of a hybrid stack: pages for its softmax layers, one recurrent state per sequence and delta-rule
// layer; onedev.kr summary of the FlashQLA talk, background paragraph).
//
// The bookkeeping is whole numbers: free pages are handed out lowest first, in the order of the request list, by
// prefix sums, so every run gives the same tables.  One CTA plans (its scans run over the requests and, until enough
// are found, over the pages' counts, 16384 of them a step); what is long, the rows of the tables and the copies, goes to
// the whole GPU in a second launch.  Copies are bound by bytes (each slot read and written once): a slot is cut into
// 16 KB chunks, the chunks of all pairs and pools stand in one line, and a warp-coalesced thread moves four 16-byte
// pieces at a time, loaded before the first is stored.  8192 pages of 16 tokens compacted, 522 MB read and written: 88 us,
// 5.9 TB/s; 64 sequences branched, 132 MB: 29 us, of which ending the old branches takes 3, the plan 7 and the copies 18.
#include "block.h"
#include "common.cuh"

namespace gdn {

namespace {

constexpr int NP_T = 1024;      // threads of a planning CTA
constexpr int CHUNK = 16384;    // bytes of a copy chunk
constexpr int COPY_T = 256;

// inclusive sum over the CTA; sh holds 32 ints.  Every thread takes part.
__device__ __forceinline__ int scan_1024(int x, int *sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    sh[lane] = y;
  }
  __syncthreads();
  return x + (warp ? sh[warp - 1] : 0);
}

constexpr int SUB = 4, STEP = SUB * 4 * NP_T;  // a step: SUB rounds of four counts per thread, 16384 in all

// r[4 k + e] = the count of page base + 4096 k + 4 tid + e (`past` past the end): neighbours in neighbouring threads
__device__ __forceinline__ void load_refs(const int *ref, int NP, int base, int past, int (&r)[4 * SUB]) {
#pragma unroll
  for (int k = 0; k < SUB; ++k) {
    const int i = base + 4 * (NP_T * k + (int)threadIdx.x);
    if (i + 4 <= NP && (reinterpret_cast<uintptr_t>(ref) & 15) == 0) {
      const int4 v = *reinterpret_cast<const int4 *>(ref + i);
      r[4 * k] = v.x; r[4 * k + 1] = v.y; r[4 * k + 2] = v.z; r[4 * k + 3] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) r[4 * k + e] = i + e < NP ? ref[i + e] : past;
    }
  }
}

// The SUB rounds' counts in one scan: 16 bits each (a round has 4096 pages at most).  n: this thread's; on return rank[k]
// pages of the step come before this thread's of round k.  Returns the step's total.
__device__ __forceinline__ int scan_rounds(const int (&n)[SUB], int (&rank)[SUB], unsigned long long *sh) {
  unsigned long long x = 0;
#pragma unroll
  for (int k = 0; k < SUB; ++k) x |= (unsigned long long)n[k] << (16 * k);
  const unsigned long long own = x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  unsigned long long y = sh[lane];  // every warp sums the warps' totals for itself
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  const unsigned long long all = __shfl_sync(0xffffffffu, y, 31), before = __shfl_sync(0xffffffffu, y, warp ? warp - 1 : 0);
  x += (warp ? before : 0) - own;
  int sum = 0;
#pragma unroll
  for (int k = 0; k < SUB; ++k) {
    rank[k] = sum + (int)(x >> (16 * k) & 0xffff);
    sum += (int)(all >> (16 * k) & 0xffff);
  }
  return sum;
}

// Calls give(rank, page) for the free pages of rank 0 .. want - 1 (ascending numbers), and returns how many free pages
// were seen (at least `want` when there are so many).  r0: the first step's counts, which the caller asks for before it
// goes through its requests, so that the two waits for memory are one.
template <class F>
__device__ __forceinline__ int hand_out(const int *ref, int NP, int want, const int (&r0)[4 * SUB], unsigned long long *sh, F give) {
  int seen = 0;
  for (int base = 0; base < NP && seen < want; base += STEP) {
    int r[4 * SUB], n[SUB], rank[SUB];
    if (base == 0) {
#pragma unroll
      for (int i = 0; i < 4 * SUB; ++i) r[i] = r0[i];
    } else {
      load_refs(ref, NP, base, 1, r);
    }
#pragma unroll
    for (int k = 0; k < SUB; ++k) {
      n[k] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) n[k] += r[4 * k + e] <= 0;
    }
    const int all = scan_rounds(n, rank, sh);
#pragma unroll
    for (int k = 0; k < SUB; ++k) {
      int x = seen + rank[k];
      if (n[k] > 0 && x < want) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (r[4 * k + e] <= 0) {
            if (x < want) give(x, base + 4 * (NP_T * k + (int)threadIdx.x) + e);
            ++x;
          }
      }
    }
    seen += all;
  }
  __syncthreads();
  return seen;
}

// free pages in all, up to `want`
__device__ __forceinline__ int count_free(const int *ref, int NP, int want, const int (&r0)[4 * SUB], unsigned long long *sh) {
  return hand_out(ref, NP, want, r0, sh, [](int, int) {});
}

__device__ __forceinline__ int pages_of(int len, int P) { return (int)(((long long)len + P - 1) / P); }

}  // namespace

// ws: prefix[m + 1] of the pages that the granted requests take
__global__ void __launch_bounds__(NP_T) pages_extend_kernel(PagesArgs a, const int *seqs, const int *add, int m, int *ok, int *pre) {
  __shared__ int sh[32];
  __shared__ unsigned long long sh64[32];
  __shared__ int granted;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  int r0[4 * SUB];
  load_refs(a.ref, a.NP, 0, 1, r0);
  // what each request needs, and the prefix of the needs in list order
  long long total = 0;
  for (int b = 0; b < m; b += NP_T) {
    const int i = b + tid;
    int need = 0;
    bool good = false;
    if (i < m) {
      const int s = seqs[i], d = add[i];
      if ((unsigned)s < (unsigned)a.S && d >= 0) {
        const int len = a.lens[s], have = pages_of(max(len, 0), a.P);
        const long long end = (long long)len + d;
        good = len >= 0 && end <= min((long long)a.W * a.P, 0x7fffffffll);  // a length has 31 bits
        if (good && len % a.P != 0 && d > 0) {  // it will write into its last page: that page has to be its own
          const int pg = a.table[s * a.ts + have - 1];
          good = (unsigned)pg < (unsigned)a.NP && a.ref[pg] == 1;
        }
        if (good) need = min(pages_of((int)end, a.P) - have, a.NP + 1);
      }
    }
    const int inc = scan_1024(need, sh);
    // past INT_MAX / 2 nothing can be granted any more, so the prefix stops growing there
    const long long upto = min(total + inc, 1ll << 30);
    if (i < m) {
      pre[i + 1] = (int)upto;
      ok[i] = good ? 1 + (need > 0) : 0;  // 2: takes pages (the prefix cannot tell where it has stopped growing)
    }
    const int all = sh[31];
    __syncthreads();
    total = min(total + all, 1ll << 30);
  }
  if (tid == 0) {
    pre[0] = 0;
    granted = 0;
  }
  __syncthreads();
  const int avail = count_free(a.ref, a.NP, (int)total, r0, sh64);
  // the requests whose pages, and all before theirs, are there
  for (int i = tid; i < m; i += NP_T) {
    if (ok[i] == 2) ok[i] = pre[i + 1] <= avail;
    if (pre[i + 1] <= avail) atomicMax(&granted, pre[i + 1]);
  }
  __syncthreads();
  const int want = granted;
  hand_out(a.ref, a.NP, want, r0, sh64, [&](int rank, int page) {
    int lo = 0, hi = m;  // the request with pre[lo] <= rank < pre[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= rank) lo = mid;
      else hi = mid;
    }
    const int s = seqs[lo];
    a.table[s * a.ts + pages_of(a.lens[s], a.P) + rank - pre[lo]] = page;
    a.ref[page] = 1;
  });
  __syncthreads();
  for (int i = tid; i < m; i += NP_T)
    if (ok[i]) a.lens[seqs[i]] += add[i];
}

// Which forks happen, the new page of each, the copy pairs.  src[i]: the parent's last page, psrc / pdst: parent and
// child, all -1 for what is not to be done; the new page is the copy's target (negative: none).
__global__ void __launch_bounds__(NP_T) pages_fork_plan_kernel(PagesArgs a, const int *parents, const int *children, int m,
                                                               int *new_page, int *src, int *psrc, int *pdst) {
  __shared__ int sh[32], few[NP_T];
  __shared__ unsigned long long sh64[32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  int *list = m <= NP_T ? few : pdst + m;  // the request of every rank
  int total = 0, r0[4 * SUB];
  load_refs(a.ref, a.NP, 0, 1, r0);
  for (int b = 0; b < m; b += NP_T) {
    const int i = b + tid;
    int need = 0, p = -1, c = -1, from = -1;
    bool good = false;
    if (i < m) {
      p = parents[i];
      c = children[i];
      good = (unsigned)p < (unsigned)a.S && (unsigned)c < (unsigned)a.S && p != c && a.lens[c] == 0;
      if (good) {
        const int len = a.lens[p];
        good = len >= 0 && len <= (long long)a.W * a.P;
        if (good && len % a.P != 0) {
          from = a.table[p * a.ts + len / a.P];
          good = (unsigned)from < (unsigned)a.NP;
          need = good;
        }
      }
    }
    const int inc = scan_1024(need, sh);
    if (i < m) {
      if (need) list[total + inc - 1] = i;
      else new_page[i] = good ? -1 : -2;
      src[i] = need ? from : -1;
      psrc[i] = good ? p : -1;
      pdst[i] = good ? c : -1;
    }
    const int all = sh[31];
    __syncthreads();
    total += all;
  }
  __syncthreads();
  const int seen = hand_out(a.ref, a.NP, total, r0, sh64, [&](int rank, int page) {
    new_page[list[rank]] = page;
    a.ref[page] = 1;
  });
  for (int r = seen + tid; r < total; r += NP_T) {  // no page left: the fork is left out
    const int i = list[r];
    new_page[i] = -2;
    src[i] = psrc[i] = pdst[i] = -1;
  }
  __syncthreads();
  for (int i = tid; i < m; i += NP_T)
    if (pdst[i] >= 0) a.lens[pdst[i]] = a.lens[psrc[i]];
}

__global__ void __launch_bounds__(256) pages_free_kernel(PagesArgs a, const int *seqs) {
  pdl_trigger();
  pdl_wait();
  const int s = seqs[blockIdx.x];
  if ((unsigned)s >= (unsigned)a.S) return;
  for (int j = blockIdx.y * 256 + threadIdx.x; j < a.W; j += 256 * gridDim.y) {
    // taken by exchange, so that a sequence named twice gives its pages back once
    const int pg = atomicExch(a.table + s * a.ts + j, -1);
    if ((unsigned)pg < (unsigned)a.NP) atomicAdd(a.ref + pg, -1);
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) a.lens[s] = 0;
}

// src / dst: the moves, ascending; *moves their number; *front how many pages are in use; map[page] the new number of a
// page that is not in front.  The launch that renames writes the counts of the pages that stay, this one the others.
__global__ void __launch_bounds__(NP_T) pages_compact_plan_kernel(PagesArgs a, const int *ref_in, int *map, int *src, int *dst, int *moves,
                                                                  int *front) {
  __shared__ unsigned long long sh[32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  int live = 0, r[4 * SUB], n[SUB], rank[SUB];
  for (int base = 0; base < a.NP; base += STEP) {
    load_refs(ref_in, a.NP, base, 0, r);
#pragma unroll
    for (int k = 0; k < SUB; ++k) {
      n[k] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) n[k] += r[4 * k + e] > 0;
    }
    live += scan_rounds(n, rank, sh);
  }
  int holes = 0, highs = 0;
  for (int base = 0; base < a.NP; base += STEP) {
    if (a.NP > STEP) load_refs(ref_in, a.NP, base, 0, r);  // one step: they are still here
    // free pages of the front, then pages to move
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      auto mine = [&](int k, int e) {
        const int i = base + 4 * (NP_T * k + tid) + e;
        return w == 0 ? i < live && r[4 * k + e] <= 0 : i >= live && r[4 * k + e] > 0;
      };
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        n[k] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) n[k] += mine(k, e);
      }
      const int all = scan_rounds(n, rank, sh);
      int *to = w ? src + highs : dst + holes;
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        int x = rank[k];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (mine(k, e)) to[x++] = base + 4 * (NP_T * k + tid) + e;
      }
      if (w) {
#pragma unroll
        for (int k = 0; k < SUB; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = base + 4 * (NP_T * k + tid) + e;
            if (i >= live && i < a.NP && r[4 * k + e] <= 0) {
              map[i] = i;
              a.ref[i] = 0;
            }
          }
      }
      if (w) highs += all;
      else holes += all;
    }
  }
  __syncthreads();
  for (int k = tid; k < highs; k += NP_T) {  // as many holes in front as pages in use behind
    const int s = src[k], d = dst[k];
    map[s] = d;
    a.ref[d] = ref_in[s];
    a.ref[s] = 0;
  }
  if (tid == 0) {
    *moves = highs;
    *front = live;
  }
}

__global__ void __launch_bounds__(COPY_T) slots_copy_kernel(const __grid_constant__ PoolList pl, const PairList l0, const PairList l1,
                                                           int count, const int *count_dev, const __grid_constant__ TableJob job) {
  pdl_trigger();
  pdl_wait();
  const PagesArgs &a = job.a;
  if (job.kind == TableJob::FORK) {
    // the children's table rows, and a reference more for every page that they share
    for (int i = blockIdx.x; i < job.m; i += gridDim.x) {
      const int p = job.psrc[i], c = job.pdst[i];
      if (p < 0) continue;
      const int len = a.lens[p], full = len / a.P;
      for (int j = threadIdx.x; j < a.W; j += COPY_T) {
        int pg = -1;
        if (j < full) {
          pg = a.table[p * a.ts + j];
          if ((unsigned)pg < (unsigned)a.NP) atomicAdd(a.ref + pg, 1);
        } else if (j == full && len % a.P != 0) {
          pg = job.new_page[i];
        }
        a.table[c * a.ts + j] = pg;
      }
    }
  } else if (job.kind == TableJob::REMAP) {
    const long long n = (long long)a.S * a.W, t0 = blockIdx.x * (long long)COPY_T + threadIdx.x, step = (long long)COPY_T * gridDim.x;
    const int front = *job.front;
    for (long long i = t0; i < n; i += step) {
      const long long at = (i / a.W) * a.ts + i % a.W;
      const int pg = job.table_in[at];
      a.table[at] = pg >= front && pg < a.NP ? job.map[pg] : pg;
    }
    // the counts of pages that stay; the others are there already
    for (long long i = t0; i < front; i += step) {
      const int x = job.ref_in[i];
      if (x > 0) a.ref[i] = x;
    }
  }
  if (count_dev) count = min(count, *count_dev);
  const long long per = pl.chunk0[pl.n], total = per * count;  // chunks of a pair in all pools
  for (long long x = blockIdx.x; x < total; x += gridDim.x) {
    const int i = (int)(x / per);
    const long long in = x - i * per;
    int p = 0;
    while (in >= pl.chunk0[p + 1]) ++p;
    const gdn_slot_pool &g = pl.p[p];
    const PairList &l = pl.list[p] ? l1 : l0;
    const int s = l.src[i], d = l.dst[i];
    if (s < 0 || d < 0 || s >= g.slots || d >= g.slots) continue;
    const long long b0 = (in - pl.chunk0[p]) * CHUNK;
    const int n16 = (int)(min((long long)CHUNK, g.bytes - b0) >> 4);
    const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const char *>(g.base) + s * g.stride + b0);
    uint4 *to = reinterpret_cast<uint4 *>(static_cast<char *>(g.base) + d * g.stride + b0);
    uint4 v[CHUNK / 16 / COPY_T];
#pragma unroll
    for (int k = 0; k < CHUNK / 16 / COPY_T; ++k)
      if ((int)threadIdx.x + k * COPY_T < n16) v[k] = __ldcs(from + threadIdx.x + k * COPY_T);
#pragma unroll
    for (int k = 0; k < CHUNK / 16 / COPY_T; ++k)
      if ((int)threadIdx.x + k * COPY_T < n16) __stcs(to + threadIdx.x + k * COPY_T, v[k]);
  }
}

cudaError_t launch_slots_copy(const PoolList &pl, const PairList (&pairs)[2], int count, const int *count_dev, const TableJob &job,
                              cudaStream_t st) {
  PoolList l = pl;
  l.chunk0[0] = 0;
  for (int i = 0; i < l.n; ++i) l.chunk0[i + 1] = l.chunk0[i] + (l.p[i].bytes + CHUNK - 1) / CHUNK;
  long long want = l.chunk0[l.n] * count;
  if (job.kind == TableJob::FORK) want = want > job.m ? want : job.m;
  if (job.kind == TableJob::REMAP) {
    const long long n = ((long long)job.a.S * job.a.W + COPY_T - 1) / COPY_T;
    want = want > n ? want : n;
  }
  if (want <= 0) return cudaSuccess;
  // Eight CTAs of 256 threads fill an SM.  Eight times as many, of which one starts as another ends, drift apart and keep
  // reads and writes mixed (8192 pages compacted: 88 us; 95 us with eight per SM that all walk in step, 100 us without a
  // limit, when most find that their pair is not among those that move).
  const long long cap = 152 * 64;
  return launch_pdl(slots_copy_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(COPY_T), 0, st, l, pairs[0], pairs[1], count,
                    count_dev, job);
}

namespace {
dim3 rows_grid(int m, int W) { return dim3((unsigned)m, (unsigned)((W + 1023) / 1024 < 64 ? (W + 1023) / 1024 : 64)); }
}  // namespace

cudaError_t launch_pages_extend(const PagesArgs &a, const int *seqs, const int *add, int m, int *ok, int *ws, cudaStream_t st) {
  return launch_pdl(pages_extend_kernel, dim3(1), dim3(NP_T), 0, st, a, seqs, add, m, ok, ws);
}
cudaError_t launch_pages_fork_plan(const PagesArgs &a, const int *parents, const int *children, int m, int *new_page, int *src,
                                   int *psrc, int *pdst, cudaStream_t st) {
  return launch_pdl(pages_fork_plan_kernel, dim3(1), dim3(NP_T), 0, st, a, parents, children, m, new_page, src, psrc, pdst);
}
cudaError_t launch_pages_free(const PagesArgs &a, const int *seqs, int m, cudaStream_t st) {
  return launch_pdl(pages_free_kernel, rows_grid(m, a.W), dim3(256), 0, st, a, seqs);
}
cudaError_t launch_pages_compact_plan(const PagesArgs &a, const int *ref_in, int *map, int *src, int *dst, int *moves, int *front,
                                      cudaStream_t st) {
  return launch_pdl(pages_compact_plan_kernel, dim3(1), dim3(NP_T), 0, st, a, ref_in, map, src, dst, moves, front);
}
}  // namespace gdn
