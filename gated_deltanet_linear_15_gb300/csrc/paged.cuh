// Work split of the attention over a paged cache, shared by its kernels.
//
// The (token, head-of-group) pairs of one sequence and key head are its query rows: row r is token r / G, query head
// h G + r % G.  A tile of MT consecutive rows reads the keys [lo, hi) that any of its rows sees, in blocks of BN
// tokens.  An item is one (sequence, tile, key head); its units are its key blocks (one when there are none).  All
// items' units stand in one line, sequence by sequence, and CTA c of C = min(grid, total) takes the units
// [total c / C, total (c + 1) / C): the same work for everyone to one block, whatever the lengths are, with at most two
// cut items per CTA.  A cut item's pieces, which consecutive CTAs hold, leave unnormalised sums, maxima and masses in
// the workspace, and a second kernel joins them in the order of the line, so the result does not depend on who finished
// first.
//
// Every CTA finds its range itself: it counts the tiles of all sequences, then the units of all tiles (two block
// scans), which costs about a microsecond and saves a planning launch.
#pragma once
#include <cuda.h>

#include "common.cuh"

namespace gdn {

struct PagedArgs {
  const void *q, *k, *v;
  void *o;
  float *lse;
  const int *table, *cu_q, *kv_lens;
  long long table_stride, q_tok, q_head, k_page, k_tok, k_head, v_page, v_tok, v_head, o_tok, o_head;  // elements
  int N, total_q, per_seq;  // per_seq: new tokens of every sequence when cu_q is NULL
  int Hq, Hkv, G, log2P, num_pages, max_pages, window;
  float scale_log2;         // scale * log2(e): the softmax runs in powers of two
  int *status;              // one word per CTA of the tensor-core kernel
  // cut items: headers [C][2] and records [C][2][MT * (D + 2)] (sums [MT][D], maxima [MT], masses [MT])
  int4 *hdr;
  float *part;
};

// header of a CTA's piece record: slot 1 holds the first piece of an item that goes on in the next CTA, slot 0 a
// piece of an item that began in an earlier one.  x: 0 none, 1 the item ends here, 2 it goes on.
// Slot 1: y = first row's token in q, z = key head, w = rows << 16 | first row's place in its group.
__host__ __device__ constexpr size_t record_floats(int MT, int D) { return (size_t)MT * (D + 2); }

struct SeqInfo {
  int qbeg, qlen, kv;
};
__device__ __forceinline__ SeqInfo seq_info(const PagedArgs &a, int n) {
  SeqInfo s;
  if (a.cu_q) {
    const int b = min(max(a.cu_q[n], 0), a.total_q), e = min(max(a.cu_q[n + 1], b), a.total_q);
    s.qbeg = b;
    s.qlen = e - b;
  } else {
    s.qbeg = n * a.per_seq;
    s.qlen = a.per_seq;
  }
  const long long room = (long long)a.max_pages << a.log2P;
  s.kv = (int)min((long long)max(a.kv_lens[n], 0), min(room, (long long)0x7fffff00));
  return s;
}

struct Tile {
  int rows;       // valid rows (0: no such tile)
  int lo, hi;     // keys that some row sees
  int blk0, nblk; // in blocks of BN
  __device__ __forceinline__ int units() const { return max(nblk, 1); }
  int pos0;       // position of token r0 / G of the sequence's new tokens
};
template <int MT, int BN>
__device__ __forceinline__ Tile tile_of(const PagedArgs &a, const SeqInfo &s, int t) {
  Tile w;  // the host keeps total_q * G below 2^31
  const unsigned R = (unsigned)s.qlen * a.G, r0 = (unsigned)t * MT;
  w.rows = R > r0 ? (int)min((unsigned)MT, R - r0) : 0;
  const int i0 = (int)(r0 / (unsigned)a.G), i1 = w.rows ? (int)((r0 + w.rows - 1) / (unsigned)a.G) : i0;
  w.pos0 = s.kv - s.qlen + i0;
  w.hi = max(0, min(s.kv, s.kv - s.qlen + i1 + 1));
  w.lo = a.window ? max(0, w.pos0 - a.window + 1) : 0;
  w.blk0 = w.lo / BN;
  w.nblk = w.rows > 0 && w.hi > w.lo ? (w.hi + BN - 1) / BN - w.blk0 : 0;
  return w;
}
template <int MT> __device__ __forceinline__ int tiles_of(const PagedArgs &a, const SeqInfo &s) {
  return (int)(((unsigned)s.qlen * a.G + MT - 1) / MT);
}

// barrier of the NT threads that look for the CTA's range (a CTA may have more)
template <int NT> __device__ __forceinline__ void plan_bar() { asm volatile("bar.sync 1, %0;\n" ::"n"(NT) : "memory"); }

// inclusive scan over threads 0 .. NT - 1 (all of them call it); sh holds NT / 32 values
template <int NT> __device__ __forceinline__ long long block_scan(long long x, long long *sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  plan_bar<NT>();
  if (lane == 31) sh[warp] = x;
  plan_bar<NT>();
  long long add = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) add += w < warp ? sh[w] : 0;
  return x + add;
}

// largest i in [0, NT) with pre[i] <= u (pre[0] = 0, non-decreasing)
template <int NT> __device__ __forceinline__ int find_slot(const long long *pre, long long u) {
  int i = 0;
#pragma unroll
  for (int s = NT / 2; s > 0; s >>= 1)
    if (pre[i + s] <= u) i += s;
  return i;
}

struct Cursor {
  int n, t, h;        // the item
  SeqInfo s;
  Tile w;
  long long u, end;   // this CTA's next unit and the end of its range
  int skip;           // units of the item that came before u
};

// Finds where this CTA's range begins.  False when it has none.  Threads 0 .. NT - 1 call it (NT a power of two).
template <int NT, int MT, int BN>
__device__ __forceinline__ bool cursor_begin(const PagedArgs &a, Cursor &c, long long (*pre)[NT + 1], long long *sh) {
  const int tid = threadIdx.x;
  // tiles of the sequences, NT equal shares of them
  const int cs = (a.N + NT - 1) / NT;
  const int n0 = min(a.N, tid * cs), n1 = min(a.N, n0 + cs);
  long long cnt = 0;
  for (int n = n0; n < n1; ++n) cnt += tiles_of<MT>(a, seq_info(a, n));
  const long long inc = block_scan<NT>(cnt, sh);
  pre[0][tid + 1] = inc;
  if (tid == 0) pre[0][0] = 0;
  plan_bar<NT>();
  const long long NTILE = pre[0][NT];
  // units of the tiles, NT equal shares of them
  const long long ct = (NTILE + NT - 1) / NT;
  auto seek = [&](long long x, int &n, int &t, SeqInfo &s) {  // tile number x of the line
    const int sl = find_slot<NT>(pre[0], x);
    n = sl * cs;
    long long left = x - pre[0][sl];
    for (;;) {
      s = seq_info(a, n);
      const int k = tiles_of<MT>(a, s);
      if (left < k) break;
      left -= k;
      ++n;
    }
    t = (int)left;
  };
  const long long x0 = min(NTILE, tid * ct), x1 = min(NTILE, x0 + ct);
  long long units = 0;
  if (x0 < x1) {
    int n, t;
    SeqInfo s;
    seek(x0, n, t, s);
    int k = tiles_of<MT>(a, s);
    for (long long x = x0;;) {
      units += tile_of<MT, BN>(a, s, t).units();
      if (++x >= x1) break;
      if (++t >= k) {
        t = 0;
        do {
          s = seq_info(a, ++n);
          k = tiles_of<MT>(a, s);
        } while (k == 0);
      }
    }
  }
  const long long uinc = block_scan<NT>(units * a.Hkv, sh);
  pre[1][tid + 1] = uinc;
  if (tid == 0) pre[1][0] = 0;
  plan_bar<NT>();
  const long long total = pre[1][NT];
  const long long C = min((long long)gridDim.x, total);
  if (blockIdx.x >= C) return false;
  c.u = total * blockIdx.x / C;
  c.end = total * (blockIdx.x + 1) / C;
  const int sl = find_slot<NT>(pre[1], c.u);
  seek(min(NTILE - 1, sl * ct), c.n, c.t, c.s);
  long long left = c.u - pre[1][sl];
  for (;;) {
    c.w = tile_of<MT, BN>(a, c.s, c.t);
    const long long per = c.w.units();
    if (left < per * a.Hkv) {
      c.h = (int)(left / per);
      c.skip = (int)(left - c.h * per);
      break;
    }
    left -= per * a.Hkv;
    if (++c.t >= tiles_of<MT>(a, c.s)) {
      c.t = 0;
      do c.s = seq_info(a, ++c.n);
      while (tiles_of<MT>(a, c.s) == 0);
    }
  }
  return true;
}

// The piece at the cursor: key blocks [b0, b1) (relative to the tile's first), whether it is the item's first and
// its last.  Returns the piece's units.
__device__ __forceinline__ int cursor_piece(const Cursor &c, int &b0, int &b1, bool &first, bool &last) {
  const int per = c.w.units();
  const int n = (int)min((long long)(per - c.skip), c.end - c.u);
  b0 = c.skip;
  b1 = min(c.w.nblk, c.skip + n);
  first = c.skip == 0;
  last = c.skip + n == per;
  return n;
}

// Moves past the piece of n units; false at the end of the range.
template <int MT, int BN> __device__ __forceinline__ bool cursor_next(const PagedArgs &a, Cursor &c, int n) {
  c.u += n;
  if (c.u >= c.end) return false;
  c.skip = 0;
  if (++c.h == a.Hkv) {
    c.h = 0;
    if (++c.t >= tiles_of<MT>(a, c.s)) {
      c.t = 0;
      do c.s = seq_info(a, ++c.n);
      while (tiles_of<MT>(a, c.s) == 0);
    }
    c.w = tile_of<MT, BN>(a, c.s, c.t);
  }
  return true;
}

// where row r of the cursor's tile lies in q and o
__device__ __forceinline__ void row_place(const PagedArgs &a, const Cursor &c, int MT, int r, int &tok, int &head) {
  const unsigned g = (unsigned)c.t * MT + r, i = g / (unsigned)a.G;
  tok = c.s.qbeg + (int)i;
  head = c.h * a.G + (int)(g - i * a.G);
}

cudaError_t launch_attn_rows(const PagedArgs &a, bool bf16_type, int D, int MT, int ctas, cudaStream_t st);
cudaError_t launch_attn_join(const PagedArgs &a, bool bf16_type, int D, int MT, int ctas, cudaStream_t st);
cudaError_t launch_attn_chunk_tc(const PagedArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, int D, int ctas,
                                 cudaStream_t st);

}  // namespace gdn
