// Work split of the attention over a paged cache, shared by its kernels.
//
// The (token, head-of-group) pairs of one sequence and key head are its query rows: row r is token r / G, query head
// h G + r % G.  A tile of MT consecutive rows reads the keys [lo, hi) that any of its rows sees, in blocks of BN
// tokens.  An item is one (sequence, tile, key head); its units are a few for its setup, then its key blocks (one when
// there are none).  All items' units stand in one line, sequence by sequence, and CTA c of C = min(grid, total) takes the
// units [total c / C, total (c + 1) / C): the same work for everyone to one block, whatever the lengths are, with at most
// two cut items per CTA.  A range that ends among an item's setup units leaves the item to the next CTA.  A cut item's
// pieces, which consecutive CTAs hold, leave unnormalised sums, maxima and masses in the workspace, and a second kernel
// joins them in the order of the line, so the result does not depend on who finished first.
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
  int *status;              // one word per CTA: 0, or 4 when a bounded wait of it ran out
  int expire;               // test hook: one wait that runs out, and nothing else
  // cut items: headers [C] and records [C][2][MT * (D + 2)] (sums [MT][D], maxima [MT], masses [MT])
  int4 *hdr;
  float *part;
};

// Records of a CTA: slot 1 holds the first piece of an item that goes on in the next CTA, slot 0 a piece of an item that
// began in an earlier one.  Header of the CTA: x the number of pieces of the item in slot 1 (0: none), y its first row's
// token in q, z its key head, w = rows << 16 | first row's place in its group.
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

// Blocks that an item counts for besides its own: what a piece costs before its first block and after its last.  Without
// them a CTA that gets many short items ends late (us without / with one / two / three blocks: rows: 8 sequences of
// 1 .. 256 new tokens in fp32 74 / 49 / 44 / 44, 64 decoded sequences 329 / 325 / 324 / 325, 32 sequences of 1 .. 8 new
// tokens 61 / 46 / 37 / 36; 256-row tiles: 2048 new tokens 114 / 68 / 56 / 53, 32 mixed prompts 397 / 323 / 274 / 280,
// 64 of 128 tokens 124 / 98 / 93 / 90).
template <int MT> constexpr int SETUP = MT <= 32 ? 2 : 3;

struct Tile {
  int rows;       // valid rows (0: no such tile)
  int lo, hi;     // keys that some row sees
  int blk0, nblk; // in blocks of BN
  int setup;      // SETUP
  __device__ __forceinline__ int units() const { return setup + max(nblk, 1); }
  int pos0;       // position of token r0 / G of the sequence's new tokens
};
template <int MT, int BN>
__device__ __forceinline__ Tile tile_of(const PagedArgs &a, const SeqInfo &s, int t) {
  Tile w;
  w.setup = SETUP<MT>;
  const unsigned R = (unsigned)s.qlen * a.G, r0 = (unsigned)t * MT;
  w.rows = R > r0 ? (int)min((unsigned)MT, R - r0) : 0;
  const int i0 = (int)(r0 / (unsigned)a.G), i1 = w.rows ? (int)((r0 + w.rows - 1) / (unsigned)a.G) : i0;
  w.pos0 = s.kv - s.qlen + i0;
  w.hi = max(0, min(s.kv, s.kv - s.qlen + i1 + 1));
  w.lo = a.window ? (int)max(0ll, (long long)w.pos0 - a.window + 1) : 0;  // pos0 < 0: fewer cached tokens than new ones
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
template <int NT, typename T> __device__ __forceinline__ T block_scan(T x, T *sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp] = x;
  plan_bar<NT>();
  T add = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) add += w < warp ? sh[w] : 0;
  return x + add;
}

// largest i in [0, NT) with pre[i] <= u (pre[0] = 0, non-decreasing)
template <int NT, typename T> __device__ __forceinline__ int find_slot(const T *pre, T u) {
  int i = 0;
#pragma unroll
  for (int s = NT / 2; s > 0; s >>= 1)
    if (pre[i + s] <= u) i += s;
  return i;
}

// 64-bit quotient; most lines are shorter than 2^32 units, for which the 32-bit division is several times as fast
__device__ __forceinline__ long long div_units(long long a, long long b) {
  if ((unsigned long long)a >> 32 == 0 && (unsigned long long)b >> 32 == 0) return (unsigned)a / (unsigned)b;
  return a / b;
}

// The split of the line: CTA c begins at unit c q + min(c, r).
struct Split {
  long long q;
  int r, C;
  __device__ __forceinline__ long long begin(int c) const { return c * q + min(c, r); }
  __device__ __forceinline__ int owner(long long u) const {  // the CTA that holds unit u
    const long long big = r * (q + 1);
    return (int)(u < big ? div_units(u, q + 1) : r + div_units(u - big, q));
  }
};

struct Cursor {
  int n, t, h;        // the item
  SeqInfo s;
  Tile w;
  int skip;           // units of the item that came before u
  long long u, end;   // this CTA's next unit and the end of its range
  Split split;
  __device__ __forceinline__ bool works() const { return skip + (end - u) > w.setup; }  // more than an item's setup
};

// shared memory of the search
template <int NT> struct PlanSmem {
  long long units[NT + 1], scan[NT / 32];
  int tiles[NT + 1];
};

// Finds where this CTA's range begins.  False when it has none.  Threads 0 .. NT - 1 call it (NT a power of two).
template <int NT, int MT, int BN>
__device__ __noinline__ bool cursor_begin_any(const PagedArgs &a, Cursor &c, PlanSmem<NT> &sm) {
  const int tid = threadIdx.x;
  // tiles of the sequences, NT equal shares of them (a thread with one sequence keeps what it read)
  const int cs = a.N / NT + (a.N % NT > 0);
  const int n0 = (int)min((long long)a.N, (long long)tid * cs), n1 = (int)min((long long)a.N, (long long)n0 + cs);
  long long cnt = 0;
  for (int n = n0; n < n1; ++n) cnt += tiles_of<MT>(a, seq_info(a, n));
  const long long inc = block_scan<NT>(cnt, sm.scan);
  sm.tiles[tid + 1] = (int)inc;
  if (tid == 0) sm.tiles[0] = 0;
  if (tid == NT - 1) sm.units[0] = inc;
  plan_bar<NT>();
  // Sequences that share no tokens have no more tiles than this (each at most one that is not full).  A cu_q that goes back
  // names tokens many times over, more tiles than 31 bits hold in the worst case: such a batch is left undone.
  const long long most = a.N + (long long)a.total_q * a.G / MT, named = sm.units[0];
  plan_bar<NT>();  // sm.units and sm.scan are written again
  if (named > most || named > 0x7fffffffll - NT) return false;
  const int NTILE = (int)named;
  // units of the tiles, NT equal shares of them
  const int ct = (NTILE + NT - 1) / NT;
  auto seek = [&](int x, int &n, int &t, SeqInfo &s) {  // tile number x of the line
    const int sl = find_slot<NT>(sm.tiles, x);
    n = sl * cs;
    int left = x - sm.tiles[sl];
    for (;;) {
      s = seq_info(a, n);
      const int k = tiles_of<MT>(a, s);
      if (left < k) break;
      left -= k;
      ++n;
    }
    t = left;
  };
  const int x0 = (int)min((long long)NTILE, (long long)tid * ct), x1 = (int)min((long long)NTILE, (long long)x0 + ct);
  long long units = 0;
  if (x0 < x1) {
    int n, t;
    SeqInfo s;
    seek(x0, n, t, s);
    int k = tiles_of<MT>(a, s);
    for (int x = x0;;) {
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
  const long long uinc = block_scan<NT>(units * a.Hkv, sm.scan);
  sm.units[tid + 1] = uinc;
  if (tid == 0) sm.units[0] = 0;
  plan_bar<NT>();
  const long long total = sm.units[NT];
  c.split.C = (int)min((long long)gridDim.x, total);
  if (blockIdx.x >= c.split.C) return false;
  c.split.q = div_units(total, c.split.C);
  c.split.r = (int)(total - c.split.q * c.split.C);
  c.u = c.split.begin(blockIdx.x);
  c.end = c.split.begin(blockIdx.x + 1);
  const int sl = find_slot<NT>(sm.units, c.u);
  seek((int)min((long long)NTILE - 1, (long long)sl * ct), c.n, c.t, c.s);
  long long left = c.u - sm.units[sl];
  for (;;) {
    c.w = tile_of<MT, BN>(a, c.s, c.t);
    const int per = c.w.units();
    if (left < (long long)per * a.Hkv) {
      c.h = (int)div_units(left, per);
      c.skip = (int)(left - (long long)c.h * per);
      break;
    }
    left -= (long long)per * a.Hkv;
    if (++c.t >= tiles_of<MT>(a, c.s)) {
      c.t = 0;
      do c.s = seq_info(a, ++c.n);
      while (tiles_of<MT>(a, c.s) == 0);
    }
  }
  return true;
}

// The same for up to 512 sequences with up to 2048 tiles, by one warp without barriers, each lane taking an equal share of
// the sequences and then of the tiles.  A CTA runs this code once, so most of its time is that of fetching instructions;
// the search above costs 64 sequences 7 us more.  seqs: what is known of the sequences, in shared memory.  Writes c (from
// one lane) and returns 1, 0 when the CTA has no work, or 2 when the batch is too large.
template <int MT, int BN> __device__ __forceinline__ int cursor_begin_warp(const PagedArgs &a, Cursor &c, const SeqInfo *seqs) {
  const int lane = threadIdx.x & 31;
  auto scan = [&](long long x) {
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  const int cs = (a.N + 31) >> 5, n0 = min(a.N, lane * cs), n1 = min(a.N, n0 + cs);
  long long cnt = 0;
#pragma unroll 1
  for (int n = n0; n < n1; ++n) cnt += tiles_of<MT>(a, seqs[n]);
  const long long inc = scan(cnt), all = __shfl_sync(0xffffffffu, inc, 31);
  if (all > 2048) return 2;
  // this lane's tiles [x0, x1); the first one's sequence is among those of the first lane whose tiles reach beyond x0
  const int tiles = (int)all, ct = (tiles + 31) >> 5, x0 = min(tiles, lane * ct), x1 = min(tiles, x0 + ct);
  int own = 0;
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1)
    if ((int)__shfl_sync(0xffffffffu, (int)inc, own + o - 1) <= x0) own += o;
  int left = x0 - __shfl_sync(0xffffffffu, (int)(inc - cnt), own);
  // walks from tile x0 on; a second time, up to unit `stop`, for the lane that holds the CTA's first one
  int n = own * cs, t = 0, k = 0;
  SeqInfo s = {0, 0, 0};
  Tile w;
  long long units = 0, stop = 1ll << 62;
  bool twice = false;
  long long u = 0, uinc = 0, mine = 0;
  Split sp = {1, 0, 1};
  for (;;) {
    if (x0 < x1) {
      int nn = n;
      t = left;
#pragma unroll 1
      for (;; ++nn) {
        s = seqs[nn];
        k = tiles_of<MT>(a, s);
        if (t < k) break;
        t -= k;
      }
      units = 0;
#pragma unroll 1
      for (int x = x0;;) {
        w = tile_of<MT, BN>(a, s, t);
        const long long per = (long long)w.units() * a.Hkv;
        if (units + per > stop) break;
        units += per;
        if (++x >= x1) break;
        for (++t; t >= k; t = 0) {
          s = seqs[++nn];
          k = tiles_of<MT>(a, s);
        }
      }
      if (twice) n = nn;
    }
    if (twice) break;
    mine = units;
    uinc = scan(units);
    const long long total = __shfl_sync(0xffffffffu, uinc, 31);
    sp.C = (int)min((long long)gridDim.x, total);
    if ((int)blockIdx.x >= sp.C) return 0;
    sp.q = div_units(total, sp.C);
    sp.r = (int)(total - sp.q * sp.C);
    u = sp.begin(blockIdx.x);
    if (lane != __ffs(__ballot_sync(0xffffffffu, uinc > u)) - 1) return 1;
    stop = u - (uinc - mine);
    twice = true;
  }
  const int per = w.units();
  c.n = n;
  c.t = t;
  c.h = (int)div_units(stop - units, per);
  c.s = s;
  c.w = w;
  c.skip = (int)(stop - units - (long long)c.h * per);
  c.u = u;
  c.end = sp.begin(blockIdx.x + 1);
  c.split = sp;
  return 1;
}

// And for up to 32 sequences with up to 32 tiles: a lane per sequence, then a lane per tile (1 us less than the search
// above for a decode step of one sequence).  Returns what it returns.
template <int MT, int BN> __device__ __forceinline__ int cursor_begin_small(const PagedArgs &a, Cursor &c) {
  if (a.N > 32) return 2;
  const int lane = threadIdx.x & 31;
  auto scan = [&](int x) {
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  SeqInfo s = {0, 0, 0};
  if (lane < a.N) s = seq_info(a, lane);
  const int k = lane < a.N ? tiles_of<MT>(a, s) : 0;
  if (__any_sync(0xffffffffu, k > 32)) return 2;
  const int inc = scan(k), tiles = __shfl_sync(0xffffffffu, inc, 31);
  if (tiles > 32) return 2;
  // lane x takes tile x of the line: its sequence is the first whose tiles reach beyond x
  int n = 0;
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1)
    if (__shfl_sync(0xffffffffu, inc, n + o - 1) <= lane) n += o;
  n = min(n, 31);
  const int t = lane - __shfl_sync(0xffffffffu, inc - k, n);
  s.qbeg = __shfl_sync(0xffffffffu, s.qbeg, n);
  s.qlen = __shfl_sync(0xffffffffu, s.qlen, n);
  s.kv = __shfl_sync(0xffffffffu, s.kv, n);
  const bool mine = lane < tiles;
  const Tile w = tile_of<MT, BN>(a, s, mine ? t : 0);
  const long long un = mine ? (long long)w.units() * a.Hkv : 0;
  if (__any_sync(0xffffffffu, un > (1 << 25))) return 2;
  const int uinc = scan((int)un), total = __shfl_sync(0xffffffffu, uinc, 31);
  const int C = min((int)gridDim.x, total);
  if ((int)blockIdx.x >= C) return 0;
  const int q = (unsigned)total / (unsigned)C, r = total - q * C;
  const int u = blockIdx.x * q + min((int)blockIdx.x, r);
  if (lane == __ffs(__ballot_sync(0xffffffffu, uinc > u)) - 1) {
    const int left = u - (uinc - (int)un), per = w.units();
    c.n = n;
    c.t = t;
    c.h = (unsigned)left / (unsigned)per;
    c.s = s;
    c.w = w;
    c.skip = left - c.h * per;
    c.u = u;
    c.end = u + q + ((int)blockIdx.x < r);
    c.split.q = q;
    c.split.r = r;
    c.split.C = C;
  }
  return 1;
}

// What every thread of the CTA does before one warp searches: the lengths of more than 32 sequences come to shared memory,
// all loads at once (256 decoded sequences of up to 128 tokens: 36.4 us, with the pages of the next
// piece asked for a piece ahead, instead of 38.0).
constexpr int WARP_SEQS = 512;
template <int NT> __device__ __forceinline__ void cursor_prepare(const PagedArgs &a, SeqInfo *seqs) {
  if (a.N <= 32 || a.N > WARP_SEQS) return;
  for (int n = threadIdx.x; n < a.N; n += NT) seqs[n] = seq_info(a, n);
  __syncthreads();
}
// One warp's search, whichever fits.  The caller's kernel has to keep its asynchronous copies off `seqs` until then.
template <int MT, int BN> __device__ __forceinline__ int cursor_begin_one_warp(const PagedArgs &a, Cursor &c, SeqInfo *seqs) {
  const int found = cursor_begin_small<MT, BN>(a, c);
  if (found != 2 || a.N > WARP_SEQS) return found;
  if (a.N <= 32) {
    const int lane = threadIdx.x & 31;
    if (lane < a.N) seqs[lane] = seq_info(a, lane);
    __syncwarp();
  }
  return cursor_begin_warp<MT, BN>(a, c, seqs);
}

// The header of a CTA whose last item goes on behind its range: c is the cursor at the item's first piece.
template <int MT> __device__ __forceinline__ int4 cut_header(const PagedArgs &a, const Cursor &c) {
  const int last = c.split.owner(c.u - c.skip + c.w.units() - 1);
  const unsigned r0 = (unsigned)c.t * MT, i = r0 / (unsigned)a.G;
  return make_int4(last - (int)blockIdx.x + 1, c.s.qbeg + (int)i, c.h, c.w.rows << 16 | (int)(r0 - i * a.G));
}

// The piece at the cursor: key blocks [b0, b1) (relative to the tile's first), whether it is the item's first and
// its last.  Returns the piece's units.
__device__ __forceinline__ int cursor_piece(const Cursor &c, int &b0, int &b1, bool &first, bool &last) {
  const int per = c.w.units();
  const int n = (int)min((long long)(per - c.skip), c.end - c.u);
  b0 = max(c.skip - c.w.setup, 0);
  b1 = min(c.w.nblk, c.skip + n - c.w.setup);
  first = c.skip <= c.w.setup;
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
  return c.works();
}

// where row r of the cursor's tile lies in q and o
__device__ __forceinline__ void row_place(const PagedArgs &a, const Cursor &c, int MT, int r, int &tok, int &head) {
  const unsigned g = (unsigned)c.t * MT + r, i = g / (unsigned)a.G;
  tok = c.s.qbeg + (int)i;
  head = c.h * a.G + (int)(g - i * a.G);
}

// rows of a tile of the row kernel for up to `rows` rows per key head, and its CTAs per SM
int attn_rows_tile(bool bf16_type, int D, int rows);
int attn_rows_per_sm(bool bf16_type, int D, int MT);
int attn_rows_box(bool bf16_type, int MT, int page_size);  // slots of a box of its tensor maps
cudaError_t launch_attn_rows(const PagedArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, bool bf16_type, int D, int MT,
                             int ctas, cudaStream_t st);
// items: an upper bound on the items of the call
cudaError_t launch_attn_join(const PagedArgs &a, bool bf16_type, int D, int MT, int ctas, int items, cudaStream_t st);
cudaError_t launch_attn_chunk_tc(const PagedArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, int D, int ctas,
                                 cudaStream_t st);

}  // namespace gdn
