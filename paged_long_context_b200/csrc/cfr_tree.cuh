// cfr_tree.cuh -- what the kernels of tree attention share: the call's
// parameters, the cut of a call into work, and the rows of a work item.
//
// A work item is (sequence b, kv head g, block rb of at most RB of its query
// rows); it spans the ceil(n_b / TT) token tiles of the sequence.  The tiles of
// all items, in that order, are one line of W units, and CTA i of G takes the
// units [W i / G, W (i + 1) / G): every CTA gets the same number of tiles
// whatever the lengths (an item counts as tree_item_cost tiles more than it has, for what beginning and
// ending one takes; those units come before its first tile).  A CTA's stretch covers at most one item's end, whole
// items, and one item's beginning, so it leaves at most two partials: slot 2 i
// for an item that began in an earlier CTA, 2 i + 1 for one that goes on in a
// later one.  Whole items are written out at once.  Every kernel computes the
// cut from seq_lens and q_lens itself; nothing is scheduled beforehand.
#pragma once

#include "cfr_common.cuh"

namespace cfr {

// In tiles.  Items of 256 rows end with 64 KiB to write (16 ragged sequences, 64 drafts, in bursts: 377 us with 0, 343
// with 2, 330 with 6, 342 with 10); smaller ones end sooner (5 drafts: 254 us with 2, 259 with 6).
template <int RB>
constexpr int tree_item_cost = RB == 256 ? 6 : 2;

struct TreeParams {
  const void *q;
  const uint8_t *k_pool[kFmtCount];
  const uint8_t *v_pool[kFmtCount];
  const float *scales[kFmtCount];
  long long pool_pages[kFmtCount];
  const int32_t *page_table;
  const uint8_t *page_fmt;
  const int32_t *seq_lens, *q_lens;
  const unsigned long long *mask;
  const int32_t *depths;
  const float *slopes;
  void *out;
  float *lse;
  float *part_acc;  // [2 G][RB][D]
  float *part_m;    // [2 G][RB], base-2 maxima
  float *part_l;    // [2 G][RB]
  uint32_t *err;
  int q_fmt, out_fmt, uniform_fmt;
  int batch, max_pages, Hq, Hkv, D, P, nq;
  int grid;             // CTAs that the cut is for
  int heads_each;       // query heads of every kv head, 0 when they differ
  float sigma, cap;     // softmax scale; cap (0: none)
  int16_t head_off[kMaxQHeads + 1];  // query heads of kv head g: heads[head_off[g] .. head_off[g + 1])
  int16_t heads[kMaxQHeads];
};

// Sequence b of a call: drafts, tokens (0 when its lengths are out of range), row
// blocks over all kv heads, tiles of each.
struct TreeSeq {
  int c, n;
  int blocks, tiles;
  bool bad;
};

template <int TT, int RB>
__device__ __forceinline__ int tree_blocks(const TreeParams &p, int c, int g) {
  const int cnt = p.heads_each ? p.heads_each : p.head_off[g + 1] - p.head_off[g];
  return (c * cnt + RB - 1) / RB;
}

// Units of a sequence's items, and the tile at unit `off` of an item.
template <int RB>
__device__ __forceinline__ long long tree_units(const TreeSeq &s) {
  return static_cast<long long>(s.blocks) * (s.tiles + tree_item_cost<RB>);
}
template <int RB>
__device__ __forceinline__ int tree_tile(long long off) {
  return off > tree_item_cost<RB> ? static_cast<int>(off - tree_item_cost<RB>) : 0;
}

template <int TT, int RB>
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int b) {
  TreeSeq s;
  s.n = p.seq_lens[b];
  s.c = p.q_lens ? p.q_lens[b] : p.nq;
  s.bad = s.c < 0 || s.c > p.nq;
  if (s.bad) s.c = p.nq;
  if (s.c > 0 && (s.n < s.c || s.n > static_cast<long long>(p.max_pages) * p.P)) s.bad = true;
  if (s.bad) s.n = 0;
  if (s.c == 0) {
    s.blocks = 0;
  } else if (p.heads_each) {
    s.blocks = p.Hkv * tree_blocks<TT, RB>(p, s.c, 0);
  } else {
    s.blocks = 0;
    for (int g = 0; g < p.Hkv; ++g) s.blocks += tree_blocks<TT, RB>(p, s.c, g);
  }
  s.tiles = s.n > TT ? (s.n + TT - 1) / TT : 1;
  return s;
}

// A stretch [u, end) of the line; `b` is the sequence that unit u lies in and
// `base` that sequence's first unit.
struct TreeCursor {
  long long u, end, base;
  int b;
};

// One piece of work: tiles [t0, t1) of an item.
struct TreeItem {
  int b, g, row0, rows;   // the item's rows: row0 .. row0 + rows - 1 of kv head g
  int t0, t1, tiles;
  int c, n, cnt;          // drafts and tokens of the sequence, query heads of g
  bool bad;
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

// First unit of CTA i's stretch, W i / G rounded down, from W / G and W % G.
struct TreeCut {
  long long each;
  uint32_t rest, G;
  __device__ __forceinline__ TreeCut(long long W, int grid) {
    G = static_cast<uint32_t>(grid);
    each = W >> 32 ? W / G : static_cast<uint32_t>(W) / G;
    rest = static_cast<uint32_t>(W - each * G);
  }
  __device__ __forceinline__ long long start(int i) const { return each * i + rest * static_cast<uint32_t>(i) / G; }
};

// Finds the cursor of unit range [lo(W), hi(W)): all NT threads call it, NT a multiple of 32;
// scratch holds NT / 32 + 2 values.  Returns W; `first` is the wanted unit as a function of W.
struct TreeScratch {
  long long warp[32];
  long long base;
  int b;
};

template <int TT, int RB, typename First>
__device__ __forceinline__ long long tree_find(const TreeParams &p, TreeScratch &s, int tid, int nt,
                                               First first, TreeCursor &cur) {
  // each thread sums a run of sequences; the run that holds the unit is walked again
  const int run = (p.batch + nt - 1) / nt;
  const int b0 = min(tid * run, p.batch), b1 = min(b0 + run, p.batch);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const TreeSeq q = tree_seq<TT, RB>(p, b);
    mine += tree_units<RB>(q);
  }
  long long incl = mine;
  const int lane = tid & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s.warp[tid >> 5] = incl;
  __syncthreads();
  long long before = 0, W = 0;
  for (int w = 0; w < nt / 32; ++w) {
    const long long x = s.warp[w];
    if (w < (tid >> 5)) before += x;
    W += x;
  }
  const long long u = first(W);
  long long at = before + incl - mine;
  if (u >= at && u < at + mine) {
    int b = b0;
    for (;; ++b) {
      const TreeSeq q = tree_seq<TT, RB>(p, b);
      const long long units = tree_units<RB>(q);
      if (u < at + units) break;
      at += units;
    }
    s.b = b;
    s.base = at;
  }
  __syncthreads();
  cur.u = u;
  cur.b = s.b;
  cur.base = s.base;
  return W;
}

// The next piece of the stretch that has tiles; false at its end.
template <int TT, int RB>
__device__ __forceinline__ bool tree_next(const TreeParams &p, TreeCursor &cur, TreeItem &it) {
  TreeSeq s;
  int item;
  do {
    if (cur.u >= cur.end) return false;
    s = tree_seq<TT, RB>(p, cur.b);
    while (cur.u >= cur.base + tree_units<RB>(s)) {
      cur.base += tree_units<RB>(s);
      s = tree_seq<TT, RB>(p, ++cur.b);
    }
    const int each = s.tiles + tree_item_cost<RB>;
    const long long off = cur.u - cur.base;
    item = off >> 32 ? static_cast<int>(off / each) : static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(each));
    const long long in = off - static_cast<long long>(item) * each;   // units of the item before u
    const long long to = min(static_cast<long long>(each), in + (cur.end - cur.u));
    it.t0 = tree_tile<RB>(in);
    it.t1 = tree_tile<RB>(to);
    cur.u += to - in;
  } while (it.t0 == it.t1);
  it.tiles = s.tiles;
  it.b = cur.b;
  it.c = s.c;
  it.n = s.n;
  it.bad = s.bad;
  if (p.heads_each) {
    const int per = tree_blocks<TT, RB>(p, s.c, 0);
    it.g = item / per;
    item -= it.g * per;
  } else {
    it.g = 0;
    while (item >= tree_blocks<TT, RB>(p, s.c, it.g)) item -= tree_blocks<TT, RB>(p, s.c, it.g++);
  }
  it.cnt = p.head_off[it.g + 1] - p.head_off[it.g];
  it.row0 = item * RB;
  it.rows = min(RB, s.c * it.cnt - it.row0);
  return true;
}

// Row r of kv head g's rows: draft i, query head h.
__device__ __forceinline__ void tree_row(const TreeParams &p, const TreeItem &it, int r, int &i, int &h) {
  i = r / it.cnt;
  h = p.heads[p.head_off[it.g] + r - i * it.cnt];
}

// Index of (sequence, draft, head) in q, out and lse rows.
__device__ __forceinline__ long long tree_out_row(const TreeParams &p, int b, int i, int h) {
  return (static_cast<long long>(b) * p.nq + i) * p.Hq + h;
}

// The drafts that draft i of sequence b sees, as bits.
__device__ __forceinline__ unsigned long long tree_bits(const TreeParams &p, int b, int i, int c) {
  const unsigned long long all = c >= 64 ? ~0ull : (1ull << c) - 1ull;
  const unsigned long long m = p.mask ? p.mask[static_cast<long long>(b) * p.nq + i]
                                      : (i >= 63 ? ~0ull : (1ull << (i + 1)) - 1ull);
  return m & all;
}

}  // namespace cfr
