// cfr_tree_tc.cu -- attention of a tree of drafted tokens on the 5th-generation
// tensor cores (tcgen05, accumulators and probabilities in TMEM) for bf16
// queries over bf16, FP8, int8 and int4 pages.
//
// A work item's query rows (drafts x query heads of one kv head) are the M
// dimension, 128 rows a tile; one 128-token tile of the cache is
//   S[128 rows x 128 tokens] = Q . K^T     (A, B from shared memory, K-major)
//   O[128 rows x D] += P . V               (A = P from TMEM, B = V, MN-major)
// Rows as M (the one-token decode has tokens as M) because a tree brings tens to
// hundreds of rows to a kv head: a thread then owns a whole row of S, so the
// maximum, the sum and the mask of a row need no exchange between threads, and P goes back
// to TMEM without touching shared memory.
//
// Online softmax with a lazy reference: a row's exponentials are taken against m_ref,
// which is moved (O and l rescaled) only when the row's maximum has passed it
// by more than 8 (a factor of 256, which bf16 and fp32 hold without loss), so
// O stays in TMEM for nearly every tile.  P is rounded to bf16, the type of V as
// an MMA operand; l sums the unrounded values in fp32.
//
// Quantised pages: codes are expanded to bf16 in shared memory (int8, int4 and
// E4M3 codes are all exact there); the K scale multiplies the fp32 score of its
// token, the V scale its probability.
//
// Two variants.
//  - Narrow (NM = 1): up to 64 rows of a kv head.  128 rows of Q would leave half
//    the tensor core's lanes and softmax threads idle, so the rows stand in Q
//    twice (or four times, up to 32 rows), and copy i of a row takes the i-th
//    half (quarter) of every tile's tokens: its own maximum, sum and O, with
//    zeros in P for the other tokens.  All four schedulers of the SM then share
//    the exponentials, and the copies are joined when an item ends.
//  - Wide (NM = 2): two row tiles of one K/V tile, each with a softmax warpgroup; K
//    and V are read once for 256 rows.  TMEM holds two S buffers of 64 tokens
//    for each row tile beside the two O, so a tile is taken in two steps.
// Either way the scores of a step are computed while the one before is in the softmax.
//
// Warps: warpgroup 0 = producer of K (warp 0), an MMA issuer for each row tile
// (1, 2), producer of V (3); then NM softmax warpgroups; with quantised pools one
// more that expands codes.  K and V tiles have a ring of slots each.
//  - bf16 rows are brought by TMA boxes straight into the 128-byte-swizzled
//    operand layout, quantised rows by bulk copies into their own rows' place
//    and expanded there.
//  - A V tile that reaches the drafts or the sequence's end is repaired before
//    the MMA sees it, by its producer or as it is expanded: rows that hold no token
//    become zeros, and non-finite values of drafts are taken out (they would reach, as 0 * NaN, rows that do
//    not see the draft) and added back at the end to the rows that see it.
//
// What bounds it.  64 rows of a kv head over 1M bf16 tokens: HBM in bursts of ten passes (670 us, 0.98 of the copy
// rate); sustained, the power cap lowers SM clocks to 1.4 GHz and it takes 800 to 840.  256 rows (64 drafts, 16
// ragged sequences): 331 us in bursts and 378 to 391 sustained, of 171 for the bytes and 131 for the MMAs, and no
// unit is full (tensor pipe 39 %, special functions 36 %, issue 38 %): two softmax warps a scheduler each go through
// wait, loads, exponentials and stores in turn.  Few rows over 16-token pages (5 drafts, the same batch): 258 us in
// bursts of 169, memory at half its rate and most stalls on loads; which role they belong to was not traced.
// Quantised pages: one softmax warp a scheduler, whose chain of steps takes 3.5K of the 4.9K
// clocks of a tile and is lengthened by instruction fetch, since the expansion, the softmax and the copies
// together fill the instruction cache (so hot loops are kept rolled and what is rare stands out of line; 64 rows,
// 8 x 32K tokens of tiers: 260 us, capped 280, of 92 for the bytes).  One short sequence: the latency of one
// tile's way through the roles (28 rows over 1K tokens: 18 us).
#include <cuda_bf16.h>

#include <climits>
#include <cstring>
#include <type_traits>

#include "cfr_cells.cuh"
#include "cfr_tc.cuh"
#include "cfr_tmap.cuh"
#include "cfr_tree.cuh"

namespace cfr {
namespace {

constexpr int TT = 128;        // tokens of a tile
constexpr int ITEM_RING = 8;   // items published
constexpr int MAX_PIECES = 17; // pages (of 8 tokens or more) that a tile can touch
constexpr float RESCALE_STEP = 8.f;

// How scores become probabilities.  PLAIN: scaled only.  GENERAL_SCORES: capped, less a distance, or both.
// FIXED_REFERENCE: capped scores lie within +- cap, so that the exponentials of every row can be taken against
// one number, with no maximum and a single pass over the scores: 2^(s - 10) of |s| <= 80 (in units of log2 e,
// caps up to 55) is between 2^-90 and 2^70, which leaves normal numbers for V, or the V scales of quantised
// pages, between 2^-36 and 2^28 (of 2^20 tokens that all stand at the cap).  (Eight
// sequences of 32K tiered tokens, capped at 50: 280 us, and 360 in two passes.)
enum TtMode { PLAIN, GENERAL_SCORES, FIXED_REFERENCE };
constexpr float TT_FIXED_CAP = 80.f, TT_FIXED_REF = 10.f;

// P and O of quantised pages are relative to one V scale, v_ref: the newest page's, or 1 where that is out of the
// ordinary or the reference is fixed.  A page's scale goes into the exponent of its tokens, from where their sum is
// taken back, only while its ratio to v_ref lies between FOLD_LEAST and FOLD_MOST: the smallest exponential
// that counts, 2^-90, then stays normal and the sum whole (with wider bounds, rows whose scores stood at -cap lost
// the pages of small V scales from their sums).  Other pages' scales multiply the probabilities token by
// token, behind the sum.
constexpr float TT_V_LEAST = 0x1p-20f, TT_V_MOST = 0x1p20f, TT_FOLD_LEAST = 0x1p-32f, TT_FOLD_MOST = 0x1p16f;

template <int D, int NM, bool QUANT>
struct TtCfg {
  static constexpr int RB = NM == 1 ? 64 : 256;  // rows of an item
  static constexpr int STEP = 128 / NM;          // tokens of a step
  static constexpr int STEPS = NM;               // steps of a tile
  static constexpr int ROW_TILE = 128 * D * 2;   // bytes of 128 bf16 rows: a Q tile, a K or V slot
  // slots that fit beside the queries (227 KB in all); heads of 64 have slots of half the size
  // K slots 0 .. NK - 1, then V slots: two rings, so that no barrier of a slot is shared by both producers
  static constexpr int NK = D == 128 ? 2 : 4;
  static constexpr int NV = (D == 128 ? 1 : 2) * (NM == 2 && QUANT ? 2 : 3);
  static constexpr int NS = NK + NV;
  // expanding warpgroups: K and V in turn by one where registers allow no more, else one for each
  static constexpr int LOADERS = QUANT ? (NM == 1 ? 2 : 1) : 0;
  // tiles whose description is kept, a power of two (see tt_producer)
  static constexpr int META = LOADERS == 2 && NK + NV + 1 >= 8 ? 16 : 8;
  static_assert(NK <= 4 && (LOADERS < 2 || NK + NV + 1 < META), "a tile's description outlives its readers");
  static constexpr int WGS = 1 + NM + LOADERS;
  static constexpr int THREADS = 128 * WGS;
  static constexpr int SOFTMAX_T0 = 128;
  // TMEM columns: S, two buffers of STEP for each row tile; O, 128 for each; narrow: P, two
  // buffers of its own, so that the zeros of other copies' tokens stay (wide: P over its S)
  static constexpr int TMEM_COLS = 512;
  static constexpr int S_COL = 0, O_COL = 256, P_COL = 384;
  __device__ static __forceinline__ uint32_t s_col(int m, int b) { return S_COL + (2 * m + b) * STEP; }
  __device__ static __forceinline__ uint32_t p_col(int m, int b) { return NM == 1 ? P_COL + 64 * b : s_col(m, b); }
};

struct TtMeta {
  uint32_t valid[4];          // tokens of the tile that take part
  int tin0, scaled;           // row of the first token in its page; bit 0: quantised pages, bit 1: int4 pages
  uint8_t fmt[MAX_PIECES + 3];
  float ks[MAX_PIECES], vs[MAX_PIECES];
};

// Page-table entries of a stretch of a sequence's pages, in shared memory; the next
// entries wait in registers, so that running out of the cached ones waits for nothing.
constexpr int PAGE_RUN = 64;
struct TtPages {
  int32_t id[PAGE_RUN];
  uint8_t fmt[PAGE_RUN];
};

struct TtNoMeta {
  int tin0, scaled;
};

template <int NS, int NM, bool QUANT, int META>
struct TtSmem {
  uint64_t slot_full[NS], slot_empty[NS], raw_full[NS];
  // by row tile and, where two steps can be under way, by the step's parity: a wait by
  // parity must begin no earlier than one phase before the one it is for
  uint64_t s_full[2 * NM], p_full[2 * NM], pv_done[2 * NM], q_full[NM], o_free[NM];
  uint64_t meta_full[META], drain[NM], meet, item_full[ITEM_RING], item_free[ITEM_RING];
  uint32_t tmem_base;
  int flag[NS], expand_go[2][2];
  unsigned long long nonfinite[ITEM_RING];  // of item k & 7: drafts whose V was repaired
  int direct[NS];                           // the slot's tile needs no expansion or repair
  TreeItem item[ITEM_RING];
  typename std::conditional<QUANT, TtMeta, TtNoMeta>::type meta[QUANT ? META : 1];
  uint32_t valid[META][4], v_valid[META][4];
  union {
    TtPages pages[2];
    TreeScratch scratch;   // (before the roles begin)
  };
  // K scale (times softmax scale and log2 e) and V scale of each token
  alignas(16) float ks[QUANT ? META : 1][QUANT ? TT : 4], vs[QUANT ? META : 1][QUANT ? TT : 4];
  // joining of the copies (narrow): 32 columns of O of every row, its maximum and sum
  alignas(16) float join[NM == 1 ? 128 : 1][36];
  float2 join_ml[NM == 1 ? 128 : 1];
  long long join_row[NM == 1 ? 64 : 1];
};

// D[128 x N] (+)= A (TMEM) . B (shared memory)
__device__ __forceinline__ void tt_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tt_ld32(uint32_t taddr, float *v) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tt_ld16(uint32_t taddr, float *v) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tt_st32(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tt_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tt_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// int8 codes 2i, 2i + 1 of a word -> bf16 pair: 128 + (c & 127) less 128, or less 256 where the sign bit
// is set (both terms share the exponent trick: 0x4300 is 128, 0x4380 is 256)
__device__ __forceinline__ uint32_t bf2_sub(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t i8x2_to_bf2(uint32_t w, uint32_t sel) {
  const uint32_t t = prmt(w, 0u, sel);  // (byte, 0, byte, 0)
  return bf2_sub((t & 0x007F007Fu) | 0x43004300u, (t & 0x00800080u) | 0x43004300u);
}
// int4 codes of byte i of a word whose nibbles were xored with 8: lo, hi = its low
// and high nibbles, one a byte -> bf16 pair (128 + nibble less 136)
__device__ __forceinline__ uint32_t i4x2_to_bf2(uint32_t lo, uint32_t hi, uint32_t sel) {
  return bf2_sub((prmt(lo, hi, sel) & 0x000F000Fu) | 0x43004300u, 0x43084308u);
}
__device__ __forceinline__ uint32_t e4m3x2_to_bf2(uint32_t w, int i) {
  const uint32_t h = e4m3x2_to_h2(w, i);
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  return pack_bf16(f.x, f.y);
}

// true when a bf16 pair holds a non-finite value: its exponent of ones carries into the sign's place
__device__ __forceinline__ uint32_t nonfinite_pair(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }
// clears the non-finite values of a pair
__device__ __forceinline__ uint32_t repair_pair(uint32_t w) {
  const uint32_t bad = nonfinite_pair(w) >> 15;   // bit 0 and bit 16
  return w & ~(bad * 0xFFFFu);
}

template <int D, int NM, bool QUANT>
struct TtCtx {
  using Cfg = TtCfg<D, NM, QUANT>;
  using Smem = TtSmem<Cfg::NS, NM, QUANT, Cfg::META>;
  const TreeParams &p;
  const CUtensorMap &kmap, &vmap;
  Smem &S;
  uint8_t *q, *slots;
  int box;  // rows of a TMA box: the largest power of two that divides P, at most 128
  __device__ __forceinline__ uint8_t *slot(int s) const { return slots + s * Cfg::ROW_TILE; }
};

// mbar_wait with its loop out of line, once for all roles
__device__ __noinline__ bool tt_wait_long(uint64_t *bar, uint32_t parity, uint32_t *err) {
  bool timed_out = false;
  return mbar_wait(bar, parity, err, &timed_out);
}
__device__ __forceinline__ bool tt_wait(uint64_t *bar, uint32_t parity, uint32_t *err, bool *timed_out) {
  if (*timed_out) return false;
  if (mbar_try_wait(bar, parity)) return true;
  if (tt_wait_long(bar, parity, err)) return true;
  *timed_out = true;
  return false;
}

// Item k of the CTA, published in place k & 7 by the producer of K as item k - 1 begins (walking the cut takes
// a few microseconds, which every role would spend between items); false past the last.  A place, and the
// notes of the item's repaired drafts in `nonfinite`, are used again 8 items later.  Roles that hold or
// hand on K/V slots are through by then: the producer is ahead of them by its slots and two
// steps, fewer than 8 tiles, and an item has at least one.  A softmax warpgroup holds none where its row tile has no
// rows, so those say themselves when they are through, by item_free.
template <typename Smem>
__device__ __forceinline__ bool tt_item(const TreeParams &p, Smem &S, uint32_t k, TreeItem &it, bool *timed_out) {
  const int i = k & (ITEM_RING - 1);
  if (!tt_wait(&S.item_full[i], (k / ITEM_RING) & 1u, p.err, timed_out)) return false;
  it = S.item[i];
  return it.rows > 0;
}

// place in a ring of slots, FIRST .. FIRST + N - 1
template <int FIRST, int N>
struct Ring {
  int s = FIRST;
  uint32_t ph = 0;
  __device__ __forceinline__ void step() {
    if (++s == FIRST + N) {
      s = FIRST;
      ph ^= 1u;
    }
  }
};
template <typename Cfg>
using KRing = Ring<0, Cfg::NK>;
template <typename Cfg>
using VRing = Ring<Cfg::NK, Cfg::NV>;

// Row i of a V tile before the MMA: zeros where it holds no token; non-finite
// values of a draft taken out and the draft noted.
template <int D>
__device__ __noinline__ void tt_repair_row(uint8_t *v, int i, bool valid, int draft, unsigned long long *noted) {
  bool bad = false;
#pragma unroll 4
  for (int ch = 0; ch < D / 8; ++ch) {
    uint4 *at = reinterpret_cast<uint4 *>(v + (ch >> 3) * (TT * 128) + sw128(i, ch & 7));
    if (!valid) {
      *at = make_uint4(0u, 0u, 0u, 0u);
    } else {
      const uint4 w = *at;
      if (nonfinite_pair(w.x) | nonfinite_pair(w.y) | nonfinite_pair(w.z) | nonfinite_pair(w.w)) {
        *at = make_uint4(repair_pair(w.x), repair_pair(w.y), repair_pair(w.z), repair_pair(w.w));
        bad = true;
      }
    }
  }
  if (bad) atomicOr(noted, 1ull << draft);
}

// ---- producers -----------------------------------------------------------------

// K (KV = 0) or V (KV = 1) of every tile, by one warp each (one code for both, for the
// instruction cache).  A tile is worked out before its slot is waited for; its copies are
// issued by one lane in uniform control flow (from the lanes that hold the pages, a
// copy took about 100 cycles to issue, and 16 of them a tile of 16-token pages bound the kernel).
//
// Tiles go from the newest to the oldest: with ALiBi, or any attention that favours the
// recent, the running maximum is then found at once and O is hardly ever rescaled.
//
// The description of the CTA's tile t is kept in place t mod META.  It may be overwritten by
// tile t + 8 because K's slot of tile t + 8 is free only when the scores of a
// tile t + 4 or later were issued (there are at most 4 slots of K), which is after the softmax of
// tile t handed over its P.  A warpgroup that expands V alone reads it too, and only the slots of V hold the
// others back for it: with tile t in its hands (and tiles of bf16 pages, which need no expansion, behind it), V is
// there up to tile t + NV - 1, scores are issued up to tile t + NV + 1 and K comes up to tile
// t + NK + NV + 1.  Heads of 64 have 6 slots of V there and keep 16 descriptions for it.
template <int D, int NM, bool QUANT>
__device__ void tt_producer(TtCtx<D, NM, QUANT> &c, TreeCursor &cur, bool *timed_out, const int KV) {
  using Cfg = TtCfg<D, NM, QUANT>;
  const TreeParams &p = c.p;
  const int lane = threadIdx.x & 31;
  TtPages &pc = c.S.pages[KV];
  uint32_t lead;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(lead));
  const int r_first = KV ? Cfg::NK : 0, r_end = KV ? Cfg::NS : Cfg::NK;
  int slot_i = r_first;
  uint32_t slot_ph = 0;
  uint32_t raw_mask = 0, used = 0;   // slots filled through raw_full; slots filled at all
  uint32_t phase_of = 0;             // the phase each was filled in
  uint32_t tile = 0, k = 0;
  const int P = p.P;
  // (bf16 pages only) a V tile whose copies are under way and that has to be repaired when they
  // are done: the next tile's copies are issued first
  int pend_slot = -1, pend_j0 = 0, pend_mi = 0, pend_item = 0;
  uint32_t raw_ph = 0;   // the phase that each slot's raw_full is in
  int pre = 0;
  const auto repair = [&]() {
    if (QUANT || pend_slot < 0) return;
    tt_wait(&c.S.raw_full[pend_slot], (raw_ph >> pend_slot) & 1u, p.err, timed_out);
    if (__any_sync(0xffffffffu, *timed_out)) {
      *timed_out = true;
      return;
    }
    raw_ph ^= 1u << pend_slot;
    raw_mask &= ~(1u << pend_slot);
    used &= ~(1u << pend_slot);
#pragma unroll 1
    for (int i = lane; i < TT; i += 32) {
      const bool valid = (c.S.v_valid[pend_mi][i >> 5] >> (i & 31)) & 1u;
      if (!valid || pend_j0 + i >= pre)
        tt_repair_row<D>(c.slot(pend_slot), i, valid, pend_j0 + i - pre, &c.S.nonfinite[pend_item]);
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.S.slot_full[pend_slot]);
    pend_slot = -1;
  };
  // (the producer of K) the CTA's next item to the other roles
  uint32_t published = 0;
  const auto publish = [&]() {
    const int i = published & (ITEM_RING - 1);
    if (published >= ITEM_RING) {
      tt_wait(&c.S.item_free[i], (published / ITEM_RING - 1) & 1u, p.err, timed_out);
      if (__any_sync(0xffffffffu, *timed_out)) {
        *timed_out = true;
        return;
      }
    }
    if (lane == 0) {
      TreeItem x;
      if (!tree_next<TT, Cfg::RB>(p, cur, x)) x.rows = 0;
      c.S.item[i] = x;
      mbar_arrive(&c.S.item_full[i]);
    }
    ++published;
  };
  for (;; ++k) {
    if (KV == 0 && published == k) publish();   // (the first)
    TreeItem item;
    const bool some = tt_item(p, c.S, k, item, timed_out);
    if (!__all_sync(0xffffffffu, some)) break;
    const TreeItem it = item;
    // (here and not by the warps that expand V: tiles that need no expansion do not wait for those)
    if (KV == 1 && lane == 0) c.S.nonfinite[k & (ITEM_RING - 1)] = 0ull;
    if (KV == 0 && lane == 0 && it.bad) set_err(p.err, CFR_DEVERR_SEQ_LEN);
    pre = it.n - it.c;
    const long long table = static_cast<long long>(it.b) * p.max_pages;
    // pages [lo, lo + PAGE_RUN) of the sequence are cached, [nlo, nlo + PAGE_RUN) wait in registers
    const int pg_first = it.t0 * TT / P;
    int lo = INT_MAX, nlo = 0;
    int32_t nid[PAGE_RUN / 32];
    uint8_t nfmt[PAGE_RUN / 32];
    const auto fetch = [&](int from) {   // pages from .. from + PAGE_RUN - 1, those of the item
#pragma unroll
      for (int i = 0; i < PAGE_RUN / 32; ++i) {
        const int pg = from + 32 * i + lane;
        if (pg >= pg_first && static_cast<long long>(pg) * P < it.n) {
          nid[i] = p.page_table[table + pg];
          nfmt[i] = p.page_fmt ? p.page_fmt[table + pg] : static_cast<uint8_t>(p.uniform_fmt);
        }
      }
    };
    for (int t = it.t1 - 1; t >= it.t0; --t, ++tile) {
      const int j0 = t * TT, rows = max(0, min(TT, it.n - j0));
      const int pg0 = j0 / P, tin0 = j0 - pg0 * P;
      const int npiece = rows > 0 ? (tin0 + rows + P - 1) / P : 0;
      if (npiece > 0 && pg0 < lo) {
        if (lo == INT_MAX) {
          nlo = pg0 + npiece - PAGE_RUN;
          fetch(nlo);
        }
        lo = nlo;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < PAGE_RUN / 32; ++i) {
          pc.id[32 * i + lane] = nid[i];
          pc.fmt[32 * i + lane] = nfmt[i];
        }
        __syncwarp();
        // the next run ends where this one can first fall short: at the pages of one more tile
        nlo = lo + MAX_PIECES - PAGE_RUN;
        fetch(nlo);
      }
      bool ok = false;
      int fmt = 0;
      long long sub = 0;
      if (lane < npiece) {
        fmt = pc.fmt[pg0 + lane - lo];
        const long long id = pc.id[pg0 + lane - lo];
        const bool known = fmt < kFmtCount;
        const bool pool = known && p.k_pool[known ? fmt : 0];
        ok = pool && id >= 0 && id < p.pool_pages[known ? fmt : 0];
        if (!ok && KV == 0) set_err(p.err, !known ? CFR_DEVERR_PAGE_FMT : !pool ? CFR_DEVERR_POOL : CFR_DEVERR_PAGE_ID);
        sub = id * p.Hkv + it.g;
      }
      const bool quant = QUANT && ok && is_quantised(fmt);
      const bool any_quant = QUANT && __any_sync(0xffffffffu, quant);
      const bool any4 = QUANT && __any_sync(0xffffffffu, quant && fmt == CFR_FMT_I4);
      float2 sc = make_float2(1.f, 1.f);
      if (QUANT && quant && KV == 0) sc = *reinterpret_cast<const float2 *>(p.scales[fmt] + sub * 2);
      // this lane's page: tile rows [a, z)
      const int a = lane == 0 ? 0 : min(rows, lane * P - tin0);
      const int z = min(rows, (lane + 1) * P - tin0);
      const int boxes = (z - a + c.box - 1) / c.box;
      const uint32_t mine = !ok ? 0u : quant ? static_cast<uint32_t>((z - a) * row_bytes(fmt, D))
                                             : static_cast<uint32_t>(boxes * c.box * D * 2);
      const uint32_t bytes = __reduce_add_sync(0xffffffffu, mine);
      const uint32_t okb = __ballot_sync(0xffffffffu, ok);
      // tokens of valid pages: lane w holds those of 32 w on
      uint32_t valid = 0xFFFFFFFFu;
      const bool full = rows == TT && okb == (0xFFFFFFFFu >> (32 - npiece));
      if (!full) {
#pragma unroll 1
        for (int w = 0; w < 4; ++w) {
          const int x = max(a - 32 * w, 0), y = min(z - 32 * w, 32);
          const uint32_t any = __reduce_or_sync(0xffffffffu, ok && x < y ? (0xFFFFFFFFu >> (32 - (y - x))) << x : 0u);
          if (lane == w) valid = any;
        }
      }
      const int mi = tile & (Cfg::META - 1);
      const bool direct = !any_quant && (KV == 0 || (full && j0 + TT <= pre));
      tt_wait(&c.S.slot_empty[slot_i], slot_ph ^ 1u, p.err, timed_out);
      if (__any_sync(0xffffffffu, *timed_out)) {
        *timed_out = true;
        break;
      }
      uint64_t *done = direct ? &c.S.slot_full[slot_i] : &c.S.raw_full[slot_i];
      if (KV == 0) {
        if constexpr (QUANT) if (lane < npiece) {
          c.S.meta[mi].fmt[lane] = ok ? static_cast<uint8_t>(fmt) : 255;
          c.S.meta[mi].ks[lane] = sc.x;
          c.S.meta[mi].vs[lane] = sc.y;
        }
        if (QUANT && lane == 0) {
          c.S.meta[mi].tin0 = tin0;
          c.S.meta[mi].scaled = any_quant ? (any4 ? 3 : 1) : 0;
        }
      }
      if (lane < 4) (KV == 0 ? c.S.valid : c.S.v_valid)[mi][lane] = valid;
      if (lane == 0) c.S.direct[slot_i] = direct;
      __syncwarp();
      if (lane == 0) {
        if (KV == 0 && !QUANT) mbar_arrive(&c.S.meta_full[mi]);
        // a tile that needs nothing is shown to the expanding warps all the same, in order
        if (QUANT && direct) mbar_arrive(&c.S.raw_full[slot_i]);
        mbar_arrive_expect_tx(done, bytes);
      }
      __syncwarp();
      used |= 1u << slot_i;
      raw_mask = direct ? raw_mask & ~(1u << slot_i) : raw_mask | (1u << slot_i);
      const bool ph_of = QUANT || direct ? slot_ph : (raw_ph >> slot_i) & 1u;
      phase_of = ph_of ? phase_of | (1u << slot_i) : phase_of & ~(1u << slot_i);
      const CUtensorMap *map = KV ? &c.vmap : &c.kmap;
      uint8_t *const slot = c.slot(slot_i);
#pragma unroll 1
      for (int f = 0; f < npiece; ++f) {
        if (!((okb >> f) & 1u)) continue;
        const long long sub_f = __shfl_sync(0xffffffffu, sub, f);
        const int a_f = f == 0 ? 0 : f * P - tin0, in_page = f == 0 ? tin0 : 0;
        uint8_t *dst = slot + a_f * 128;
        if (QUANT && any_quant) {
          const int fmt_f = __shfl_sync(0xffffffffu, fmt, f);
          const uint32_t mine_f = __shfl_sync(0xffffffffu, mine, f);
          if (is_quantised(fmt_f)) {
            const uint8_t *pool = KV ? p.v_pool[fmt_f] : p.k_pool[fmt_f];
            // (places: see tt_expand)
            if (lead)
              bulk_g2s(D == 128 && fmt_f == CFR_FMT_I4 ? dst + TT * 128 : dst,
                       pool + (sub_f * P + in_page) * row_bytes(fmt_f, D), mine_f, done);
            continue;
          }
        }
        int y = static_cast<int>(sub_f * P + in_page);
        const int z_f = min(rows, (f + 1) * P - tin0);
#pragma unroll 1
        for (int x = a_f; x < z_f; x += c.box, y += c.box, dst += c.box * 128)
          if (lead)
#pragma unroll
            for (int half = 0; half < D / 64; ++half) tma_load_2d(dst + half * (TT * 128), map, half * 64, y, done);
      }
      repair();
      if (*timed_out) break;
      if (!QUANT && !direct) {
        pend_slot = slot_i;
        pend_j0 = j0;
        pend_mi = mi;
        pend_item = k & (ITEM_RING - 1);
      }
      if (KV == 0 && t == it.t1 - 1) publish();   // the item after this one, once this one is under way
      if (++slot_i == r_end) {
        slot_i = r_first;
        slot_ph ^= 1u;
      }
    }
    if (!*timed_out) repair();   // (the drafts are this item's)
    if (*timed_out) break;
  }
  if (*timed_out && lane == 0) {
    // leave no copy in flight
    for (int s = 0; s < Cfg::NS; ++s) {
      bool late = false;
      if ((used >> s) & 1u)
        tt_wait((raw_mask >> s) & 1u ? &c.S.raw_full[s] : &c.S.slot_full[s], (phase_of >> s) & 1u, p.err, &late);
    }
  }
}

// ---- expansion -------------------------------------------------------------------

// Eight bytes of codes a 32-bit word at a time: int8 and E4M3 codes give two bf16 words
// a word, int4 codes four.
template <int FMT>
__device__ __forceinline__ void expand_word(uint32_t w, uint32_t *o) {
  if constexpr (FMT == CFR_FMT_I8) {
    o[0] = i8x2_to_bf2(w, 0x4140u);
    o[1] = i8x2_to_bf2(w, 0x4342u);
  } else if constexpr (FMT == CFR_FMT_FP8) {
    o[0] = e4m3x2_to_bf2(w, 0);
    o[1] = e4m3x2_to_bf2(w, 1);
  } else {
    const uint32_t x = w ^ 0x88888888u;
    const uint32_t lo = x & 0x0F0F0F0Fu, hi = (x >> 4) & 0x0F0F0F0Fu;
    o[0] = i4x2_to_bf2(lo, hi, 0x4400u);
    o[1] = i4x2_to_bf2(lo, hi, 0x5511u);
    o[2] = i4x2_to_bf2(lo, hi, 0x6622u);
    o[3] = i4x2_to_bf2(lo, hi, 0x7733u);
  }
}

// 64 values of a row, N 16-byte pieces of codes in the order (x + turn) mod N, into one half
// of a slot; `row` is the row's place there and `swz` its swizzle, (row mod 8) * 16.
template <int FMT, int N>
__device__ __forceinline__ void expand_half(uint32_t row, uint32_t swz, int turn, uint4 (&raw)[N]) {
  // in two rounds of half the pieces, the second's moved to the first's registers: unrolled over all of them the code of
  // the formats fell out of the instruction cache
#pragma unroll 1
  for (int x0 = 0; x0 < N; x0 += N / 2) {
#pragma unroll
  for (int x = 0; x < N / 2; ++x) {
    const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
    const uint32_t at = static_cast<uint32_t>((x0 + x + turn) & (N - 1)) * (128 / N);   // its first byte in the row
#pragma unroll
    for (int y = 0; y < 8 / N; ++y) {   // 16 bytes of bf16
      uint32_t o[4];
      if constexpr (N == 4) {
        expand_word<FMT>(w[2 * y], o);
        expand_word<FMT>(w[2 * y + 1], o + 2);
      } else {
        expand_word<FMT>(w[y], o);
      }
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((at + 16 * y) ^ swz)), "r"(o[0]), "r"(o[1]),
                   "r"(o[2]), "r"(o[3])
                   : "memory");
    }
  }
#pragma unroll
  for (int x = 0; x < N / 2; ++x) raw[x] = raw[x + N / 2];
  }
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// Expansion (and V repair) of caches with quantised pages: thread i owns row i.
// `which`: K slots (0), V slots (1) or both in turn (2).  It takes part in the release
// of every slot, so that it is never a phase behind a slot's barrier.  What bounds it is
// the latency of one warp's chain on each scheduler, hence a warpgroup each for K and V.
template <int D, int NM>
__device__ void tt_expand(TtCtx<D, NM, true> &c, bool *timed_out, const int which) {
  using Cfg = TtCfg<D, NM, true>;
  const TreeParams &p = c.p;
  const int i = threadIdx.x & 127;
  const int bar = 1 + (which & 1);
  KRing<Cfg> kr;
  VRing<Cfg> vr;
  uint32_t tile = 0;
  for (uint32_t k = 0;; ++k) {
    // one thread waits, the barrier hands on its outcome
    int *go = &c.S.expand_go[which & 1][k & 1];
    if (i == 0) *go = tt_wait(&c.S.item_full[k & (ITEM_RING - 1)], (k / ITEM_RING) & 1u, p.err, timed_out) ? 1 : 0;
    named_sync(bar, 128);
    if (!*go) *timed_out = true;
    TreeItem it;
    if (!tt_item(p, c.S, k, it, timed_out)) return;
    const int pre = it.n - it.c;
    for (int t = it.t1 - 1; t >= it.t0; --t, ++tile) {
      const int mi = tile & (Cfg::META - 1);
      const TtMeta &m = c.S.meta[mi];
#pragma unroll 1
      for (int kv = which == 1 ? 1 : 0; kv < (which == 0 ? 1 : 2); ++kv) {
        const int slot = kv ? vr.s : kr.s;
        const uint32_t ph = kv ? vr.ph : kr.ph;
        if (i == 0) {
          // (the description of the tile is K's; the warpgroup of V has it by meta_full)
          bool got = which != 1 || tt_wait(&c.S.meta_full[mi], (tile / Cfg::META) & 1u, p.err, timed_out);
          got = got && tt_wait(&c.S.raw_full[slot], ph, p.err, timed_out);
          c.S.flag[slot] = got ? 1 : 0;
        }
        named_sync(bar, 128);
        if (!c.S.flag[slot]) {
          *timed_out = true;
          return;
        }
        (void)mbar_try_wait(&c.S.raw_full[slot], ph);
        if (which == 1) (void)mbar_try_wait(&c.S.meta_full[mi], (tile / Cfg::META) & 1u);
        const bool direct = c.S.direct[slot];
        const bool any4 = m.scaled & 2;   // 4-bit rows among the tile's
        const bool valid = (c.S.valid[mi][i >> 5] >> (i & 31)) & 1u;
        const int pc = p.P >= TT ? (m.tin0 + i >= p.P ? 1 : 0) : (m.tin0 + i) / p.P;
        const int fmt = valid ? m.fmt[pc] : 255;
        if (kv == 0) {
          c.S.ks[mi][i] = valid ? m.ks[pc] * (p.sigma * kLog2e) : 0.f;
          c.S.vs[mi][i] = valid ? m.vs[pc] : 0.f;
        }
        if (!direct) {
          uint8_t *op = c.slot(slot);
          const int a = pc == 0 ? 0 : pc * p.P - m.tin0;   // first row of the row's page
          const bool eight = fmt == CFR_FMT_I8 || fmt == CFR_FMT_FP8, four = fmt == CFR_FMT_I4;
          const int draft = t * TT + i - pre;
          // 64 values at a time (a row of one half of the slot); codes are read in an order that
          // spreads a warp's lanes over the banks
          const uint32_t base = smem_u32(op), row = base + i * 128, swz = (i & 7) * 16;
          if (D == 128) {
            // 8-bit rows lie where the row's first half goes, so each thread overwrites its own; 4-bit rows
            // lie in the second half's place of their page's rows, which is written once all were read
            const uint32_t src = base + TT * 128 + a * 128 + (i - a) * 64;
#pragma unroll 1
            for (int hh = 1; hh >= 0; --hh) {
              if (eight) {
                uint4 raw[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) raw[x] = ld_shared16(row + hh * 64 + 16 * ((x + i) & 3));
                if (fmt == CFR_FMT_I8)
                  expand_half<CFR_FMT_I8, 4>(row + hh * (TT * 128), swz, i, raw);
                else
                  expand_half<CFR_FMT_FP8, 4>(row + hh * (TT * 128), swz, i, raw);
              }
              if (any4) {
                const int h4 = hh ^ 1;   // first half first
                uint4 raw[2];
                if (four) {
#pragma unroll
                  for (int x = 0; x < 2; ++x) raw[x] = ld_shared16(src + h4 * 32 + 16 * ((x + (i >> 1)) & 1));
                }
                if (h4 == 1) named_sync(bar, 128);
                if (four) expand_half<CFR_FMT_I4, 2>(row + h4 * (TT * 128), swz, i >> 1, raw);
              }
            }
          } else {
            uint4 raw[4], raw4[2];
            const uint32_t src = base + a * 128 + (i - a) * (eight ? D : D / 2);
            if (eight) {
#pragma unroll
              for (int x = 0; x < 4; ++x) raw[x] = ld_shared16(src + 16 * ((x + i) & 3));
            } else if (four) {
#pragma unroll
              for (int x = 0; x < 2; ++x) raw4[x] = ld_shared16(src + 16 * ((x + (i >> 1)) & 1));
            }
            named_sync(bar, 128);  // every row is in registers before any is written
            if (fmt == CFR_FMT_I8) expand_half<CFR_FMT_I8, 4>(row, swz, i, raw);
            if (fmt == CFR_FMT_FP8) expand_half<CFR_FMT_FP8, 4>(row, swz, i, raw);
            if (four) expand_half<CFR_FMT_I4, 2>(row, swz, i >> 1, raw4);
          }
          // a V row without a token, or of a draft (int8 and int4 codes are finite)
          if (kv == 1 && (eight || four ? fmt == CFR_FMT_FP8 && draft >= 0 : !valid || draft >= 0))
            tt_repair_row<D>(op, i, valid, draft, &c.S.nonfinite[k & (ITEM_RING - 1)]);
          fence_async_smem();
        }
        named_sync(bar, 128);
        if (i == 0) {
          if (!direct) mbar_arrive(&c.S.slot_full[slot]);
          if (kv == 0) mbar_arrive(&c.S.meta_full[mi]);
          mbar_arrive(&c.S.slot_empty[slot]);
        }
        if (kv)
          vr.step();
        else
          kr.step();
      }
    }
  }
}

// ---- MMA issue ------------------------------------------------------------------

// The MMAs of row tile m, by one warp (two row tiles: two warps, so that neither
// waits for the other's softmax).  The whole warp walks the steps and one lane
// issues: with control flow and operands the same in every lane, descriptors
// stay in uniform registers (from a lone lane each MMA took 80 to 100 cycles to
// issue, for 32 to 64 of tensor time).
template <int D, int NM, bool QUANT>
__device__ void tt_issue(TtCtx<D, NM, QUANT> &c, bool *timed_out, int m_) {
  using Cfg = TtCfg<D, NM, QUANT>;
  const TreeParams &p = c.p;
  const auto same = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
  const int m = NM == 1 ? 0 : same(m_);
  const uint32_t tmem = same(c.S.tmem_base);
  const uint32_t qa = same(smem_u32(c.q)) + m * Cfg::ROW_TILE, sa = same(smem_u32(c.slots));
  uint32_t lead;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(lead));
  constexpr uint32_t qk_desc = tc_idesc(1, 0, 0, Cfg::STEP), pv_desc = tc_idesc(1, 0, 1, D);
  constexpr int STEP_BYTES = Cfg::STEP * 128;     // of a step's rows in each 64-column half of a slot
  KRing<Cfg> kr;
  VRing<Cfg> vr;
  uint32_t cnt = 0, items = 0;                    // steps and items of the row tile so far
  const auto wait = [&](uint64_t *bar, uint32_t par) {
    tt_wait(bar, par, p.err, timed_out);
    return __all_sync(0xffffffffu, !*timed_out) != 0;
  };
  bool go = true;
  for (uint32_t k = 0; go; ++k) {
    TreeItem item;
    const bool some = tt_item(p, c.S, k, item, timed_out);
    if (!__all_sync(0xffffffffu, some)) break;
    const int steps = same((item.t1 - item.t0) * Cfg::STEPS);
    if (NM == 2 && same(item.rows) <= 128 * m) {
      // no rows here: the slots go by
      for (int s = 0; s < steps / Cfg::STEPS && go; ++s) {
        go = wait(&c.S.slot_full[kr.s], kr.ph);
        if (go && lead) mbar_arrive(&c.S.slot_empty[kr.s]);
        if (go) go = wait(&c.S.slot_full[vr.s], vr.ph);
        if (go && lead) mbar_arrive(&c.S.slot_empty[vr.s]);
        kr.step();
        vr.step();
      }
      continue;
    }
    go = wait(&c.S.q_full[m], items & 1u);
    if (!go) break;
    // step -1 only issues the scores of step 0
    for (int s = -1; s < steps; ++s) {
      if (s + 1 < steps) {
        const int h = (s + 1) % Cfg::STEPS;
        if (h == 0) go = wait(&c.S.slot_full[kr.s], kr.ph);
        if (!go) break;
        tc_fence_after();
        const uint32_t n = cnt + (s < 0 ? 0 : 1);
        const uint32_t d = tmem + Cfg::s_col(m, n & 1);
        const uint64_t a = tc_sdesc(qa, 16, 1024, 2);
        const uint64_t b = tc_sdesc(sa + kr.s * Cfg::ROW_TILE + h * STEP_BYTES, 16, 1024, 2);
        if (lead) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t off = ((k >> 2) * (TT * 128) + (k & 3) * 32) >> 4;
            tc_mma(d, a + off, b + off, qk_desc, k > 0 ? 1u : 0u);
          }
          tc_commit(&c.S.s_full[2 * m + (n & 1)]);
          if (h == Cfg::STEPS - 1) tc_commit(&c.S.slot_empty[kr.s]);
        }
        if (h == Cfg::STEPS - 1) kr.step();
      }
      if (s < 0) continue;
      const int h = s % Cfg::STEPS, b = cnt & 1;
      if (h == 0) go = wait(&c.S.slot_full[vr.s], vr.ph);
      if (go && s == 0) go = wait(&c.S.o_free[m], (items & 1u) ^ 1u);
      if (go) go = wait(&c.S.p_full[2 * m + b], (cnt >> 1) & 1u);
      if (!go) break;
      tc_fence_after();
      const uint32_t d = tmem + Cfg::O_COL + m * 128, a = tmem + Cfg::p_col(m, b);
      const uint64_t v = tc_sdesc(sa + vr.s * Cfg::ROW_TILE + h * STEP_BYTES, TT * 128, 1024, 2);
      if (lead) {
#pragma unroll
        for (int k = 0; k < Cfg::STEP / 16; ++k)
          tt_mma_ts(d, a + k * 8, v + static_cast<uint64_t>(k * 2048 >> 4), pv_desc, s > 0 || k > 0 ? 1u : 0u);
        tc_commit(&c.S.pv_done[2 * m + b]);
        if (h == Cfg::STEPS - 1) tc_commit(&c.S.slot_empty[vr.s]);
      }
      ++cnt;
      if (h == Cfg::STEPS - 1) vr.step();
    }
    ++items;
  }
  // nothing of the tensor cores may be in flight when TMEM is freed
  if (lead) tc_commit(&c.S.drain[m]);
  bool late = false;
  tt_wait(&c.S.drain[m], 0, p.err, &late);
}

// ---- softmax ---------------------------------------------------------------------

struct TtRow {
  unsigned long long bits;   // drafts that the row sees
  long long out_row;
  float slope;               // times log2 e
  int pos;
  int row, copy, width;      // row of the item, its copy, tokens of a step that the copy takes
  bool real;
};

// This thread's row of the item.
template <int D, int NM, bool GENERAL>
__device__ __forceinline__ void tt_row(const TreeParams &p, const TreeItem &it, int m, int r, TtRow &w) {
  if (NM == 1) {
    const int lg = it.rows <= 32 ? 5 : 6;   // four copies of 32 rows, or two of 64
    w.row = r & ((1 << lg) - 1);
    w.copy = r >> lg;
    w.width = 1 << lg;
  } else {
    w.row = m * 128 + r;
    w.copy = 0;
    w.width = 128 / NM;
  }
  w.real = w.row < it.rows;
  w.bits = 0;
  w.out_row = 0;
  w.slope = 0.f;
  w.pos = 0;
  if (w.real) {
    int i, h;
    tree_row(p, it, it.row0 + w.row, i, h);
    w.bits = tree_bits(p, it.b, i, it.c);
    w.out_row = tree_out_row(p, it.b, i, h);
    if (GENERAL && p.slopes) {
      w.slope = p.slopes[h] * kLog2e;
      w.pos = it.n - it.c + (p.depths ? p.depths[static_cast<long long>(it.b) * p.nq + i] : i);
    }
  }
}

// The row's query into the A operand (rows past the item's are zeros), asynchronously;
// tt_show_q makes it the tensor cores' and says so.
template <int D, int NM, bool QUANT>
__device__ __forceinline__ void tt_load_q(TtCtx<D, NM, QUANT> &c, int m, int r, const TtRow &w) {
  const uint32_t q = smem_u32(c.q + m * TtCfg<D, NM, QUANT>::ROW_TILE);
  const uint8_t *src = static_cast<const uint8_t *>(c.p.q) + w.out_row * (D * 2);
  const uint32_t bytes = w.real ? 16u : 0u;   // of 16: the rest is zeros
#pragma unroll
  for (int ch = 0; ch < D / 8; ++ch)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(q + (ch >> 3) * (TT * 128) + sw128(r, ch & 7)),
                 "l"(src + 16 * ch), "r"(bytes)
                 : "memory");
}
template <int D, int NM, bool QUANT>
__device__ __forceinline__ void tt_show_q(TtCtx<D, NM, QUANT> &c, int m) {
  asm volatile("cp.async.wait_all;" ::: "memory");
  fence_async_smem();
  mbar_arrive(&c.S.q_full[m]);
}

// Values of drafts that the MMA was not shown, back into the rows of O in TMEM (`noted`: the
// drafts, for this thread's row, whose tokens from `first` on, `width` of a tile, are its copy's: another copy's weight
// beside the draft's may be 0, and its 0 * infinity NaN).  Called by whole warps.
template <int D>
__device__ __noinline__ void tt_add_back(const TreeParams &p, const TreeItem &it, unsigned long long noted, int first, int width,
                                         uint32_t o_at) {
#pragma unroll 1
  for (int ch = 0; ch < D / 16; ++ch) {
    float o[16];
    tt_ld16(o_at + 16 * ch, o);
    tc_wait_ld();
#pragma unroll 1
    for (int d = 0; d < it.c; ++d) {
      if (!((noted >> d) & 1ull)) continue;
      const int j = it.n - it.c + d;
      if (static_cast<uint32_t>((j & (TT - 1)) - first) >= static_cast<uint32_t>(width)) continue;
      const long long cell = static_cast<long long>(it.b) * p.max_pages + j / p.P;
      const int fmt = p.page_fmt ? p.page_fmt[cell] : p.uniform_fmt;
      const uint8_t *v = p.v_pool[fmt] +
                         ((p.page_table[cell] * static_cast<long long>(p.Hkv) + it.g) * p.P + j % p.P) * row_bytes(fmt, D);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float y = fmt == CFR_FMT_BF16
                            ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(v)[16 * ch + i]) << 16)
                            : e4m3_at(v[16 * ch + i], 0);
        if (!(fabsf(y) < INFINITY)) o[i] += y;
      }
    }
    tt_st16(o_at + 16 * ch, reinterpret_cast<const uint32_t *>(o));
  }
  tt_wait_st();
}

// The 16 values of each of four neighbouring lanes' rows, exchanged so that lane j holds values 4 j .. 4 j + 3
// of all four rows (o[4 k ..]: row k).  Four lanes then write 64 bytes of a row; a lane writing
// its own row touches a line for itself, and the lines of an item took longer than its tiles' exponentials.
__device__ __forceinline__ void tt_turn4(float (&o)[16], int lane) {
#pragma unroll
  for (int step = 2; step >= 1; step >>= 1) {
    const bool up = lane & step;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (b & step) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float &lo = o[4 * b + i], &hi = o[4 * (b + step) + i];
        const float got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, step);
        if (up)
          lo = got;
        else
          hi = got;
      }
    }
  }
}

// N finished output values of a row (or, where `part`, of its partial) from column col on
template <int N>
__device__ __forceinline__ void tt_put(const TreeParams &p, bool part, long long row, int col, const float *o) {
  if (part || p.out_fmt == CFR_FMT_F32) {
    float4 *dst = reinterpret_cast<float4 *>((part ? p.part_acc : static_cast<float *>(p.out)) + row * p.D + col);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  } else {
    uint2 *dst = reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + row * p.D + col);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) dst[i] = make_uint2(pack_bf16(o[4 * i], o[4 * i + 1]), pack_bf16(o[4 * i + 2], o[4 * i + 3]));
  }
}

// Caps: c2 tanh(u) of u = s / cap, c2 = cap log2 e (scores are in units of log2 e from here on).
// Up to |u| = 3/4 tanh(u) = u + u z q(z), z = u^2, q of degree 4 with the least greatest relative
// error of the whole (2^-24.7 with its coefficients in fp32, found by exchange): multiply-adds, where the closed form takes two of the 16
// special functions a clock and SM, three with the exponential that follows (the ragged batch of 64 drafts,
// capped at 50: 576 us with the closed form, 497 with this).
constexpr float TT_CAP_NEAR = 0.75f;
__device__ __forceinline__ float2 tt_cap_near(float2 u, float c2) {
  const float2 z = mul2(u, u), w = mul2(u, make_float2(c2, c2));
  float2 q = make_float2(-0.0047694905661046505f, -0.0047694905661046505f);
  q = fma2(q, z, make_float2(0.019664913415908813f, 0.019664913415908813f));
  q = fma2(q, z, make_float2(-0.0533902570605278f, -0.0533902570605278f));
  q = fma2(q, z, make_float2(0.13326521217823029f, 0.13326521217823029f));
  q = fma2(q, z, make_float2(-0.3333306908607483f, -0.3333306908607483f));
  return fma2(mul2(w, z), q, w);
}
// c2 - 2 c2 / (1 + e^(2 u)), off by 2^-22 of c2
__device__ __forceinline__ float tt_cap_far(float u, float c2) {
  return fmaf(-2.f * c2, rcp_approx(1.f + exp2_approx(u * (2.f * kLog2e))), c2);
}

// Finishes, in TMEM, the scores of a step that has tokens which a row does not see.  Out
// of line and rolled: the roles of the kernel share the SM's instruction cache, and
// with these paths inside the loop its hit rate fell to 76 % and fetching
// instructions bound the kernel (a step took 2.5 times as long).
template <bool GENERAL>
__device__ __noinline__ void tt_masked(const TreeParams &p, uint32_t s_at, int width, unsigned long long seen,
                                       const float *ks, float scale, float slope, int pos, int pre, int off, int c, int b) {
  const float to_u = 1.f / (p.cap * kLog2e), c2 = p.cap * kLog2e;
#pragma unroll 1
  for (int ch = 0; ch < width; ch += 16) {
    float x[16];
    tt_ld16(s_at + ch, x);
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int d = ch + i - off;   // draft
      float y = x[i] * (ks ? ks[ch + i] : scale);
      if (GENERAL && p.cap > 0.f) {
        const float u = y * to_u;
        y = fabsf(u) <= TT_CAP_NEAR ? tt_cap_near(make_float2(u, u), c2).x : tt_cap_far(u, c2);
      }
      if (GENERAL && p.slopes) {
        int far = pre + d - pos;
        if (d >= 0 && d < c && p.depths) far = pre + p.depths[static_cast<long long>(b) * p.nq + d] - pos;
        y = fmaf(slope, static_cast<float>(far), y);
      }
      x[i] = (seen >> (ch + i)) & 1ull ? y : -INFINITY;
    }
    tt_st16(s_at + ch, reinterpret_cast<const uint32_t *>(x));
  }
  tt_wait_st();
}

template <int D, int NM, bool QUANT, int MODE>
__device__ void tt_softmax(TtCtx<D, NM, QUANT> &c, bool *timed_out) {
  using Cfg = TtCfg<D, NM, QUANT>;
  constexpr bool GENERAL = MODE != PLAIN, FIXED = MODE == FIXED_REFERENCE;
  const TreeParams &p = c.p;
  const int m = NM == 2 ? (threadIdx.x - Cfg::SOFTMAX_T0) >> 7 : 0;
  const int r = threadIdx.x & 127;
  const uint32_t lanes = c.S.tmem_base + (static_cast<uint32_t>(r & 96) << 16);   // this warp's TMEM lanes
  const uint32_t o_at = lanes + Cfg::O_COL + m * 128;
  const float scale = p.sigma * kLog2e;
  // caps: c2 tanh(s / cap), s / cap in units of log2 e / 2 being the score times cap_k1 (see tt_cap_far)
  const float c2 = p.cap * kLog2e, cap_k1 = GENERAL ? 2.f / p.cap : 0.f;
  // scores that a thread holds at once: a step's 64 where the code for them fits the instruction cache beside
  // the other roles (in registers throughout: 1M tokens 764 us against 865), 32 with the expansion of codes
  constexpr int CH = QUANT ? 32 : 64;
  uint32_t cnt = 0, tile = 0, next_k = 0;   // steps of this row tile, tiles of the CTA, items read
  uint32_t met = 0;                    // meetings of the warpgroup's threads so far
  int zeroed = 0;                      // (narrow) the width for which P's other columns are zeros
  // every wait's outcome is the warp's: TMEM instructions are for whole warps
  const auto wait = [&](uint64_t *bar, uint32_t par) {
    tt_wait(bar, par, p.err, timed_out);
    if (__any_sync(0xffffffffu, *timed_out)) *timed_out = true;
    return !*timed_out;
  };
  // all threads of the warpgroup (a named barrier would have no time limit)
  const auto meet = [&]() {
    mbar_arrive(&c.S.meet);
    return wait(&c.S.meet, met++ & 1u);
  };
  // this warp is through with the place of item k, and with its notes
  const auto leave = [&](uint32_t k) {
    __syncwarp();
    if ((r & 31) == 0) mbar_arrive(&c.S.item_free[k & (ITEM_RING - 1)]);
  };
  // reads the next item: 0 if there is none, 1 if it has rows for this row tile, 2 if not
  const auto peek = [&](TreeItem &x) {
    const bool some = tt_item(p, c.S, next_k, x, timed_out);
    if (!__all_sync(0xffffffffu, some)) return 0;
    ++next_k;
    return m * 128 < x.rows ? 1 : 2;
  };
  TreeItem it, next;
  TtRow row{}, next_row{};
  float ref = -INFINITY, l = 0.f;
  float v_ref = 1.f, v_log = 0.f;      // the V scale that P and O are relative to, and its logarithm
  uint32_t item_of = 0;                // its number
  // joins the copies and writes an item's rows, or its partials
  const auto finish = [&]() {
    if (!wait(&c.S.pv_done[2 * m + ((cnt - 1) & 1)], ((cnt - 1) >> 1) & 1u)) return false;
    tc_fence_after();
    const unsigned long long noted = c.S.nonfinite[item_of & (ITEM_RING - 1)] & row.bits;
    leave(item_of);
    if (__any_sync(0xffffffffu, noted != 0ull)) tt_add_back<D>(p, it, noted, row.copy * row.width, NM == 1 ? row.width : TT, o_at);
    const bool whole = it.whole();
    const long long slot = (2LL * blockIdx.x + (it.t0 > 0 ? 0 : 1)) * Cfg::RB + row.row;
    const long long to_row = whole ? row.out_row : slot;
    // the copies of a row meet at their common maximum
    float f = 1.f, ref_all = ref, l_all = l;
    const int copies = NM == 1 ? 128 / row.width : 1;
    if (NM == 1) {
      c.S.join_ml[r] = make_float2(ref, l);
      if (row.copy == 0) c.S.join_row[row.row] = to_row;
      if (!meet()) return false;   // (nothing below can fail, so the barriers there need no limit)
      for (int i = 0; i < copies; ++i) ref_all = fmaxf(ref_all, c.S.join_ml[row.row + i * row.width].x);
      l_all = 0.f;
      for (int i = 0; i < copies; ++i) {
        const float2 o = c.S.join_ml[row.row + i * row.width];
        l_all += ref_all == -INFINITY ? o.y : o.y * exp2_approx(o.x - ref_all);
      }
      f = ref_all == -INFINITY ? 1.f : exp2_approx(ref - ref_all);
    }
    if (whole) f = l_all == 0.f ? 0.f : f / l_all;
    if (QUANT) f *= v_ref;
    if constexpr (NM == 2) {
      long long to4[4];   // the four lanes' rows, -1: none
#pragma unroll
      for (int i = 0; i < 4; ++i) to4[i] = __shfl_sync(0xffffffffu, row.real ? to_row : -1ll, (r & 28) + i);
#pragma unroll 1
      for (int ch = 0; ch < D / 16; ++ch) {
        float o[16];
        tt_ld16(o_at + 16 * ch, o);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = l_all == 0.f ? 0.f : o[i] * f;
        tt_turn4(o, r & 31);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (to4[i] >= 0) {
            const float v[4] = {o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]};
            tt_put<4>(p, !whole, to4[i], 16 * ch + 4 * (r & 3), v);
          }
      }
    } else {
      // 32 columns at a time meet in shared memory; a row's 32 are put together by eight lanes
      const int sub = r & 7;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        float o[32];
        tt_ld32(o_at + 32 * ch, o);
        tc_wait_ld();
        float4 *at = reinterpret_cast<float4 *>(c.S.join[r]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          at[i] = l_all == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                               : make_float4(o[4 * i] * f, o[4 * i + 1] * f, o[4 * i + 2] * f, o[4 * i + 3] * f);
        named_sync(3, 128);
#pragma unroll 1
        for (int x = r >> 3; x < it.rows; x += 16) {
          float4 y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            y[i] = i < copies ? *reinterpret_cast<const float4 *>(&c.S.join[x + i * row.width][4 * sub])
                              : make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 t = make_float4((y[0].x + y[1].x) + (y[2].x + y[3].x), (y[0].y + y[1].y) + (y[2].y + y[3].y),
                                       (y[0].z + y[1].z) + (y[2].z + y[3].z), (y[0].w + y[1].w) + (y[2].w + y[3].w));
          const float v[4] = {t.x, t.y, t.z, t.w};
          tt_put<4>(p, !whole, c.S.join_row[x], 32 * ch + 4 * sub, v);
        }
        named_sync(3, 128);
      }
    }
    tc_fence_before();
    mbar_arrive(&c.S.o_free[m]);
    if (row.real && row.copy == 0) {
      if (!whole) {
        p.part_m[slot] = ref_all;
        p.part_l[slot] = l_all;
      } else if (p.lse) {
        p.lse[row.out_row] = l_all == 0.f ? -INFINITY : (ref_all + log2f(l_all)) / kLog2e;
      }
    }
    return true;
  };
  next.t0 = next.t1 = 0;
  int look = 2;
  for (;;) {
    if (look == 2) {
      do {
        if (next_k > 0) leave(next_k - 1);
        tile += next.t1 - next.t0;
        look = peek(next);
      } while (look == 2);
      if (look == 1) {
        tt_row<D, NM, GENERAL>(p, next, m, r, next_row);
        tt_load_q<D, NM, QUANT>(c, m, r, next_row);
        tt_show_q<D, NM, QUANT>(c, m);
      }
    }
    if (look == 0 || *timed_out) return;
    it = next;
    row = next_row;
    item_of = next_k - 1;
    // the item after this one, which is published by now (one further on is not before this one is under way):
    // its rows are known well before its queries go in, which is when the last scores of this
    // one are done, under their softmax
    look = peek(next);
    if (*timed_out) return;
    if (look == 1) tt_row<D, NM, GENERAL>(p, next, m, r, next_row);
    const int pre = it.n - it.c;
    const int first = row.copy * row.width;   // the copy's first token of a step
    const bool wide = NM == 2 || row.width == 64;
    const bool in_one = p.P % row.width == 0;   // a step's tokens are of one page
    const bool idle = !__any_sync(0xffffffffu, row.real);
    ref = -INFINITY;
    l = 0.f;
    if (NM == 1 && zeroed != row.width) {
      const uint32_t z[16] = {};
#pragma unroll 1
      for (int i = 0; i < 8; ++i) tt_st16(lanes + Cfg::P_COL + 16 * i, z);
      tt_wait_st();
      zeroed = row.width;
    }
    const int steps = (it.t1 - it.t0) * Cfg::STEPS;
    for (int s = 0; s < steps; ++s, ++cnt) {
      const int b = cnt & 1, h = s % Cfg::STEPS;
      const int mi = tile & (Cfg::META - 1);
      // (scores first: they say that the tile META before this one was described, whatever tiles this
      // warpgroup passed over)
      if (!wait(&c.S.s_full[2 * m + b], (cnt >> 1) & 1u)) return;
      if (look == 1 && s + 1 == steps) tt_load_q<D, NM, QUANT>(c, m, r, next_row);
      if (h == 0 && !wait(&c.S.meta_full[mi], (tile / Cfg::META) & 1u)) return;
      tc_fence_after();
      if (idle) {   // a warp without rows: what it leaves in P reaches no other row
        tc_fence_before();
        mbar_arrive(&c.S.p_full[2 * m + b]);
        if (h == Cfg::STEPS - 1) ++tile;
        continue;
      }
      const uint32_t s_at = lanes + Cfg::s_col(m, b) + first;
      const int in_tile = h * Cfg::STEP + first;                // the copy's first token in the tile
      const int off = pre - ((it.t1 - 1 - s / Cfg::STEPS) * TT + in_tile);  // its tokens before the drafts
      unsigned long long seen = c.S.valid[mi][in_tile >> 5];
      if (wide) seen |= static_cast<unsigned long long>(c.S.valid[mi][(in_tile >> 5) + 1]) << 32;
      const bool masked = off < row.width || seen != (wide ? ~0ull : 0xFFFFFFFFull);
      const bool scaled = QUANT && c.S.meta[QUANT ? mi : 0].scaled;
      // scales of one page serve the whole step where it lies in one; the V scale then goes into the exponent
      const float *ks = &c.S.ks[QUANT ? mi : 0][QUANT ? in_tile : 0], *vs = &c.S.vs[QUANT ? mi : 0][QUANT ? in_tile : 0];
      if (masked)   // tokens before the drafts, and the drafts of the row's bits
        seen &= off >= 64 ? ~0ull : off > 0 ? (row.bits << off) | ((1ull << off) - 1ull) : off > -64 ? row.bits >> -off : 0ull;
      if (QUANT && !FIXED && s == 0) {
        const float newest = !scaled ? 1.f : in_one ? vs[0] : seen ? vs[63 - __clzll(static_cast<long long>(seen))] : 1.f;
        v_ref = newest >= TT_V_LEAST && newest <= TT_V_MOST ? newest : 1.f;
        v_log = lg2_approx(v_ref);
      }
      // (the same for the whole warp, TMEM instructions depend on it: v_ref may differ between rows)
      bool one_page = QUANT && scaled && in_one && ks[0] > 0.f && ks[0] < 1e30f && vs[0] >= v_ref * TT_FOLD_LEAST &&
                      vs[0] <= v_ref * TT_FOLD_MOST;
      if (QUANT && !FIXED) one_page = __all_sync(0xffffffffu, one_page);
      // Scores as they enter the exponential, in units of log2 e: times the softmax scale
      // (left to the exponential where nothing else is to be done), the pages' scales,
      // capped, less the distance, -inf where the row does not see the token.  Steps with
      // unseen tokens, one or two of an item, are finished out of line.
      float sc = one_page ? ks[0] : scale;
      if (masked) {
        tt_masked<GENERAL>(p, s_at, row.width, seen, scaled ? ks : nullptr, scale, row.slope, row.pos, pre, off, it.c, it.b);
        sc = 1.f;
      }
      const bool finish_here = !masked && ((QUANT && scaled && !one_page) || (GENERAL && (p.cap > 0.f || (!FIXED && p.slopes))));
      const float sc_in = sc;
      if (finish_here) sc = 1.f;
      const bool half = CH == 64 && row.width == 32;   // (the rest of x is not used then)
      float x[CH], top = -INFINITY;
      const auto load = [&](int ch) {
        tt_ld32(s_at + ch, x);
        if (CH == 64 && !half) tt_ld32(s_at + ch + 32, x + CH - 32);
        tc_wait_ld();
      };
      const auto complete = [&](int ch) {
        float mul = sc_in;   // what is still to be multiplied
        if (QUANT && scaled && !one_page) {
#pragma unroll
          for (int i = 0; i < CH; i += 4) {
            if (i == 32 && half) break;
            const float4 k4 = *reinterpret_cast<const float4 *>(ks + ch + i);
            const float2 y = mul2(make_float2(x[i], x[i + 1]), make_float2(k4.x, k4.y));
            const float2 z = mul2(make_float2(x[i + 2], x[i + 3]), make_float2(k4.z, k4.w));
            x[i] = y.x;
            x[i + 1] = y.y;
            x[i + 2] = z.x;
            x[i + 3] = z.y;
          }
          mul = 1.f;
        }
        if (GENERAL && p.cap > 0.f) {
          if constexpr (QUANT) {
            // the closed form throughout: with the polynomial's code beside the expansion's, fetching instructions
            // took longer than the special functions (tiers of 32K tokens: 356 us against 318)
            const float2 k1 = make_float2(mul * cap_k1, mul * cap_k1);
#pragma unroll
            for (int i = 0; i < CH; i += 2) {
              const float2 y = mul2(make_float2(x[i], x[i + 1]), k1);
              const float2 z = add2(make_float2(exp2_approx(y.x), exp2_approx(y.y)), make_float2(1.f, 1.f));
              x[i] = rcp_approx(z.x);
              x[i + 1] = rcp_approx(z.y);
              if (!FIXED) {   // (else with the reference, below)
                const float2 w = fma2(make_float2(x[i], x[i + 1]), make_float2(-2.f * c2, -2.f * c2), make_float2(c2, c2));
                x[i] = w.x;
                x[i + 1] = w.y;
              }
            }
          } else {
            const float to_u = mul * cap_k1 * (0.5f / kLog2e);
            const float2 u2 = make_float2(to_u, to_u);
            float most[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < CH; i += 2) {
              if (i == 32 && half) break;
              const float2 u = mul2(make_float2(x[i], x[i + 1]), u2);
              x[i] = u.x;
              x[i + 1] = u.y;
              most[0] = fmaxf(most[0], fabsf(u.x));
              most[1] = fmaxf(most[1], fabsf(u.y));
            }
            if (__any_sync(0xffffffffu, fmaxf(most[0], most[1]) > TT_CAP_NEAR)) {
#pragma unroll
              for (int i = 0; i < CH; ++i) {
                if (i == 32 && half) break;
                x[i] = tt_cap_far(x[i], c2);
              }
            } else {
#pragma unroll
              for (int i = 0; i < CH; i += 2) {
                if (i == 32 && half) break;
                const float2 y = tt_cap_near(make_float2(x[i], x[i + 1]), c2);
                x[i] = y.x;
                x[i + 1] = y.y;
              }
            }
          }
          mul = 1.f;
        }
        if (GENERAL && !FIXED && p.slopes) {
          const float base = row.slope * static_cast<float>(pre - off + ch - row.pos);
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            if (i == 32 && half) break;
            x[i] = fmaf(x[i], mul, fmaf(row.slope, static_cast<float>(i), base));
          }
        }
      };
      if constexpr (!FIXED) {
        // CH tokens at a time, the last first; the second pass then begins with the
        // ones that are in registers
#pragma unroll 1
        for (int ch = half ? 0 : row.width - CH; ch >= 0; ch -= CH) {
          load(ch);
          if ((QUANT || GENERAL) && finish_here) {
            complete(ch);
            if (CH == 32 && ch > 0) tt_st32(s_at + ch, reinterpret_cast<const uint32_t *>(x));
          }
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int i = 4; i < CH; i += 4) {
            if (i == 32 && half) break;
#pragma unroll
            for (int y = 0; y < 4; ++y) mx[y] = fmaxf(mx[y], x[i + y]);
          }
          top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
        }
        if (CH == 32 && (QUANT || GENERAL) && finish_here) tt_wait_st();
      }
      top *= sc;
      if (FIXED) {
        ref = TT_FIXED_REF;
      } else if (s == 0) {
        ref = top;
      } else if (__any_sync(0xffffffffu, top > ref + RESCALE_STEP)) {
        // O of the steps so far moves to the new reference
        if (!wait(&c.S.pv_done[2 * m + ((cnt - 1) & 1)], ((cnt - 1) >> 1) & 1u)) return;
        tc_fence_after();
        const float to = fmaxf(ref, top);
        const float f = to == -INFINITY ? 1.f : exp2_approx(ref - to);
        l *= f;
        ref = to;
#pragma unroll 1
        for (int ch = 0; ch < D / 16; ++ch) {
          float o[16];
          tt_ld16(o_at + 16 * ch, o);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] *= f;
          tt_st16(o_at + 16 * ch, reinterpret_cast<const uint32_t *>(o));
        }
        tt_wait_st();
      }
      // p = 2^(s - ref), its sum, and P as the MMA's operand
      float less = ref == -INFINITY ? 0.f : -ref, back = 1.f;
      if constexpr (QUANT) {
        // V scales are taken relative to the newest page's.  A row's largest exponential is often 1, which bf16 holds,
        // but not its product with a scale, and in a row that one token rules that rounding is the row's (int4
        // pages with steep ALiBi: outputs 0.0030 off in the mean square, 0.0019 so; 0.0017 is their own rounding)
        const float vs0 = one_page ? vs[0] : 1.f, vs0_log = lg2_approx(vs0);   // (2^-22 off, like the exponential)
        less += vs0_log - v_log;
        back = vs0 == v_ref ? 1.f : v_ref * rcp_approx(vs0);
      }
      if (FIXED && QUANT && finish_here) {
        less += c2;
        sc = -2.f * c2;
      }
      const float2 less2 = make_float2(less, less), sc2 = make_float2(sc, sc);
      float2 sum[2] = {};
      const uint32_t p_at = lanes + Cfg::p_col(m, b) + first / 2;
      const auto exps = [&](int ch, auto by_token) {
#pragma unroll
        for (int i0 = 0; i0 < CH; i0 += 32) {
          if (i0 == 32 && half) break;
          uint32_t w[16];
#pragma unroll
          for (int i = i0; i < i0 + 32; i += 2) {
            const float2 y = fma2(make_float2(x[i], x[i + 1]), sc2, less2);
            float2 e = make_float2(exp2_approx(y.x), exp2_approx(y.y));
            sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], e);
            if (decltype(by_token)::value) e = mul2(e, *reinterpret_cast<const float2 *>(vs + ch + i));
            w[(i - i0) >> 1] = pack_bf16(e.x, e.y);
          }
          tt_st16(p_at + (ch + i0) / 2, w);   // (over columns of S that were read before)
        }
      };
      const bool by_token = QUANT && scaled && !one_page;
#pragma unroll 1
      for (int ch = 0; ch < row.width; ch += CH) {
        if (FIXED || ch > 0) load(ch);
        if (FIXED && finish_here) complete(ch);
        if (QUANT && by_token)
          exps(ch, std::true_type());
        else
          exps(ch, std::false_type());
      }
      const float2 s01 = add2(sum[0], sum[1]);
      l += (s01.x + s01.y) * back;
      tt_wait_st();
      tc_fence_before();
      mbar_arrive(&c.S.p_full[2 * m + b]);
      if (h == Cfg::STEPS - 1) ++tile;
    }
    if (look == 1) tt_show_q<D, NM, QUANT>(c, m);
    if (!finish()) return;
  }
}

// ---- kernel ------------------------------------------------------------------------

template <int D, int NM, bool QUANT>
constexpr size_t tt_head() {
  return (sizeof(typename TtCtx<D, NM, QUANT>::Smem) + 1023) / 1024 * 1024;
}
template <int D, int NM, bool QUANT>
constexpr size_t tt_smem() {
  using Cfg = TtCfg<D, NM, QUANT>;
  return tt_head<D, NM, QUANT>() + static_cast<size_t>(NM + Cfg::NS) * Cfg::ROW_TILE + 1024;
}

template <int D, int NM, bool QUANT, int MODE>
__global__ void __launch_bounds__((TtCfg<D, NM, QUANT>::THREADS), 1)
    tree_tc_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
  using Cfg = TtCfg<D, NM, QUANT>;
  using Smem = TtSmem<Cfg::NS, NM, QUANT, Cfg::META>;
  static_assert(tt_smem<D, NM, QUANT>() <= 227 * 1024, "shared memory of a block");
  extern __shared__ uint8_t raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
  Smem &S = *reinterpret_cast<Smem *>(base);
  const int warp = threadIdx.x >> 5;
  TtCtx<D, NM, QUANT> c{p, kmap, vmap, S, base + tt_head<D, NM, QUANT>(),
                        base + tt_head<D, NM, QUANT>() + NM * Cfg::ROW_TILE, min(128, p.P & -p.P)};
  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg::NS; ++i) {
      mbar_init(&S.slot_full[i], 1);
      mbar_init(&S.slot_empty[i], NM + (QUANT ? 1 : 0));   // the MMAs' reads, and the expanding warps
      mbar_init(&S.raw_full[i], 1);
    }
    for (int i = 0; i < 2 * NM; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 128);
      mbar_init(&S.pv_done[i], 1);
    }
    for (int i = 0; i < NM; ++i) {
      mbar_init(&S.q_full[i], 128);
      mbar_init(&S.o_free[i], 128);
      mbar_init(&S.drain[i], 1);
    }
    for (int i = 0; i < Cfg::META; ++i) mbar_init(&S.meta_full[i], 1);
    for (int i = 0; i < ITEM_RING; ++i) {
      mbar_init(&S.item_full[i], 1);
      mbar_init(&S.item_free[i], 4 * NM);   // the softmax warps
    }
    mbar_init(&S.meet, 128);
    fence_mbar_init();
  }
  if (threadIdx.x == 96 && p.pool_pages[CFR_FMT_BF16] > 0) {   // (the host encodes no map of an empty pool)
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem_base)),
                 "r"(Cfg::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  TreeCursor cur;
  const long long W = tree_find<TT, Cfg::RB>(
      p, S.scratch, threadIdx.x, Cfg::THREADS,
      [&](long long w) { return TreeCut(w, p.grid).start(blockIdx.x); }, cur);
  cur.end = TreeCut(W, p.grid).start(blockIdx.x + 1);
  tc_fence_after();   // (tree_find synchronises the block)
  griddep_launch_dependents();   // the merge may find its cuts meanwhile; it waits for this grid's results
  bool timed_out = false;
  const int wg = warp >> 2;
  if (wg == 0) {
    if (warp == 0 || warp == 3) {
      tt_producer<D, NM, QUANT>(c, cur, &timed_out, warp & 1);
    } else if (warp <= NM) {
      tt_issue<D, NM, QUANT>(c, &timed_out, warp - 1);
    }
  } else if (wg <= NM) {
    tt_softmax<D, NM, QUANT, MODE>(c, &timed_out);
  } else if constexpr (QUANT) {
    tt_expand<D, NM>(c, &timed_out, Cfg::LOADERS == 1 ? 2 : wg - NM - 1);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(S.tmem_base), "r"(Cfg::TMEM_COLS) : "memory");
  }
}

template <int D, int NM, bool QUANT, int MODE>
cudaError_t launch(const TreeParams &p, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t s) {
  using Cfg = TtCfg<D, NM, QUANT>;
  auto kernel = tree_tc_kernel<D, NM, QUANT, MODE>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(tt_smem<D, NM, QUANT>()));
  if (e != cudaSuccess) return e;
  kernel<<<p.grid, Cfg::THREADS, tt_smem<D, NM, QUANT>(), s>>>(p, k, v);
  return cudaGetLastError();
}

template <int D, int NM, bool QUANT>
cudaError_t launch_mode(const TreeParams &p, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t s) {
  if (p.cap > 0.f && !p.slopes && p.cap * kLog2e <= TT_FIXED_CAP) return launch<D, NM, QUANT, FIXED_REFERENCE>(p, k, v, s);
  return p.cap > 0.f || p.slopes ? launch<D, NM, QUANT, GENERAL_SCORES>(p, k, v, s) : launch<D, NM, QUANT, PLAIN>(p, k, v, s);
}

}  // namespace

// Whether the tensor-core kernel takes the call: bf16 queries, no fp32 pages, pages a multiple of 8 tokens, and
// a cap between 2^-10 and 2^10 (the closed form of the tanh, see tt_cap_far, is off by 2^-22 of the cap, whatever the
// score, which at 2^10 is still below the rounding of P).
bool tree_tc_supported(const TreeParams &p) {
  if (p.q_fmt != CFR_FMT_BF16 || p.P % 8 != 0 || p.P > (1 << 24)) return false;
  if (p.cap > 0.f && !(p.cap >= 0x1p-10f && p.cap <= 0x1p10f)) return false;
  if (p.page_fmt ? p.k_pool[CFR_FMT_F32] != nullptr : p.uniform_fmt == CFR_FMT_F32) return false;
  return p.pool_pages[CFR_FMT_BF16] * p.Hkv <= 0x7fffffffLL / p.P;   // rows of a tensor map
}

// Rows of a work item, which chooses the variant: narrow up to 64 rows of a kv head, else wide.  (On the wide variant
// 28 rows over 1K tokens took 31 us of GPU time against 19, 64 rows over 1M tokens 943 against 654, 64 rows of
// capped scores over tiers 459 against 279.)
int tree_tc_rows(int most_rows) { return most_rows > 64 ? 256 : 64; }

cudaError_t launch_tree_tc(const TreeParams &p, int rb, cudaStream_t s) {
  CUtensorMap k, v;
  std::memset(&k, 0, sizeof(k));
  std::memset(&v, 0, sizeof(v));
  const int box = p.P & -p.P;
  if (p.k_pool[CFR_FMT_BF16] && p.pool_pages[CFR_FMT_BF16] > 0) {
    const long long rows = p.pool_pages[CFR_FMT_BF16] * p.Hkv * p.P;
    if (!encode_pool_map(&k, p.k_pool[CFR_FMT_BF16], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, rows, p.D, box < 128 ? box : 128) ||
        !encode_pool_map(&v, p.v_pool[CFR_FMT_BF16], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, rows, p.D, box < 128 ? box : 128))
      return cudaErrorInvalidValue;
  }
  bool quant = !p.page_fmt && is_quantised(p.uniform_fmt);
  if (p.page_fmt) quant = p.k_pool[CFR_FMT_I8] || p.k_pool[CFR_FMT_I4] || p.k_pool[CFR_FMT_FP8];
  if (p.D == 128) {
    if (rb == 64)
      return quant ? launch_mode<128, 1, true>(p, k, v, s) : launch_mode<128, 1, false>(p, k, v, s);
    return quant ? launch_mode<128, 2, true>(p, k, v, s) : launch_mode<128, 2, false>(p, k, v, s);
  }
  if (rb == 64)
    return quant ? launch_mode<64, 1, true>(p, k, v, s) : launch_mode<64, 1, false>(p, k, v, s);
  return quant ? launch_mode<64, 2, true>(p, k, v, s) : launch_mode<64, 2, false>(p, k, v, s);
}

}  // namespace cfr
