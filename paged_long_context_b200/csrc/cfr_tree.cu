// cfr_tree.cu -- attention of a tree of drafted tokens over the paged cache: the
// general kernel (any formats, page sizes and types, fp32 throughout), the merge
// of partials, and the C ABI.
//
// s_ij = sigma q_i . k_j, capped as cap tanh(s / cap), minus the ALiBi distance;
// tokens before the drafts are seen by every row, drafts by the row's mask bits.
// The softmax runs online over tiles of tokens: with m the running maximum,
// l <- l 2^(m - m') + sum 2^(s - m'), acc <- acc 2^(m - m') + sum 2^(s - m') v.
//
// The general kernel keeps 32 rows and a tile of 64 tokens in shared memory as
// fp32 and computes both products with fp32 multiply-adds.  It is the one that
// fp32 caches and queries take, whose 24-bit products the tensor cores do not
// have, and it is bound by the shared-memory reads that feed those multiply-adds and by the barriers of its one
// stage, between a tile's loads, scores and products (8 drafts over two fp32 sequences of 8K tokens: 153 us, 14 of the
// 74 TFLOP/s that the fp32 units have; 64 drafts over 16 ragged bf16 sequences: 12.2 ms, on the tensor cores 0.38).
#include <climits>
#include <cstring>

#include "cfr_cells.cuh"
#include "cfr_tree.cuh"

namespace cfr {

bool tree_tc_supported(const TreeParams &p);
int tree_tc_rows(int most_rows);
cudaError_t launch_tree_tc(const TreeParams &p, int rb, cudaStream_t s);

namespace {

constexpr int kGenTT = 64, kGenRB = 32, kGenThreads = 256;

template <int D>
struct GenSmem {
  float q[kGenRB][D];
  float k[kGenTT][D + 4];   // + 4: the 16 tokens that a warp reads at once lie in different banks
  float v[kGenTT][D];
  float s[kGenRB][kGenTT + 4];
  unsigned long long bits[kGenRB];
  float slope[kGenRB];      // times log2 e
  int pos[kGenRB];          // position of the row's draft
  int tok_pos[kGenTT];
  float k_scale[kGenTT], v_scale[kGenTT];
  long long tok_at[kGenTT];  // byte offset of the token's row in its pool
  int tok_fmt[kGenTT];      // -1: the token takes no part
  TreeScratch scratch;
};

__device__ __forceinline__ void decode8(int fmt, const uint8_t *row, int c8, float scale, float (&x)[kVec]) {
  switch (fmt) {
    case CFR_FMT_F32: decode_raw<CFR_FMT_F32>(load_raw<CFR_FMT_F32>(row, c8), 1.f, x); break;
    case CFR_FMT_BF16: decode_raw<CFR_FMT_BF16>(load_raw<CFR_FMT_BF16>(row, c8), 1.f, x); break;
    case CFR_FMT_I8: decode_raw<CFR_FMT_I8>(load_raw<CFR_FMT_I8>(row, c8), scale, x); break;
    case CFR_FMT_I4: decode_raw<CFR_FMT_I4>(load_raw<CFR_FMT_I4>(row, c8), scale, x); break;
    default: decode_raw<CFR_FMT_FP8>(load_raw<CFR_FMT_FP8>(row, c8), scale, x); break;
  }
}

__device__ __forceinline__ void put(const TreeParams &p, long long e, float x) {
  if (p.out_fmt == CFR_FMT_F32)
    static_cast<float *>(p.out)[e] = x;
  else
    static_cast<__nv_bfloat16 *>(p.out)[e] = __float2bfloat16_rn(x);
}

// places of the tile's tokens (threads 0 .. TT - 1)
template <int D>
__device__ __forceinline__ void gen_resolve(const TreeParams &p, GenSmem<D> &S, const TreeItem &it, int t0, int i) {
  const int j = t0 + i;
  int fmt = -1;
  if (j < it.n) {
    const long long cell = static_cast<long long>(it.b) * p.max_pages + j / p.P;
    const long long slot = p.page_table[cell];
    const int f = p.page_fmt ? static_cast<int>(p.page_fmt[cell]) : p.uniform_fmt;
    if (f >= kFmtCount) {
      set_err(p.err, CFR_DEVERR_PAGE_FMT);
    } else if (!p.k_pool[f]) {
      set_err(p.err, CFR_DEVERR_POOL);
    } else if (slot < 0 || slot >= p.pool_pages[f]) {
      set_err(p.err, CFR_DEVERR_PAGE_ID);
    } else {
      fmt = f;
      S.tok_at[i] = ((slot * p.Hkv + it.g) * p.P + j % p.P) * row_bytes(f, D);
      float2 sc = make_float2(1.f, 1.f);
      if (is_quantised(f)) sc = *reinterpret_cast<const float2 *>(p.scales[f] + (slot * p.Hkv + it.g) * 2);
      S.k_scale[i] = sc.x;
      S.v_scale[i] = sc.y;
    }
  }
  S.tok_fmt[i] = fmt;
  const int k = j - (it.n - it.c);  // draft number
  S.tok_pos[i] = (p.slopes && k >= 0 && k < it.c)
                     ? it.n - it.c + (p.depths ? p.depths[static_cast<long long>(it.b) * p.nq + k] : k)
                     : j;
}

template <int D>
__global__ void __launch_bounds__(kGenThreads) tree_general_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  GenSmem<D> &S = *reinterpret_cast<GenSmem<D> *>(raw);
  constexpr int DV = D / 32;  // values of a row that a lane accumulates
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  TreeCursor cur;
  const int cta = blockIdx.x;
  const long long W = tree_find<kGenTT, kGenRB>(
      p, S.scratch, tid, kGenThreads, [&](long long w) { return TreeCut(w, p.grid).start(cta); }, cur);
  cur.end = TreeCut(W, p.grid).start(cta + 1);
  TreeItem it;
  while (tree_next<kGenTT, kGenRB>(p, cur, it)) {
    __syncthreads();
    if (it.bad && tid == 0) set_err(p.err, CFR_DEVERR_SEQ_LEN);
    for (int e = tid; e < kGenRB * (D / kVec); e += kGenThreads) {
      const int r = e / (D / kVec), c8 = e % (D / kVec);
      float x[kVec] = {};
      if (r < it.rows) {
        int i, h;
        tree_row(p, it, it.row0 + r, i, h);
        const uint8_t *src = static_cast<const uint8_t *>(p.q) +
                             tree_out_row(p, it.b, i, h) * row_bytes(p.q_fmt, D);
        decode8(p.q_fmt, src, c8, 1.f, x);
        if (c8 == 0) {
          S.bits[r] = tree_bits(p, it.b, i, it.c);
          S.slope[r] = p.slopes ? p.slopes[h] * kLog2e : 0.f;
          S.pos[r] = it.n - it.c + (p.slopes && p.depths ? p.depths[static_cast<long long>(it.b) * p.nq + i] : i);
        }
      } else if (c8 == 0) {
        S.bits[r] = 0;
        S.slope[r] = 0.f;
        S.pos[r] = 0;
      }
#pragma unroll
      for (int k = 0; k < kVec; ++k) S.q[r][c8 * kVec + k] = x[k];
    }
    // warp w owns rows 4 w .. 4 w + 3 in the softmax and the accumulation
    float m[4], l[4], acc[4][DV];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int d = 0; d < DV; ++d) acc[r][d] = 0.f;
    }
    for (int t = it.t0; t < it.t1; ++t) {
      const int j0 = t * kGenTT;
      __syncthreads();
      if (tid < kGenTT) gen_resolve(p, S, it, j0, tid);
      __syncthreads();
      for (int e = tid; e < 2 * kGenTT * (D / kVec); e += kGenThreads) {
        const int kv = e >= kGenTT * (D / kVec);
        const int f = kv ? e - kGenTT * (D / kVec) : e;
        const int i = f / (D / kVec), c8 = f % (D / kVec);
        float x[kVec] = {};
        const int fmt = S.tok_fmt[i];
        if (fmt >= 0)
          decode8(fmt, (kv ? p.v_pool[fmt] : p.k_pool[fmt]) + S.tok_at[i], c8, kv ? S.v_scale[i] : S.k_scale[i], x);
        float *dst = kv ? &S.v[i][c8 * kVec] : &S.k[i][c8 * kVec];
        reinterpret_cast<float4 *>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
      }
      __syncthreads();
      {  // scores: two rows by four tokens a thread
        const int r0 = (tid >> 4) * 2, c0 = tid & 15;
        float s[2][4] = {};
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
          const float4 a = *reinterpret_cast<const float4 *>(&S.q[r0][d]);
          const float4 b = *reinterpret_cast<const float4 *>(&S.q[r0 + 1][d]);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float4 k = *reinterpret_cast<const float4 *>(&S.k[c0 + 16 * x][d]);
            s[0][x] = fmaf(a.x, k.x, fmaf(a.y, k.y, fmaf(a.z, k.z, fmaf(a.w, k.w, s[0][x]))));
            s[1][x] = fmaf(b.x, k.x, fmaf(b.y, k.y, fmaf(b.z, k.z, fmaf(b.w, k.w, s[1][x]))));
          }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int r = r0 + y;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int i = c0 + 16 * x, k = j0 + i - (it.n - it.c);
            float v = s[y][x] * p.sigma;
            // (tanh x is x to 2^-24 of it below 2^-12; a large cap's quotient would be denormal)
            if (p.cap > 0.f && !(fabsf(v) < p.cap * 0x1p-12f)) v = p.cap * tanhf(v / p.cap);
            v = v * kLog2e - S.slope[r] * static_cast<float>(S.pos[r] - S.tok_pos[i]);
            const bool sees = S.tok_fmt[i] >= 0 && (k < 0 || ((S.bits[r] >> k) & 1ull));
            S.s[r][i] = sees ? v : -INFINITY;
          }
        }
      }
      __syncthreads();
      const bool draft_tile = j0 + kGenTT > it.n - it.c;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float *row = S.s[4 * warp + r];
        const float a = row[lane], b = row[lane + 32];
        float mx = fmaxf(a, b);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        // fmaxf drops NaN scores; they must reach the row's result
        const float mn = fmaxf(m[r], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float pa = exp2_approx(a - ref), pb = exp2_approx(b - ref);
        float sum = pa + pb;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float alpha = exp2_approx(m[r] - ref);
        l[r] = fmaf(l[r], alpha, sum);
        m[r] = mn;
#pragma unroll
        for (int d = 0; d < DV; ++d) acc[r][d] *= alpha;
        // a token that the row does not see is marked, so that its values are left out, not multiplied by 0
        row[lane] = a == -INFINITY ? -1.f : pa;
        row[lane + 32] = b == -INFINITY ? -1.f : pb;
      }
      __syncwarp();
      for (int i = 0; i < kGenTT; ++i) {
        float vv[DV];
#pragma unroll
        for (int d = 0; d < DV; ++d) vv[d] = S.v[i][lane * DV + d];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float w = S.s[4 * warp + r][i];
          if (draft_tile && w == -1.f) continue;
          const float ww = w == -1.f ? 0.f : w;
#pragma unroll
          for (int d = 0; d < DV; ++d) acc[r][d] = fmaf(ww, vv[d], acc[r][d]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * warp + r;
      if (row >= it.rows) continue;
      if (it.whole()) {
        int i, h;
        tree_row(p, it, it.row0 + row, i, h);
        const long long o = tree_out_row(p, it.b, i, h);
        const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
#pragma unroll
        for (int d = 0; d < DV; ++d) put(p, o * D + lane * DV + d, l[r] == 0.f ? 0.f : acc[r][d] * inv);
        if (p.lse && lane == 0) p.lse[o] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) / kLog2e;
      } else {
        const long long s = (2LL * cta + (it.t0 > 0 ? 0 : 1)) * kGenRB + row;
#pragma unroll
        for (int d = 0; d < DV; ++d) p.part_acc[s * D + lane * DV + d] = acc[r][d];
        if (lane == 0) {
          p.part_m[s] = m[r];
          p.part_l[s] = l[r];
        }
      }
    }
  }
}

// ---- merge -------------------------------------------------------------------

// Partials of the items that several CTAs share.  CTA x stands for the cut
// between CTAs x and x + 1 of the attention: where that cut is the first inside
// an item, it merges the item, 8 rows a block, a warp each.  A warp's lanes first
// weigh 32 partials at once, then take their sums four at a time.  The partials
// count in the order of the tiles, so the result does not depend on timing.
// Block (0, 0) waits for the attention's end whatever it has to merge: were all blocks
// gone before it, what follows in the stream could start under the attention.
template <int TT, int RB, int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  __shared__ TreeScratch scratch;
  constexpr int DV = D / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  TreeCursor cur;
  const int cut = blockIdx.x + 1;
  // (the cut comes from the call's inputs: found while the attention is still running)
  const long long W = tree_find<TT, RB>(
      p, scratch, tid, 256, [&](long long w) { return TreeCut(w, p.grid).start(cut); }, cur);
  const auto leave = [] {
    if (blockIdx.x == 0 && blockIdx.y == 0) griddep_wait();
  };
  if (cur.u >= W) return leave();
  const TreeCut c(W, p.grid);
  // the item that the cut falls into, and its first unit
  TreeItem it;
  long long first;
  {
    const TreeSeq s = tree_seq<TT, RB>(p, cur.b);
    const int each = s.tiles + tree_item_cost<RB>;
    first = cur.base + (cur.u - cur.base) / each * each;
    TreeCursor all{first, first + each, cur.base, cur.b};
    if (!tree_next<TT, RB>(p, all, it)) return leave();
  }
  const long long last = first + it.tiles + tree_item_cost<RB>;
  if (tree_tile<RB>(cur.u - first) == 0) return leave();                           // no tiles before the cut
  const long long before = c.start(cut - 1);
  if (before >= first && tree_tile<RB>(before - first) > 0) return leave();         // an earlier cut parts the item too
  const int row = blockIdx.y * 8 + warp;
  if (row >= it.rows) return leave();
  griddep_wait();
  float M = -INFINITY, L = 0.f, acc[DV] = {};
  for (int i0 = cut - 1; i0 < p.grid && c.start(i0) < last; i0 += 32) {
    // lane x: the partial that CTA i0 + x left
    const int i = i0 + lane;
    float m = -INFINITY, l = 0.f;
    int slot = 0;
    if (i < p.grid) {
      const long long lo = c.start(i), hi = c.start(i + 1);
      const int t0 = lo <= first ? 0 : tree_tile<RB>(lo - first), t1 = tree_tile<RB>(min(hi, last) - first);
      if (lo < last && t0 < t1) {
        slot = 2 * i + (t0 > 0 ? 0 : 1);
        m = p.part_m[static_cast<long long>(slot) * RB + row];
        l = p.part_l[static_cast<long long>(slot) * RB + row];
      }
    }
    if (l == 0.f) m = -INFINITY;
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float mn = fmaxf(M, top);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float a = exp2_approx(M - ref), b = l == 0.f ? 0.f : exp2_approx(m - ref);
    float sum = l * b;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    L = L * a + sum;
#pragma unroll
    for (int d = 0; d < DV; ++d) acc[d] *= a;
    uint32_t some = __ballot_sync(0xffffffffu, l != 0.f);
    while (some) {
      float v[4][DV], w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int from = some ? __ffs(some) - 1 : 0;
        w[x] = some ? __shfl_sync(0xffffffffu, b, from) : 0.f;
        const int sl = __shfl_sync(0xffffffffu, slot, from);
        const float *src = p.part_acc + (static_cast<long long>(sl) * RB + row) * D + lane * DV;
#pragma unroll
        for (int d = 0; d < DV; ++d) v[x][d] = some ? src[d] : 0.f;
        some &= some - 1;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int d = 0; d < DV; ++d) acc[d] = fmaf(v[x][d], w[x], acc[d]);
    }
    M = mn;
  }
  int i, h;
  tree_row(p, it, it.row0 + row, i, h);
  const long long o = tree_out_row(p, it.b, i, h);
  const float inv = 1.f / L;
#pragma unroll
  for (int d = 0; d < DV; ++d) put(p, o * D + lane * DV + d, L == 0.f ? 0.f : acc[d] * inv);
  if (p.lse && lane == 0) p.lse[o] = L == 0.f ? -INFINITY : (M + log2f(L)) / kLog2e;
}

// ---- host --------------------------------------------------------------------

constexpr int kTreeMaxDevices = 64;

// SM count of the current device (cached per device), 0 on failure
int tree_sms() {
  static int cache[kTreeMaxDevices];
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < kTreeMaxDevices && cache[dev] > 0) return cache[dev];
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < kTreeMaxDevices) cache[dev] = v;
  return v;
}

// CTAs of the general kernel: two fit an SM
int general_grid(int sms) { return 2 * sms; }

struct TreeWs {
  size_t part_m, part_l, part_acc, total;
};
TreeWs tree_ws(int slots, int rb, int d) {
  TreeWs w;
  const size_t rows = static_cast<size_t>(slots) * rb;
  w.part_m = 0;
  w.part_l = (rows * 4 + 255) / 256 * 256;
  w.part_acc = 2 * w.part_l;
  w.total = w.part_acc + rows * d * 4;
  return w;
}

// Scratch of the larger of the two kernels' cuts: the general one (two CTAs an SM,
// 32 rows) or the tensor-core one (one CTA an SM, 64 or 256 rows).  `rows`: the
// most rows that a kv head can have.
TreeWs tree_scratch(int sms, int rows, int d) {
  const TreeWs a = tree_ws(2 * general_grid(sms), kGenRB, d), b = tree_ws(2 * sms, tree_tc_rows(rows), d);
  return a.total > b.total ? a : b;
}

template <int TT, int RB>
cudaError_t launch_tree_merge(const TreeParams &p, cudaStream_t s) {
  const dim3 grid(p.grid - 1, RB / 8);
  return p.D == 128 ? launch_after_previous(tree_merge_kernel<TT, RB, 128>, grid, dim3(256), 0, s, p)
                    : launch_after_previous(tree_merge_kernel<TT, RB, 64>, grid, dim3(256), 0, s, p);
}

template <int D>
cudaError_t launch_general(const TreeParams &p, cudaStream_t s) {
  const size_t smem = sizeof(GenSmem<D>);
  cudaError_t e = cudaFuncSetAttribute(tree_general_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  tree_general_kernel<D><<<p.grid, kGenThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace cfr

using namespace cfr;

extern "C" {

size_t cfr_paged_decode_tree_workspace_size(int32_t batch, int32_t num_queries,
                                            int32_t num_q_heads, int32_t num_kv_heads,
                                            int32_t head_dim) {
  if (batch <= 0 || num_queries <= 0 || num_queries > CFR_TREE_MAX_QUERIES || num_q_heads <= 0 ||
      num_q_heads > kMaxQHeads || num_kv_heads <= 0 || num_kv_heads > kMaxQHeads ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  const int sms = tree_sms();
  if (sms <= 0) return 0;
  return tree_scratch(sms, num_queries * num_q_heads, head_dim).total;
}

cfr_status cfr_paged_decode_tree(const void *q, int32_t q_fmt, const cfr_kv_pool *kv,
                                 const int32_t *page_table, int32_t max_pages,
                                 const int32_t *seq_lens, int32_t batch,
                                 const uint8_t *page_fmt, int32_t uniform_fmt,
                                 int32_t num_q_heads, int32_t num_queries,
                                 const int32_t *q_lens, const uint64_t *tree_mask,
                                 const int32_t *depths, const int32_t *head_map,
                                 const float *alibi_slopes, float softmax_scale,
                                 float logit_cap, void *out, int32_t out_fmt, float *lse,
                                 void *workspace, size_t workspace_bytes, uint32_t *err_word,
                                 void *stream) {
  CacheView c;
  cfr_status st = make_view(kv, page_table, max_pages, page_fmt, uniform_fmt, batch, kAllFormats,
                            err_word, &c);
  if (st != CFR_OK) return st;
  if (!q || !ptr_aligned(q, 16) || !out || !ptr_aligned(out, 16) || !seq_lens) return CFR_ERR_INVALID_ARG;
  if ((q_fmt != CFR_FMT_F32 && q_fmt != CFR_FMT_BF16) || (out_fmt != CFR_FMT_F32 && out_fmt != CFR_FMT_BF16))
    return CFR_ERR_INVALID_ARG;
  if (num_queries < 1 || num_q_heads < 1) return CFR_ERR_INVALID_ARG;
  if (num_queries > CFR_TREE_MAX_QUERIES || num_q_heads > kMaxQHeads) return CFR_ERR_UNSUPPORTED;
  if (!(softmax_scale >= 0.f) || softmax_scale == INFINITY) return CFR_ERR_INVALID_ARG;
  if (!(logit_cap >= 0.f) || logit_cap == INFINITY) return CFR_ERR_INVALID_ARG;
  // (tokens are counted past the last one's tile)
  if (static_cast<long long>(max_pages) * kv->page_tokens > INT_MAX - 1024) return CFR_ERR_OVERFLOW;
  if (!head_map && num_q_heads % kv->num_kv_heads != 0) return CFR_ERR_INVALID_ARG;
  TreeParams p;
  std::memset(&p, 0, sizeof(p));
  int count[kMaxQHeads + 1] = {};
  for (int h = 0; h < num_q_heads; ++h) {
    const int g = head_map ? head_map[h] : h / (num_q_heads / kv->num_kv_heads);
    if (g < 0 || g >= kv->num_kv_heads) return CFR_ERR_INVALID_ARG;
    ++count[g];
  }
  p.heads_each = count[0];
  for (int g = 0; g < kv->num_kv_heads; ++g) {
    p.head_off[g + 1] = static_cast<int16_t>(p.head_off[g] + count[g]);
    if (count[g] != count[0]) p.heads_each = 0;
  }
  for (int h = 0, fill[kMaxQHeads + 1] = {}; h < num_q_heads; ++h) {
    const int g = head_map ? head_map[h] : h / (num_q_heads / kv->num_kv_heads);
    p.heads[p.head_off[g] + fill[g]++] = static_cast<int16_t>(h);
  }
  const int sms = tree_sms();
  if (sms <= 0) return CFR_ERR_CUDA;
  if (!workspace || !ptr_aligned(workspace, 256) ||
      workspace_bytes < tree_scratch(sms, num_queries * num_q_heads, kv->head_dim).total)
    return CFR_ERR_WORKSPACE;
  for (int f = 0; f < kFmtCount; ++f) {
    p.k_pool[f] = c.k_pool[f];
    p.v_pool[f] = c.v_pool[f];
    p.scales[f] = c.scales[f];
    p.pool_pages[f] = c.pool_pages[f];
  }
  p.q = q;
  p.page_table = page_table;
  p.page_fmt = page_fmt;
  p.seq_lens = seq_lens;
  p.q_lens = q_lens;
  p.mask = reinterpret_cast<const unsigned long long *>(tree_mask);
  p.depths = depths;
  p.slopes = alibi_slopes;
  p.out = out;
  p.lse = lse;
  p.err = err_word;
  p.q_fmt = q_fmt;
  p.out_fmt = out_fmt;
  p.uniform_fmt = uniform_fmt;
  p.batch = batch;
  p.max_pages = max_pages;
  p.Hq = num_q_heads;
  p.Hkv = kv->num_kv_heads;
  p.D = kv->head_dim;
  p.P = kv->page_tokens;
  p.nq = num_queries;
  p.sigma = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf(static_cast<float>(kv->head_dim));
  p.cap = logit_cap;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int most = 0;
  for (int g = 0; g < kv->num_kv_heads; ++g) most = count[g] > most ? count[g] : most;
  const bool tc = tree_tc_supported(p);
  const int rb = tc ? tree_tc_rows(most * num_queries) : kGenRB;
  p.grid = tc ? sms : general_grid(sms);
  const TreeWs w = tree_ws(2 * p.grid, rb, p.D);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.part_m = reinterpret_cast<float *>(ws + w.part_m);
  p.part_l = reinterpret_cast<float *>(ws + w.part_l);
  p.part_acc = reinterpret_cast<float *>(ws + w.part_acc);
  cudaError_t e = tc ? launch_tree_tc(p, rb, s) : p.D == 128 ? launch_general<128>(p, s) : launch_general<64>(p, s);
  if (e != cudaSuccess) return CFR_ERR_CUDA;
  e = !tc ? launch_tree_merge<kGenTT, kGenRB>(p, s)
      : rb == 64 ? launch_tree_merge<128, 64>(p, s)
                  : launch_tree_merge<128, 256>(p, s);
  return e == cudaSuccess ? CFR_OK : CFR_ERR_CUDA;
}

}  // extern "C"
