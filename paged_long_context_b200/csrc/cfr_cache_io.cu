// cfr_cache_io.cu -- a ragged chunk of new tokens into pages of any storage
// format (quantised as it is written), and cached tokens back as dense rows.
//
// Write.  A quantised page has one scale per kv head for K and one for V, so a
// page, not a row, is what can be coded on its own:
//   scale' = max(kept ? scale : 0, max|x| / Q),
//   kept rows: code <- nearest(code * scale / scale') when scale' > scale,
//   new rows:  code  = nearest(x / scale').
// A team of 32 to 256 threads takes one (touched page of a sequence, kv head, K or V):
// its new rows come into shared memory by asynchronous copies, pass 1 takes max|x|
// over them and pass 2 codes them.  Which pages are touched stands in device memory
// only, so the grid covers the most pages that `num_rows` rows of `batch`
// sequences can touch: sequence b's k-th touched page is number
// row_offsets[b] / P + 2 b + k, and a CTA finds its b by search.  (L rows touch at
// most L / P + 2 pages of P, wherever they start, so the numbers never collide.)
//
// Read-back.  One CTA per few rows of the output; the rows' places are
// resolved once, one row a thread, and every thread then expands vectors of
// eight values.
//
// Floor of both: HBM, dense rows once and stored rows once.  The write comes to 3.1 TB/s (34K bf16 tokens of 8
// heads of 128 into int4 pages: 52 us): about twelve instructions a value take half the
// issue slots, and a page's two passes leave gaps that three blocks an SM do not
// close.  Read-back of long chunks runs near the copy rate (eight sequences of 9K to 32K tokens of tiers to bf16: 176
// us, 6.1 TB/s); shorter ones are a wave or two of blocks (34K int4 tokens to bf16: 43 us, 4.1 TB/s; 8K: 11 us).
#include <type_traits>

#include "cfr_cells.cuh"

namespace cfr {
namespace {

struct ChunkParams {
  CacheView c;
  const int32_t *row_off, *starts;
  const void *k_in, *v_in;  // write
  void *k_out, *v_out;      // read
  long long k_stride, v_stride;
  int num_rows;
};

// the chunk of sequence b: its dense rows [r0, r0 + n) and first token; n = 0,
// with the error word set, when its offsets or tokens are out of range
struct Chunk {
  int r0, n, start;
};
__device__ __forceinline__ Chunk chunk_of(const ChunkParams &p, int r0, int r1, int start) {
  Chunk k{r0, 0, start};
  if (k.r0 == r1 && k.r0 >= 0 && r1 <= p.num_rows) return k;
  if (k.r0 < 0 || r1 < k.r0 || r1 > p.num_rows || k.start < 0 ||
      static_cast<long long>(k.start) + (r1 - k.r0) > static_cast<long long>(p.c.max_pages) * p.c.P) {
    set_err(p.c.err, CFR_DEVERR_SEQ_LEN);
    return k;
  }
  k.n = r1 - k.r0;
  return k;
}
__device__ __forceinline__ Chunk chunk_of(const ChunkParams &p, int b) {
  return chunk_of(p, p.row_off[b], p.row_off[b + 1], p.starts[b]);
}

// ---- write -------------------------------------------------------------------

// A block's new rows wait in shared memory between the passes, up to 64 KiB of them (a page of 256 tokens x 128
// bf16 values; three such blocks fit an SM, so that one's loads run under the others' encoding).
constexpr int kWriteStage = 65536;
constexpr int kWriteThreads = 256;
constexpr int kTeamVectors = 16;       // vectors of a page for each thread of a team, up to the block's threads

// Eight values of vector v stored as codes: by the quotients where the scale allows it, else (and where a NaN is
// among integers) with the division.
template <int DST, bool CLAMP>
__device__ __forceinline__ void store_coded(uint8_t *dst, int v, const float (&x)[kVec], float scale, float r, bool fast) {
  if (!fast || !store_quotients8<DST, CLAMP>(dst, v, x, r, scale)) store8(DST, dst, static_cast<long long>(v) * kVec, scale, x);
}

__device__ __forceinline__ void copy_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src)
               : "memory");
}

// the kept rows of a page (nvec vectors) under a new scale
template <int FMT>
__device__ __forceinline__ void store_kept(uint8_t *page, int tid, int T, int nvec, float old, float scale, float r, bool fast) {
#pragma unroll 1
  for (int v = tid; v < nvec; v += T) {
    float x[kVec];
    decode_raw<FMT>(load_raw<FMT>(page, v), old, x);
    store_coded<FMT, true>(page, v, x, scale, r, fast);
  }
}

// T = 32 .. 256 threads, a team, take a page of one kv head, K or V: a sixteenth of its vectors,
// so that what a page costs before its values (finding the sequence, resolving the page, joining the
// maxima) is spread over sixteen vectors a thread.  (34K tokens into pages of 32 as int4, written and read back:
// 96 us with sixteen, 100 with eight, 160 with two; into pages of 64: 97 with sixteen, 123 with thirty-two.)
//
// Warp 0 works out the block's page, once for all.
struct WritePage {
  long long slot, src_row;   // of the first new row, in the dense rows
  int fmt, tin, rows;        // fmt -1: nothing to write; first new row of the page, new rows
  int which;                 // first (kv head, K or V) of the block
};

__device__ __forceinline__ void find_page(const ChunkParams &p, int blocks, int each, WritePage *at) {
  const int lane = threadIdx.x, P = p.c.P;
  const int seg = blockIdx.x / blocks;
  // the last sequence whose first touched page is numbered seg or less, 32 probes at a time; its offsets
  // and start come with the probes, not behind them
  int lo = 0, hi = p.c.batch, r0, r1, start;
  do {
    const int step = (hi - lo + 31) >> 5;
    const int i = static_cast<int>(min(lo + static_cast<long long>(lane) * step, hi - 1LL));
    r0 = p.row_off[i];
    r1 = p.row_off[i + 1];
    start = p.starts[i];
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, lane == 0 || (lo + static_cast<long long>(lane) * step < hi &&
                                                                         r0 / P + 2LL * i <= seg)));
    r0 = __shfl_sync(0xffffffffu, r0, last);
    r1 = __shfl_sync(0xffffffffu, r1, last);
    start = __shfl_sync(0xffffffffu, start, last);
    lo += last * step;
    hi = min(hi, lo + step);
  } while (hi - lo > 1);
  if (lane > 0) return;
  at->fmt = -1;
  at->which = (blockIdx.x - seg * blocks) * each;
  const Chunk mine = chunk_of(p, r0, r1, start);
  const int k = seg - (mine.r0 / P + 2 * lo);   // page of the sequence's touched ones
  if (mine.n == 0 || k < 0) return;
  const long long lp = mine.start / P + static_cast<long long>(k);
  const long long t0 = max(static_cast<long long>(mine.start), lp * P);
  const long long t1 = min(static_cast<long long>(mine.start) + mine.n, (lp + 1) * P);
  int fmt;
  long long slot;
  if (t0 >= t1 || !resolve_page(p.c, lo, static_cast<int>(lp), kAllFormats, fmt, slot)) return;
  at->fmt = fmt;
  at->slot = slot;
  at->src_row = mine.r0 + (t0 - mine.start);
  at->tin = static_cast<int>(t0 - lp * P);
  at->rows = static_cast<int>(t1 - t0);
}

// `blocks`: blocks of a touched page; 1 << shift: threads of a team; team_stage: its bytes of shared memory
template <int IN>
__global__ void __launch_bounds__(kWriteThreads, 3) write_kernel(const __grid_constant__ ChunkParams p, int blocks, int shift, int team_stage) {
  extern __shared__ __align__(16) uint8_t stage[];
  __shared__ WritePage page_of;
  __shared__ float red[kWriteThreads / 32];
  const int T = 1 << shift, team = threadIdx.x >> shift, tid = threadIdx.x & (T - 1);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.c.batch; i += blockDim.x) chunk_of(p, i);   // reports all that are out of order
  if (threadIdx.x < 32) find_page(p, blocks, blockDim.x >> shift, &page_of);
  __syncthreads();
  const int fmt = page_of.fmt, which = page_of.which + team;
  if (fmt < 0 || which >= 2 * p.c.Hkv) return;   // (only barriers of a team below)
  const int g = which >> 1, kv = which & 1, D = p.c.D;
  const long long slot = page_of.slot;
  const int tin = page_of.tin;
  const int vshift = D == 128 ? 4 : 3, vpr = 1 << vshift;   // vectors of a row
  const int nvec = page_of.rows << vshift;
  constexpr int EB = IN == CFR_FMT_F32 ? 4 : 2;
  const long long stride = (kv ? p.v_stride : p.k_stride) * EB;
  const uint8_t *src = static_cast<const uint8_t *>(kv ? p.v_in : p.k_in) + page_of.src_row * stride +
                       static_cast<long long>(g) * D * EB;
  uint8_t *page = (kv ? p.c.v_pool[fmt] : p.c.k_pool[fmt]) + row_at(p.c, fmt, slot, g, 0);
  uint8_t *rows = page + static_cast<long long>(tin) * row_bytes(fmt, D);
  constexpr int VB = kVec * EB;   // bytes of a vector
  // a thread's vectors are tid, tid + T, ...: the same place of rows T / vpr apart
  src += (tid >> vshift) * stride + (tid & (vpr - 1)) * VB;
  const long long step = (T >> vshift) * stride;
  if (!is_quantised(fmt)) {
#pragma unroll 4
    for (int v = tid; v < nvec; v += T, src += step) {
      float x[kVec];
      decode_raw<IN>(load_raw<IN>(src, 0), 1.f, x);
      store8(fmt, rows, static_cast<long long>(v) * kVec, 1.f, x);
    }
    return;
  }
  // the new rows, each vector by the thread that takes it in both passes
  const int held = min(nvec, team_stage / VB);   // those that shared memory has room for (the others are read twice)
  uint8_t *mine = stage + team * team_stage;
  const uint8_t *at = src;
#pragma unroll 4
  for (int v = tid; v < held; v += T, at += step) {
    copy_async16(mine + v * VB, at);
    if (VB == 32) copy_async16(mine + v * VB + 16, at + 16);
  }
  float *stored = p.c.scales[fmt] + (slot * p.c.Hkv + g) * 2 + kv;
  const float old = *stored;
  asm volatile("cp.async.wait_all;" ::: "memory");
  // pass 1: max|x| of the new rows
  float amax = 0.f;
  uint32_t m = 0u;
  const auto take = [&](const RawVec<IN> &raw) {
    if constexpr (IN == CFR_FMT_BF16) {
      m = absmax_acc(absmax_acc(absmax_acc(absmax_acc(m, raw.a.x), raw.a.y), raw.a.z), raw.a.w);
    } else {
      float x[kVec];
      decode_raw<IN>(raw, 1.f, x);
#pragma unroll
      for (int e = 0; e < kVec; ++e) amax = fmaxf(amax, fabsf(x[e]));
    }
  };
#pragma unroll 4
  for (int v = tid; v < held; v += T) take(load_raw<IN>(mine, v));
  const int first_far = tid + (held - tid + T - 1) / T * T;   // the thread's first vector past those (held >= T or all)
#pragma unroll 1
  for (int v = first_far; v < nvec; v += T, at += step) take(load_raw<IN>(at, 0));
  if (IN == CFR_FMT_BF16) amax = absmax_value(m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  // (every thread has read the old scale once it is past the barrier)
  if (T == 32) {
    __syncwarp();
  } else {
    float *mine_red = red + team * (T / 32);
    if ((tid & 31) == 0) mine_red[tid >> 5] = amax;
    named_sync(1 + team, T);
    amax = mine_red[tid & (T / 32 - 1)];
#pragma unroll
    for (int o = kWriteThreads / 64; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  }
  float scale = __fdiv_rn(amax, qmax_of(fmt));
  if (tin > 0) scale = fmaxf(scale, old);
  if (tid == 0) *stored = scale;
  const bool fast = scale >= kQuotientMin && scale <= kQuotientMax;
  const float r = __frcp_rn(scale);
  // the kept rows under the new scale; pass 2: codes of the new ones
  const int kept = tin > 0 && scale != old ? tin << vshift : 0;
  const auto store = [&](auto dst) {
    constexpr int DST = decltype(dst)::value;
    store_kept<DST>(page, tid, T, kept, old, scale, r, fast && fabsf(old) <= scale);   // (|code * old| <= Q scale but for -Q - 1)
#pragma unroll 1
    for (int v = tid; v < nvec; v += T, src += step) {
      float x[kVec];
      decode_raw<IN>(v < held ? load_raw<IN>(mine, v) : load_raw<IN>(src, 0), 1.f, x);
      store_coded<DST, false>(rows, v, x, scale, r, fast);
    }
  };
  if (fmt == CFR_FMT_I8)
    store(std::integral_constant<int, CFR_FMT_I8>());
  else if (fmt == CFR_FMT_I4)
    store(std::integral_constant<int, CFR_FMT_I4>());
  else
    store(std::integral_constant<int, CFR_FMT_FP8>());
}

// ---- read --------------------------------------------------------------------

constexpr int kReadThreads = 256;

// One row (of K or V), nvec vectors over its heads, by one warp, U vectors a lane at a time:
// a lane keeps its place in a head and steps over 32 / (vectors of a head) heads.
template <int SRC, int OUT>
__device__ __forceinline__ void read_row(const uint8_t *src, long long head_bytes, const float *scales, uint8_t *dst, int nvec,
                                         int vshift, int lane) {
  constexpr int U = SRC == CFR_FMT_F32 ? 2 : 4;
  const int hstep = 32 >> vshift;
  const long long step = hstep * head_bytes;
  const RawVec<SRC> *at = reinterpret_cast<const RawVec<SRC> *>(src + (lane >> vshift) * head_bytes) + (lane & ((1 << vshift) - 1));
  if (is_quantised(SRC)) scales += 2 * (lane >> vshift);
#pragma unroll 1
  for (int v0 = lane; v0 < nvec; v0 += 32 * U) {
    RawVec<SRC> raw[U];
    float scale[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (v0 + 32 * u < nvec) {
        raw[u] = *at;
        scale[u] = is_quantised(SRC) ? *scales : 1.f;
      }
      at = reinterpret_cast<const RawVec<SRC> *>(reinterpret_cast<const uint8_t *>(at) + step);
      if (is_quantised(SRC)) scales += 2 * hstep;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + 32 * u;
      if (v >= nvec) continue;
      if constexpr (SRC == OUT) {
        reinterpret_cast<RawVec<SRC> *>(dst)[v] = raw[u];
      } else {
        float x[kVec];
        decode_raw<SRC>(raw[u], scale[u], x);
        store8(OUT, dst, static_cast<long long>(v) * kVec, 1.f, x);
      }
    }
  }
}

// places of a block's rows
struct ReadRows {
  int fmt[32], tin[32];
  long long slot[32];
  uint32_t present;   // formats among them
};

// the block's rows of one format, a warp taking a row of K or of V at a time
template <int SRC, int OUT>
__device__ __forceinline__ void read_rows(const ChunkParams &p, const ReadRows &s, int per, int row0) {
  if (!((s.present >> SRC) & 1u)) return;
  constexpr int EB = OUT == CFR_FMT_F32 ? 4 : 2;
  const int lane = threadIdx.x & 31;
  const int vshift = p.c.D == 128 ? 4 : 3, nvec = p.c.Hkv << vshift;
  const long long head_bytes = static_cast<long long>(p.c.P) * row_bytes(SRC, p.c.D);
#pragma unroll 1
  for (int i = threadIdx.x >> 5; i < 2 * per; i += kReadThreads / 32) {
    const int r = i >> 1, kv = i & 1;
    if (s.fmt[r] != SRC) continue;
    const uint8_t *src = (kv ? p.c.v_pool[SRC] : p.c.k_pool[SRC]) + row_at(p.c, SRC, s.slot[r], 0, s.tin[r]);
    const float *scales = is_quantised(SRC) ? p.c.scales[SRC] + s.slot[r] * p.c.Hkv * 2 + kv : nullptr;
    uint8_t *dst = static_cast<uint8_t *>(kv ? p.v_out : p.k_out) +
                   static_cast<long long>(row0 + r) * (kv ? p.v_stride : p.k_stride) * EB;
    read_row<SRC, OUT>(src, head_bytes, scales, dst, nvec, vshift, lane);
  }
}

// `per`: rows of a block, at most 32
template <int OUT>
__global__ void __launch_bounds__(kReadThreads, 6) read_kernel(const __grid_constant__ ChunkParams p, int per) {
  __shared__ ReadRows s;
  const int tid = threadIdx.x;
  const int row0 = blockIdx.x * per;
  if (tid < 32) {
    const int row = row0 + tid;
    int fmt = -1;
    long long slot = 0;
    int tin = 0;
    if (tid < per && row < p.num_rows) {
      // the last sequence whose rows begin at or before this one
      int lo = 0, hi = p.c.batch;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.row_off[mid] <= row)
          lo = mid;
        else
          hi = mid;
      }
      const Chunk k = chunk_of(p, lo);
      if (k.n > 0 && row >= k.r0 && row < k.r0 + k.n) {
        const int j = k.start + (row - k.r0);
        if (!resolve_page(p.c, lo, j / p.c.P, kAllFormats, fmt, slot)) fmt = -1;
        tin = j % p.c.P;
      }
    }
    s.fmt[tid] = fmt;
    s.tin[tid] = tin;
    s.slot[tid] = slot;
    const uint32_t present = __reduce_or_sync(0xffffffffu, fmt >= 0 ? 1u << fmt : 0u);
    if (tid == 0) s.present = present;
  }
  if (blockIdx.x == 0)
    for (int i = tid; i < p.c.batch; i += kReadThreads) chunk_of(p, i);
  __syncthreads();
  // format by format: one loop that chose at every row kept the registers of all of them
  read_rows<CFR_FMT_BF16, OUT>(p, s, per, row0);
  read_rows<CFR_FMT_I8, OUT>(p, s, per, row0);
  read_rows<CFR_FMT_I4, OUT>(p, s, per, row0);
  read_rows<CFR_FMT_FP8, OUT>(p, s, per, row0);
  read_rows<CFR_FMT_F32, OUT>(p, s, per, row0);
}

// tokens of a page, whose vectors are counted in 32 bits
constexpr int kMaxChunkPage = 1 << 24;

// host checks shared by both directions
cfr_status chunk_params(const cfr_kv_pool *kv, const int32_t *page_table, int32_t max_pages,
                        const uint8_t *page_fmt, int32_t uniform_fmt, int32_t batch,
                        const int32_t *row_offsets, const int32_t *starts, const void *k,
                        int64_t k_stride, const void *v, int64_t v_stride, int32_t dense_fmt,
                        int32_t num_rows, uint32_t *err_word, ChunkParams *p) {
  cfr_status st = make_view(kv, page_table, max_pages, page_fmt, uniform_fmt, batch, kAllFormats,
                            err_word, &p->c);
  if (st != CFR_OK) return st;
  if (dense_fmt != CFR_FMT_F32 && dense_fmt != CFR_FMT_BF16) return CFR_ERR_INVALID_ARG;
  if (kv->page_tokens > kMaxChunkPage) return CFR_ERR_UNSUPPORTED;
  if (num_rows < 0 || !row_offsets || !starts) return CFR_ERR_INVALID_ARG;
  if (num_rows > 0 && (!rows_ok(k, k_stride, kv->num_kv_heads, kv->head_dim, dense_fmt) ||
                       !rows_ok(v, v_stride, kv->num_kv_heads, kv->head_dim, dense_fmt)))
    return CFR_ERR_INVALID_ARG;
  p->row_off = row_offsets;
  p->starts = starts;
  p->k_stride = k_stride;
  p->v_stride = v_stride;
  p->num_rows = num_rows;
  p->k_in = p->v_in = nullptr;
  p->k_out = p->v_out = nullptr;
  return CFR_OK;
}

}  // namespace
}  // namespace cfr

using namespace cfr;

extern "C" {

cfr_status cfr_write_kv(const cfr_kv_pool *kv, const int32_t *page_table, int32_t max_pages,
                        const uint8_t *page_fmt, int32_t uniform_fmt, int32_t batch,
                        const int32_t *row_offsets, const int32_t *starts, const void *k_new,
                        int64_t k_stride, const void *v_new, int64_t v_stride, int32_t new_fmt,
                        int32_t num_rows, uint32_t *err_word, void *stream) {
  ChunkParams p;
  cfr_status st = chunk_params(kv, page_table, max_pages, page_fmt, uniform_fmt, batch, row_offsets,
                               starts, k_new, k_stride, v_new, v_stride, new_fmt, num_rows, err_word, &p);
  if (st != CFR_OK) return st;
  const long long segs = static_cast<long long>(num_rows) / kv->page_tokens + 2LL * batch;
  const int vectors = kv->page_tokens * (kv->head_dim / kVec), heads2 = 2 * kv->num_kv_heads;
  int shift = 5;
  while (1 << shift < kWriteThreads && kTeamVectors << shift < vectors) ++shift;
  const int each = kWriteThreads >> shift;
  const int page_blocks = (heads2 + each - 1) / each;
  const long long blocks = segs * page_blocks;
  if (segs > INT_MAX / 2 || blocks > INT_MAX) return CFR_ERR_OVERFLOW;
  if (num_rows == 0) return CFR_OK;
  p.k_in = k_new;
  p.v_in = v_new;
  const int room = kWriteStage / each, vector_bytes = new_fmt == CFR_FMT_F32 ? 32 : 16;
  const int team_stage = vectors < room / vector_bytes ? vectors * vector_bytes : room;
  const auto launch = [&](auto kernel) {
    if (each * team_stage > 47 * 1024 &&   // (48 KiB without, the block's fixed shared memory among them)
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWriteStage) != cudaSuccess)
      return CFR_ERR_CUDA;
    kernel<<<static_cast<unsigned>(blocks), kWriteThreads, each * team_stage, static_cast<cudaStream_t>(stream)>>>(
        p, page_blocks, shift, team_stage);
    return cudaGetLastError() == cudaSuccess ? CFR_OK : CFR_ERR_CUDA;
  };
  return new_fmt == CFR_FMT_F32 ? launch(write_kernel<CFR_FMT_F32>) : launch(write_kernel<CFR_FMT_BF16>);
}

cfr_status cfr_read_kv(const cfr_kv_pool *kv, const int32_t *page_table, int32_t max_pages,
                       const uint8_t *page_fmt, int32_t uniform_fmt, int32_t batch,
                       const int32_t *row_offsets, const int32_t *starts, void *k_out,
                       int64_t k_stride, void *v_out, int64_t v_stride, int32_t out_fmt,
                       int32_t num_rows, uint32_t *err_word, void *stream) {
  ChunkParams p;
  cfr_status st = chunk_params(kv, page_table, max_pages, page_fmt, uniform_fmt, batch, row_offsets,
                               starts, k_out, k_stride, v_out, v_stride, out_fmt, num_rows, err_word, &p);
  if (st != CFR_OK) return st;
  if (num_rows == 0) return CFR_OK;
  p.k_out = k_out;
  p.v_out = v_out;
  // rows of a block: 32 from 600 blocks on (four an SM, of the six that are resident), fewer for
  // short chunks, which have to reach all SMs (eight sequences of 9K to 32K tokens of tiers: 178 us with 32, 203
  // with 4; 333 int8 tokens: 7.8 us with 32, 3.1 with 4)
  int per = 32;
  while (per > 4 && num_rows < per * 600) per >>= 1;
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(num_rows) + per - 1) / per);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (out_fmt == CFR_FMT_F32)
    read_kernel<CFR_FMT_F32><<<blocks, kReadThreads, 0, s>>>(p, per);
  else
    read_kernel<CFR_FMT_BF16><<<blocks, kReadThreads, 0, s>>>(p, per);
  return cudaGetLastError() == cudaSuccess ? CFR_OK : CFR_ERR_CUDA;
}

}  // extern "C"
