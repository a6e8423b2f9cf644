// cfr_cache_io.cu -- a ragged chunk of new tokens into pages of any storage
// format (quantised as it is written), and cached tokens back as dense rows.
//
// Write.  A quantised page has one scale per kv head for K and one for V, so a
// page, not a row, is what can be coded on its own:
//   scale' = max(kept ? scale : 0, max|x| / Q),
//   kept rows: code <- nearest(code * scale / scale') when scale' > scale,
//   new rows:  code  = nearest(x / scale').
// One CTA per (touched page of a sequence, kv head, K or V): pass 1 takes max|x|
// over the page's new rows and pass 2 codes them, from registers when the rows fit them.  Which pages
// are touched stands in device memory only, so the grid covers the most pages
// that `num_rows` rows of `batch` sequences can touch: sequence b's k-th touched page is CTA
// row_offsets[b] / P + 2 b + k, and a CTA finds its b by comparing all of them
// at once.  (L rows touch at most L / P + 2 pages of P, wherever they start, so
// the numbers never collide.)
//
// Read-back.  One CTA per few rows of the output; the rows' places are
// resolved once, one row a thread, and every thread then expands vectors of
// eight values.
//
// Both are bound by HBM: dense rows once, stored rows once.
#include "cfr_cells.cuh"

namespace cfr {
namespace {

struct ChunkParams {
  CacheView c;
  const int32_t *row_off, *starts;
  const void *k_in, *v_in;  // write
  void *k_out, *v_out;      // read
  long long k_stride, v_stride;
  int dense_fmt, num_rows;
};

// the chunk of sequence b: its dense rows [r0, r0 + n) and first token; n = 0,
// with the error word set, when its offsets or tokens are out of range
struct Chunk {
  int r0, n, start;
};
__device__ __forceinline__ Chunk chunk_of(const ChunkParams &p, int b) {
  Chunk k{p.row_off[b], 0, p.starts[b]};
  const int r1 = p.row_off[b + 1];
  if (k.r0 == r1 && k.r0 >= 0 && r1 <= p.num_rows) return k;
  if (k.r0 < 0 || r1 < k.r0 || r1 > p.num_rows || k.start < 0 ||
      static_cast<long long>(k.start) + (r1 - k.r0) > static_cast<long long>(p.c.max_pages) * p.c.P) {
    set_err(p.c.err, CFR_DEVERR_SEQ_LEN);
    return k;
  }
  k.n = r1 - k.r0;
  return k;
}

// ---- write -------------------------------------------------------------------

// vectors a thread holds between the passes: 512 threads hold a page of 256 tokens x 128 bf16 values, with
// two blocks on an SM, so that one's loads run under the other's encoding
template <int IN>
constexpr int kWriteResident = IN == CFR_FMT_F32 ? 4 : 8;

// Stores vectors v0, v0 + T, ... (in `buf`) of a page's new rows as codes.  Vectors near a
// tie (a warp nearly always has one) are marked and, behind the loop, read and encoded again with the
// division, one copy of whose code serves all: unrolled over `buf` it overran the
// instruction cache, whose refills took a third of the kernel's time.
template <int IN, int DST, int R, typename Again>
__device__ __forceinline__ void store_coded(uint8_t *dst, const RawVec<IN> (&buf)[R], int v0, int T, int nvec, float scale,
                                            bool fast, float r_lo, float r_hi, Again again) {
  uint32_t redo = 0u;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int v = v0 + i * T;
    if (v >= nvec) continue;
    float x[kVec];
    decode_raw<IN>(buf[i], 1.f, x);
    uint32_t tb[kVec];
    const bool near = codes8_fast<DST>(x, r_lo, r_hi, tb);
    if (near || !fast)
      redo |= 1u << i;
    else
      store_codes8<DST>(dst, v, tb);
  }
#pragma unroll 1
  while (redo) {
    const int v = v0 + (__ffs(redo) - 1) * T;
    redo &= redo - 1;
    float x[kVec];
    decode_raw<IN>(again(v), 1.f, x);
    uint32_t tb[kVec];
    codes8_exact<DST>(x, scale, tb);
    store_codes8<DST>(dst, v, tb);
  }
}

template <int IN>
__global__ void __launch_bounds__(512, IN == CFR_FMT_F32 ? 1 : 2) write_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int R = kWriteResident<IN>;
  __shared__ int found;   // the block's sequence
  __shared__ float red[16];
  const int tid = threadIdx.x, T = blockDim.x;
  const int heads2 = 2 * p.c.Hkv;
  const int which = blockIdx.x % heads2;
  const int seg = blockIdx.x / heads2;
  const int g = which >> 1, kv = which & 1;
  const int P = p.c.P, D = p.c.D;
  if (tid == 0) found = -1;
  __syncthreads();
  for (int i = tid; i < p.c.batch; i += T) {
    const int r0 = p.row_off[i], r1 = p.row_off[i + 1];
    // (more than one, where offsets are out of order)
    if (r0 / P + 2 * i <= seg && (i + 1 == p.c.batch || r1 / P + 2 * (i + 1) > seg)) atomicMax(&found, i);
    if (blockIdx.x == 0) chunk_of(p, i);   // reports offsets that no other block would look at
  }
  __syncthreads();
  const int b = found;
  if (b < 0) return;
  const Chunk mine = chunk_of(p, b);
  const int r0 = mine.r0, n = mine.n, start = mine.start;
  if (n == 0) return;
  const long long lp = start / P + (seg - (r0 / P + 2 * b));  // the block's logical page
  const long long t0 = max(static_cast<long long>(start), lp * P);
  const long long t1 = min(static_cast<long long>(start) + n, (lp + 1) * P);
  if (t0 >= t1) return;
  int fmt;
  long long slot;
  if (!resolve_page(p.c, b, static_cast<int>(lp), kAllFormats, fmt, slot)) return;
  const int tin = static_cast<int>(t0 - lp * P);  // first new row of the page
  const int vshift = D == 128 ? 4 : 3, vpr = 1 << vshift;   // vectors of a row
  const int nvec = static_cast<int>(t1 - t0) << vshift;
  constexpr int EB = IN == CFR_FMT_F32 ? 4 : 2;
  const long long stride = (kv ? p.v_stride : p.k_stride) * EB;
  const uint8_t *src = static_cast<const uint8_t *>(kv ? p.v_in : p.k_in) + (r0 + (t0 - start)) * stride +
                       static_cast<long long>(g) * D * EB;
  uint8_t *page = (kv ? p.c.v_pool[fmt] : p.c.k_pool[fmt]) + row_at(p.c, fmt, slot, g, 0);
  uint8_t *rows = page + static_cast<long long>(tin) * row_bytes(fmt, D);
  RawVec<IN> buf[R];
  const auto vec = [&](int v) { return load_raw<IN>(src + (v >> vshift) * stride, v & (vpr - 1)); };
  const auto load = [&](int v0) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (v0 + i * T < nvec) buf[i] = vec(v0 + i * T);
  };
  if (!is_quantised(fmt)) {
#pragma unroll 1
  for (int v0 = tid; v0 < nvec; v0 += R * T) {
      load(v0);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int v = v0 + i * T;
        if (v >= nvec) continue;
        float x[kVec];
        decode_raw<IN>(buf[i], 1.f, x);
        store8(fmt, rows, static_cast<long long>(v) * kVec, 1.f, x);
      }
    }
    return;
  }
  // pass 1: max|x| of the new rows
  float *stored = p.c.scales[fmt] + (slot * p.c.Hkv + g) * 2 + kv;
  const float old = *stored;
  float amax = 0.f;
#pragma unroll 1
  for (int v0 = tid; v0 < nvec; v0 += R * T) {
    load(v0);
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (v0 + i * T >= nvec) continue;
      if constexpr (IN == CFR_FMT_BF16) {
        m = absmax_acc(absmax_acc(absmax_acc(absmax_acc(m, buf[i].a.x), buf[i].a.y), buf[i].a.z), buf[i].a.w);
      } else {
        float x[kVec];
        decode_raw<IN>(buf[i], 1.f, x);
#pragma unroll
        for (int e = 0; e < kVec; ++e) amax = fmaxf(amax, fabsf(x[e]));
      }
    }
    if (IN == CFR_FMT_BF16) amax = fmaxf(amax, absmax_value(m));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((tid & 31) == 0) red[tid >> 5] = amax;
  __syncthreads();  // every thread has read the old scale by here
  amax = red[0];
  for (int w = 1; w < T / 32; ++w) amax = fmaxf(amax, red[w]);
  float scale = __fdiv_rn(amax, qmax_of(fmt));
  if (tin > 0) {
    scale = fmaxf(scale, old);
    if (scale != old) {  // the kept rows, each vector by one thread
      for (int v = tid; v < tin << vshift; v += T) {
        float x[kVec];
        if (fmt == CFR_FMT_I8)
          decode_raw<CFR_FMT_I8>(load_raw<CFR_FMT_I8>(page, v), old, x);
        else if (fmt == CFR_FMT_I4)
          decode_raw<CFR_FMT_I4>(load_raw<CFR_FMT_I4>(page, v), old, x);
        else
          decode_raw<CFR_FMT_FP8>(load_raw<CFR_FMT_FP8>(page, v), old, x);
        store8(fmt, page, static_cast<long long>(v) * kVec, scale, x);
      }
    }
  }
  if (tid == 0) *stored = scale;
  // pass 2: codes, from the registers where the rows fit them
  const bool fast = scale >= 1.17549435e-38f && scale <= 3.40282347e+38f;  // normal and finite
  const float r = __frcp_rn(scale), r_lo = __fmul_rn(r, 1.f - 0x1p-20f), r_hi = __fmul_rn(r, 1.f + 0x1p-20f);
  const bool resident = nvec <= R * T;
#pragma unroll 1
  for (int v0 = tid; v0 < nvec; v0 += R * T) {
    if (!resident) load(v0);
    if (fmt == CFR_FMT_I8)
      store_coded<IN, CFR_FMT_I8, R>(rows, buf, v0, T, nvec, scale, fast, r_lo, r_hi, vec);
    else if (fmt == CFR_FMT_I4)
      store_coded<IN, CFR_FMT_I4, R>(rows, buf, v0, T, nvec, scale, fast, r_lo, r_hi, vec);
    else
      store_coded<IN, CFR_FMT_FP8, R>(rows, buf, v0, T, nvec, scale, fast, r_lo, r_hi, vec);
  }
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
  p->dense_fmt = dense_fmt;
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
  const long long blocks = segs * kv->num_kv_heads * 2;
  if (blocks > INT_MAX) return CFR_ERR_OVERFLOW;
  if (num_rows == 0) return CFR_OK;
  p.k_in = k_new;
  p.v_in = v_new;
  // threads for one vector each of a small page, up to 512
  int threads = kv->page_tokens * (kv->head_dim / kVec);
  threads = threads < 64 ? 64 : threads > 512 ? 512 : (threads + 31) / 32 * 32;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (new_fmt == CFR_FMT_F32)
    write_kernel<CFR_FMT_F32><<<static_cast<unsigned>(blocks), threads, 0, s>>>(p);
  else
    write_kernel<CFR_FMT_BF16><<<static_cast<unsigned>(blocks), threads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? CFR_OK : CFR_ERR_CUDA;
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
  // rows of a block: 32 where that leaves a block for every SM several times over, fewer for
  // short chunks (a few hundred rows have to reach all SMs)
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
