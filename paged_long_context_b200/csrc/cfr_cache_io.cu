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

constexpr int kWriteResident = 8;  // vectors a thread holds between the passes

template <int IN>
__global__ void __launch_bounds__(512) write_kernel(const __grid_constant__ ChunkParams p) {
  __shared__ int sb;
  __shared__ float red[16];
  const int tid = threadIdx.x, T = blockDim.x;
  const int heads2 = 2 * p.c.Hkv;
  const int which = blockIdx.x % heads2;
  const int seg = blockIdx.x / heads2;
  const int g = which >> 1, kv = which & 1;
  if (tid == 0) sb = -1;
  __syncthreads();
  for (int i = tid; i < p.c.batch; i += T) {
    const int lo = p.row_off[i] / p.c.P + 2 * i;
    if (lo <= seg && (i + 1 == p.c.batch || p.row_off[i + 1] / p.c.P + 2 * (i + 1) > seg)) sb = i;
    if (blockIdx.x == 0) chunk_of(p, i);  // reports offsets that no CTA below would look at
  }
  __syncthreads();
  const int b = sb;
  if (b < 0) return;
  const Chunk k = chunk_of(p, b);
  if (k.n == 0) return;
  const int P = p.c.P, D = p.c.D;
  const long long lp = k.start / P + (seg - (k.r0 / P + 2 * b));  // the CTA's logical page
  const long long t0 = max(static_cast<long long>(k.start), lp * P);
  const long long t1 = min(static_cast<long long>(k.start) + k.n, (lp + 1) * P);
  if (t0 >= t1) return;
  int fmt;
  long long slot;
  if (!resolve_page(p.c, b, static_cast<int>(lp), kAllFormats, fmt, slot)) return;
  const int tin = static_cast<int>(t0 - lp * P);  // first new row of the page
  const int vpr = D / kVec;                       // vectors of a row
  const int nvec = static_cast<int>(t1 - t0) * vpr;
  const long long stride = kv ? p.v_stride : p.k_stride;
  constexpr int EB = IN == CFR_FMT_F32 ? 4 : 2;
  const uint8_t *src = static_cast<const uint8_t *>(kv ? p.v_in : p.k_in) +
                       ((k.r0 + (t0 - k.start)) * stride + static_cast<long long>(g) * D) * EB;
  uint8_t *page = (kv ? p.c.v_pool[fmt] : p.c.k_pool[fmt]) + row_at(p.c, fmt, slot, g, 0);
  const auto load = [&](int v) {
    const int row = v / vpr;
    return load_raw<IN>(src + row * stride * EB, v - row * vpr);
  };
  float scale = 1.f;
  RawVec<IN> buf[kWriteResident];
  const bool resident = nvec <= kWriteResident * T;
  if (is_quantised(fmt)) {
    float amax = 0.f;
    for (int v0 = 0; v0 < nvec; v0 += kWriteResident * T) {
#pragma unroll
      for (int i = 0; i < kWriteResident; ++i)
        if (v0 + i * T + tid < nvec) buf[i] = load(v0 + i * T + tid);
#pragma unroll
      for (int i = 0; i < kWriteResident; ++i) {
        if (v0 + i * T + tid < nvec) {
          float x[kVec];
          decode_raw<IN>(buf[i], 1.f, x);
#pragma unroll
          for (int e = 0; e < kVec; ++e) amax = fmaxf(amax, fabsf(x[e]));
        }
      }
    }
    float *stored = p.c.scales[fmt] + (slot * p.c.Hkv + g) * 2 + kv;
    const float old = *stored;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    __syncthreads();  // every thread has read the old scale by here
    amax = red[0];
    for (int w = 1; w < T / 32; ++w) amax = fmaxf(amax, red[w]);
    scale = __fdiv_rn(amax, qmax_of(fmt));
    if (tin > 0) {
      scale = fmaxf(scale, old);
      if (scale != old) {  // the kept rows, each vector by one thread
        for (int v = tid; v < tin * vpr; v += T) {
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
  }
  const long long base = static_cast<long long>(tin) * D;
  for (int v0 = 0; v0 < nvec; v0 += kWriteResident * T) {
    if (!resident || !is_quantised(fmt)) {
#pragma unroll
      for (int i = 0; i < kWriteResident; ++i)
        if (v0 + i * T + tid < nvec) buf[i] = load(v0 + i * T + tid);
    }
#pragma unroll
    for (int i = 0; i < kWriteResident; ++i) {
      const int v = v0 + i * T + tid;
      if (v < nvec) {
        float x[kVec];
        decode_raw<IN>(buf[i], 1.f, x);
        store8(fmt, page, base + static_cast<long long>(v) * kVec, scale, x);
      }
    }
  }
}

// ---- read --------------------------------------------------------------------

constexpr int kReadThreads = 256, kReadRows = 8;

template <int OUT>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ChunkParams p) {
  __shared__ int sfmt[kReadRows], stin[kReadRows];
  __shared__ long long sslot[kReadRows];
  const int tid = threadIdx.x;
  const int row0 = blockIdx.x * kReadRows;
  if (tid < kReadRows) {
    const int row = row0 + tid;
    int fmt = -1;
    long long slot = 0;
    int tin = 0;
    if (row < p.num_rows) {
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
    sfmt[tid] = fmt;
    stin[tid] = tin;
    sslot[tid] = slot;
  }
  if (blockIdx.x == 0)
    for (int i = tid; i < p.c.batch; i += kReadThreads) chunk_of(p, i);
  __syncthreads();
  const int D = p.c.D, vpr = D / kVec;
  const int per = p.c.Hkv * vpr;  // vectors of a row of K or V
  constexpr int EB = OUT == CFR_FMT_F32 ? 4 : 2;
  for (int i = tid; i < 2 * kReadRows * per; i += kReadThreads) {
    const int kv = i >= kReadRows * per;
    const int e = kv ? i - kReadRows * per : i;
    const int r = e / per, in_row = e - r * per;
    const int fmt = sfmt[r];
    if (fmt < 0) continue;
    const int g = in_row / vpr, c8 = in_row - g * vpr;
    const uint8_t *src = (kv ? p.c.v_pool[fmt] : p.c.k_pool[fmt]) + row_at(p.c, fmt, sslot[r], g, stin[r]);
    const float scale = is_quantised(fmt) ? p.c.scales[fmt][(sslot[r] * p.c.Hkv + g) * 2 + kv] : 1.f;
    float x[kVec];
    switch (fmt) {
      case CFR_FMT_F32: decode_raw<CFR_FMT_F32>(load_raw<CFR_FMT_F32>(src, c8), 1.f, x); break;
      case CFR_FMT_BF16: decode_raw<CFR_FMT_BF16>(load_raw<CFR_FMT_BF16>(src, c8), 1.f, x); break;
      case CFR_FMT_I8: decode_raw<CFR_FMT_I8>(load_raw<CFR_FMT_I8>(src, c8), scale, x); break;
      case CFR_FMT_I4: decode_raw<CFR_FMT_I4>(load_raw<CFR_FMT_I4>(src, c8), scale, x); break;
      default: decode_raw<CFR_FMT_FP8>(load_raw<CFR_FMT_FP8>(src, c8), scale, x); break;
    }
    uint8_t *dst = static_cast<uint8_t *>(kv ? p.v_out : p.k_out) +
                   (static_cast<long long>(row0 + r) * (kv ? p.v_stride : p.k_stride) + static_cast<long long>(g) * D) * EB;
    store8(OUT, dst, c8 * kVec, 1.f, x);
  }
}

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
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(num_rows) + kReadRows - 1) / kReadRows);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (out_fmt == CFR_FMT_F32)
    read_kernel<CFR_FMT_F32><<<blocks, kReadThreads, 0, s>>>(p);
  else
    read_kernel<CFR_FMT_BF16><<<blocks, kReadThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? CFR_OK : CFR_ERR_CUDA;
}

}  // extern "C"
