// cfr_rope.cu -- norms of queries and keys for each head, their position
// rotation, and the write of K and V into the hot tier, in one pass.
//
//   y <- y * rsqrt(mean(y^2) + eps) * w,   (a, b) <- (a c - b s, b c + a s)
//
// with c, s the cosine and sine of position * inv_freq.  The angle is reduced to
// one turn in fp64 (a position of a million times a frequency of 1 has an fp32
// ulp of 0.06 rad); its sine and cosine, the norm's sum and the products are
// fp32, rounded once where the row is stored.
//
// One CTA per token: its cosines and sines are computed once, by its first
// rotary_dim / 2 threads, and serve all of its query and key rows.  A row of
// head_dim values is head_dim / 8 lanes of eight values, 16 bytes of bf16 each;
// the row's sum of squares and, for pairs half a rotation apart, the partner
// values travel by shuffles, so nothing but the sines goes through shared
// memory.  Bound by HBM: every value is read once and written once.
#include "cfr_cells.cuh"

namespace cfr {
namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
  CacheView c;
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  void *q_out;
  const float *q_weight, *k_weight;
  const int32_t *rope_pos, *seq_ids, *token_ids;
  const double *inv_freq;
  float eps;
  int num_q_heads, rot, interleaved;
};

template <int IN, int D>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LPR = D / kVec;               // lanes of one row
  constexpr int RPI = kRopeThreads / LPR;     // rows of one step
  __shared__ float2 cs[D / 2];
  __shared__ long long place[3];              // format (-1: not written), slot, row
  const long long t = blockIdx.x;
  const int tid = threadIdx.x;
  if (tid < p.rot / 2) {
    constexpr double kInvTurn = 0.15915494309189533577;  // 1 / (2 pi)
    const double turns = static_cast<double>(p.rope_pos[t]) * p.inv_freq[tid] * kInvTurn;
    const float r = static_cast<float>(turns - rint(turns));
    float s, c;
    sincospif(2.f * r, &s, &c);
    cs[tid] = make_float2(c, s);
  }
  if (tid == kRopeThreads - 1) {
    const int b = p.seq_ids[t], j = p.token_ids[t];
    int fmt = -1;
    long long slot = 0;
    if (b >= 0 && j >= 0) {
      if (b >= p.c.batch || j >= static_cast<long long>(p.c.max_pages) * p.c.P)
        set_err(p.c.err, CFR_DEVERR_SEQ_LEN);
      else if (!resolve_page(p.c, b, j / p.c.P, kHotFormats, fmt, slot))
        fmt = -1;
    }
    place[0] = fmt;
    place[1] = slot;
    place[2] = j >= 0 ? j % p.c.P : 0;
  }
  __syncthreads();
  const int fmt = static_cast<int>(place[0]);
  const int rows = p.num_q_heads + 2 * p.c.Hkv;
  const int c8 = tid % LPR;                    // this lane's chunk of a row
  const int hl = p.rot / 16;                   // lanes of half a rotation
  const bool turned = c8 * kVec < p.rot;
  for (int r0 = 0; r0 < rows; r0 += RPI) {     // every lane of a warp takes every step
    const int r = r0 + tid / LPR;
    const bool is_q = r < p.num_q_heads, is_v = r >= p.num_q_heads + p.c.Hkv;
    const int head = is_q ? r : is_v ? r - p.num_q_heads - p.c.Hkv : r - p.num_q_heads;
    float x[kVec] = {};
    if (r < rows) {
      const void *src = is_q ? p.q : is_v ? p.v : p.k;
      const long long e = t * (is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride) +
                          static_cast<long long>(head) * D;
      decode_raw<IN>(load_raw<IN>(static_cast<const uint8_t *>(src) + e * (IN == CFR_FMT_F32 ? 4 : 2), c8), 1.f, x);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float *w = is_v ? nullptr : is_q ? p.q_weight : p.k_weight;
    if (w) {
      const float rs = rsqrtf(sum * (1.f / D) + p.eps);
      const float4 w0 = reinterpret_cast<const float4 *>(w)[2 * c8], w1 = reinterpret_cast<const float4 *>(w)[2 * c8 + 1];
      const float wv[kVec] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int i = 0; i < kVec; ++i) x[i] = x[i] * rs * wv[i];
    }
    if (p.interleaved) {
      if (turned && !is_v) {
#pragma unroll
        for (int i = 0; i < kVec; i += 2) {
          const float2 t2 = cs[c8 * (kVec / 2) + i / 2];
          const float a = x[i], b = x[i + 1];
          x[i] = a * t2.x - b * t2.y;
          x[i + 1] = b * t2.x + a * t2.y;
        }
      }
    } else if (p.rot > 0) {
      const bool upper = c8 >= hl;
      const int other = (tid & 31) - c8 + (turned ? (upper ? c8 - hl : c8 + hl) : c8);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float y = __shfl_sync(0xffffffffu, x[i], other);
        if (turned && !is_v) {
          const float2 t2 = cs[(upper ? c8 - hl : c8) * kVec + i];
          x[i] = upper ? fmaf(x[i], t2.x, y * t2.y) : fmaf(x[i], t2.x, -y * t2.y);
        }
      }
    }
    if (r < rows) {
      if (is_q) {
        const long long e = (t * p.num_q_heads + r) * D;
        store8(IN, static_cast<uint8_t *>(p.q_out) + e * (IN == CFR_FMT_F32 ? 4 : 2), c8 * kVec, 1.f, x);
      } else if (fmt >= 0) {
        uint8_t *pool = is_v ? p.c.v_pool[fmt] : p.c.k_pool[fmt];
        store8(fmt, pool + row_at(p.c, fmt, place[1], head, static_cast<int>(place[2])), c8 * kVec, 1.f, x);
      }
    }
  }
}

template <int IN>
void launch_rope(const RopeParams &p, int tokens, cudaStream_t s) {
  if (p.c.D == 128)
    rope_kernel<IN, 128><<<tokens, kRopeThreads, 0, s>>>(p);
  else
    rope_kernel<IN, 64><<<tokens, kRopeThreads, 0, s>>>(p);
}

}  // namespace
}  // namespace cfr

using namespace cfr;

extern "C" {

cfr_status cfr_qk_norm_rope_append(const cfr_kv_pool *kv, const int32_t *page_table,
                                   int32_t max_pages, const uint8_t *page_fmt,
                                   int32_t uniform_fmt, int32_t batch, const void *q,
                                   int64_t q_stride, const void *k, int64_t k_stride,
                                   const void *v, int64_t v_stride, int32_t in_fmt,
                                   int32_t num_tokens, int32_t num_q_heads,
                                   const float *q_weight, const float *k_weight, float eps,
                                   const int32_t *rope_positions, const double *inv_freq,
                                   int32_t rotary_dim, int32_t interleaved, void *q_out,
                                   const int32_t *seq_ids, const int32_t *token_ids,
                                   uint32_t *err_word, void *stream) {
  RopeParams p;
  cfr_status st = make_view(kv, page_table, max_pages, page_fmt, uniform_fmt, batch, kHotFormats,
                            err_word, &p.c);
  if (st != CFR_OK) return st;
  if (in_fmt != CFR_FMT_F32 && in_fmt != CFR_FMT_BF16) return CFR_ERR_INVALID_ARG;
  if (num_tokens < 0 || num_q_heads <= 0 || rotary_dim < 0 || !(eps >= 0.f) || eps == INFINITY)
    return CFR_ERR_INVALID_ARG;
  if (num_q_heads > kMaxQHeads || rotary_dim % 16 != 0 || rotary_dim > kv->head_dim)
    return CFR_ERR_UNSUPPORTED;
  if (num_tokens == 0) return CFR_OK;
  if (!rows_ok(q, q_stride, num_q_heads, kv->head_dim, in_fmt) ||
      !rows_ok(k, k_stride, kv->num_kv_heads, kv->head_dim, in_fmt) ||
      !rows_ok(v, v_stride, kv->num_kv_heads, kv->head_dim, in_fmt))
    return CFR_ERR_INVALID_ARG;
  if (!q_out || !ptr_aligned(q_out, 16) || !seq_ids || !token_ids) return CFR_ERR_INVALID_ARG;
  if (!ptr_aligned(q_weight, 16) || !ptr_aligned(k_weight, 16)) return CFR_ERR_INVALID_ARG;
  if (rotary_dim > 0 && (!rope_positions || !inv_freq || !ptr_aligned(inv_freq, 8)))
    return CFR_ERR_INVALID_ARG;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out = q_out;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.rope_pos = rope_positions;
  p.seq_ids = seq_ids;
  p.token_ids = token_ids;
  p.inv_freq = inv_freq;
  p.eps = eps;
  p.num_q_heads = num_q_heads;
  p.rot = rotary_dim;
  p.interleaved = interleaved != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (in_fmt == CFR_FMT_F32)
    launch_rope<CFR_FMT_F32>(p, num_tokens, s);
  else
    launch_rope<CFR_FMT_BF16>(p, num_tokens, s);
  return cudaGetLastError() == cudaSuccess ? CFR_OK : CFR_ERR_CUDA;
}

}  // extern "C"
