// cfr_rope.cu -- norms of queries and keys for each head, their position
// rotation, and the write of K and V into the hot tier, in one pass.
//
//   y <- y * rsqrt(mean(y^2) + eps) * w,   (a, b) <- (a c - b s, b c + a s)
//
// with c, s the cosine and sine of position * inv_freq.  The angle is reduced to
// an eighth of a turn either way in fp64 (a position of a million times a frequency of 1 has an fp32
// ulp of 0.06 rad, and half a turn in fp32 is still 2^-26 of a turn off); its sine and cosine, the norm's sum
// and the products are fp32, rounded once where the row is stored.
//
// A CTA takes one token of a short step, four of a long one: their cosines and
// sines are computed once, a thread each, behind one barrier, and serve all query
// and key rows, the first token's values being on their way meanwhile.  A row is
// head_dim / 8 lanes of eight values: where pairs lie half a rotation apart, four
// values of each half, so that a rotation needs no other lane; the row's sum of
// squares is the only thing that travels by shuffles.
//
// Every value is read once and written once, so HBM is the floor; a long step is bound by
// instruction issue, 21 instructions a value at 69 % of the issue slots: 17K tokens of 32 + 2 x 8 bf16 heads of
// 128 take 96 us, 4.5 TB/s (0.68 of the copy rate).  A decode step of one token: 3.4 us of GPU time, the launch and
// one chain of lookups.
#include "cfr_cells.cuh"

namespace cfr {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;   // most tokens of a CTA

struct RopeParams {
  CacheView c;
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  void *q_out;
  const float *q_weight, *k_weight;
  const int32_t *rope_pos, *seq_ids, *token_ids;
  const double *inv_freq;
  float eps;
  int num_q_heads, rot, num_tokens, per;   // per: tokens of a CTA
};

// four consecutive stored values
template <int FMT>
struct Quad {
  uint2 w;
};
template <>
struct Quad<CFR_FMT_F32> {
  uint4 w;
};
__device__ __forceinline__ void unpack4(const Quad<CFR_FMT_F32> &q, float *x) {
  x[0] = __uint_as_float(q.w.x);
  x[1] = __uint_as_float(q.w.y);
  x[2] = __uint_as_float(q.w.z);
  x[3] = __uint_as_float(q.w.w);
}
__device__ __forceinline__ void unpack4(const Quad<CFR_FMT_BF16> &q, float *x) {
  x[0] = bf16_lo(q.w.x);
  x[1] = bf16_hi(q.w.x);
  x[2] = bf16_lo(q.w.y);
  x[3] = bf16_hi(q.w.y);
}
__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void put4(int fmt, uint8_t *row, int e, const float *x) {
  if (fmt == CFR_FMT_F32)
    *reinterpret_cast<float4 *>(row + 4 * e) = make_float4(x[0], x[1], x[2], x[3]);
  else
    *reinterpret_cast<uint2 *>(row + 2 * e) = make_uint2(pair_bf16(x[0], x[1]), pair_bf16(x[2], x[3]));
}

template <int IN, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, IN == CFR_FMT_F32 ? 3 : 4) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LPR = D / kVec;               // lanes of one row
  constexpr int RPI = kRopeThreads / LPR;     // rows of one step
  constexpr int AHEAD = 3;                    // steps whose rows are loaded at once
  constexpr int EB = IN == CFR_FMT_F32 ? 4 : 2;
  __shared__ __align__(16) float cosines[kRopeTokens][D / 2], sines[kRopeTokens][D / 2];
  __shared__ long long place[kRopeTokens][2];  // format (-1: not written); row of the first head in its pool
  const long long first_t = static_cast<long long>(blockIdx.x) * p.per;
  const int tokens = static_cast<int>(min(static_cast<long long>(p.per), p.num_tokens - first_t));
  const int tid = threadIdx.x;
  const int hq = p.num_q_heads, hkv = p.c.Hkv, rows = hq + 2 * hkv;
  const int c8 = tid % LPR, r_mine = tid / LPR;
  // this lane's values: e0 .. e0 + 3 and e1 .. e1 + 3, the halves of four pairs where they lie
  // half a rotation apart and the lane is one that turns
  const bool turned = c8 * kVec < p.rot;
  const bool halves = turned && !INTERLEAVED;
  const int e0 = halves ? 4 * c8 : kVec * c8, gap = halves ? p.rot / 2 : 4;   // e1 = e0 + gap
  // rows of q, k, v in a line, row r at its base + r * D values
  const uint8_t *from_q = static_cast<const uint8_t *>(p.q) + (first_t * p.q_stride + e0) * EB;
  const uint8_t *from_k = static_cast<const uint8_t *>(p.k) + (first_t * p.k_stride + e0 - hq * D) * EB;
  const uint8_t *from_v = static_cast<const uint8_t *>(p.v) + (first_t * p.v_stride + e0 - (hq + hkv) * D) * EB;
  Quad<IN> lo[AHEAD], hi[AHEAD];
  const auto load = [&](int r0) {
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) {
      const int r = r0 + s * RPI + r_mine;
      if (r >= rows) continue;
      const uint8_t *at = (r < hq ? from_q : r < hq + hkv ? from_k : from_v) + r * (D * EB);
      lo[s] = *reinterpret_cast<const Quad<IN> *>(at);
      hi[s] = *reinterpret_cast<const Quad<IN> *>(at + gap * EB);
    }
  };
  load(0);
  const int pairs = p.rot / 2;
  for (int i = tid; i < tokens * pairs; i += kRopeThreads) {
    const int k = i / pairs, f = i - k * pairs;
    constexpr double kInvTurn = 0.15915494309189533577;  // 1 / (2 pi)
    const double turns = static_cast<double>(p.rope_pos[first_t + k]) * p.inv_freq[f] * kInvTurn;
    const double quarters = rint(4. * turns);
    const float r = static_cast<float>(turns - 0.25 * quarters);
    float s, c;
    sincospif(2.f * r, &s, &c);
    // turned back by the quarters
    const int n = static_cast<int>(static_cast<long long>(quarters) & 3);
    cosines[k][f] = n == 0 ? c : n == 1 ? -s : n == 2 ? -c : s;
    sines[k][f] = n == 0 ? s : n == 1 ? c : n == 2 ? -s : -c;
  }
  if (tid >= kRopeThreads - tokens) {   // (the last threads have no sine of one token to compute)
    const int k = kRopeThreads - 1 - tid;
    const int b = p.seq_ids[first_t + k], j = p.token_ids[first_t + k];
    int fmt = -1;
    long long slot = 0;
    if (b >= 0 && j >= 0) {
      if (b >= p.c.batch || j >= static_cast<long long>(p.c.max_pages) * p.c.P)
        set_err(p.c.err, CFR_DEVERR_SEQ_LEN);
      else if (!resolve_page(p.c, b, j / p.c.P, kHotFormats, fmt, slot))
        fmt = -1;
    }
    place[k][0] = fmt;
    place[k][1] = slot * hkv * p.c.P + (j >= 0 ? j % p.c.P : 0);
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < tokens; ++k) {
    if (k > 0) {
      from_q += p.q_stride * EB;
      from_k += p.k_stride * EB;
      from_v += p.v_stride * EB;
      load(0);
    }
    const int fmt = static_cast<int>(place[k][0]);
    float cs[4], sn[4];
    if (turned) {
      // pairs 4 c8 .. 4 c8 + 3, either way
      const float4 c4 = reinterpret_cast<const float4 *>(cosines[k])[c8], s4 = reinterpret_cast<const float4 *>(sines[k])[c8];
      cs[0] = c4.x, cs[1] = c4.y, cs[2] = c4.z, cs[3] = c4.w;
      sn[0] = s4.x, sn[1] = s4.y, sn[2] = s4.z, sn[3] = s4.w;
    }
    // where rows go, the same way: head h of K or V is P rows behind head h - 1 in its page
    const int eb_page = fmt == CFR_FMT_F32 ? 4 : 2;
    const long long head_bytes = static_cast<long long>(p.c.P) * D * eb_page;
    uint8_t *const to_q = static_cast<uint8_t *>(p.q_out) + ((first_t + k) * hq * D + e0) * EB;
    uint8_t *to_k = nullptr, *to_v = nullptr;
    if (fmt >= 0) {
      const long long first = (place[k][1] * D + e0) * eb_page;
      to_k = p.c.k_pool[fmt] + first - hq * head_bytes;
      to_v = p.c.v_pool[fmt] + first - (hq + hkv) * head_bytes;
    }
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += AHEAD * RPI) {     // every lane of a warp takes every step
      if (r0 > 0) load(r0);
#pragma unroll
      for (int s = 0; s < AHEAD; ++s) {
        if (r0 + s * RPI >= rows) break;
        const int r = r0 + s * RPI + r_mine;
        const bool is_q = r < hq, is_v = r >= hq + hkv;
        float x[kVec] = {};
        if (r < rows) {
          unpack4(lo[s], x);
          unpack4(hi[s], x + 4);
        }
        if (p.q_weight || p.k_weight) {
          float2 sq = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < kVec; i += 2) sq = fma2(make_float2(x[i], x[i + 1]), make_float2(x[i], x[i + 1]), sq);
          float sum = sq.x + sq.y;
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          const float *w = is_v ? nullptr : is_q ? p.q_weight : p.k_weight;
          if (w) {
            const float rs = rsqrtf(sum * (1.f / D) + p.eps);
            const float4 w0 = *reinterpret_cast<const float4 *>(w + e0), w1 = *reinterpret_cast<const float4 *>(w + e0 + gap);
            const float wv[kVec] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int i = 0; i < kVec; i += 2) {
              const float2 y = mul2(mul2(make_float2(x[i], x[i + 1]), make_float2(rs, rs)), make_float2(wv[i], wv[i + 1]));
              x[i] = y.x;
              x[i + 1] = y.y;
            }
          }
        }
        if (turned && !is_v) {
          if constexpr (INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = x[2 * i], b = x[2 * i + 1];
              x[2 * i] = a * cs[i] - b * sn[i];
              x[2 * i + 1] = b * cs[i] + a * sn[i];
            }
          } else {
            // two pairs an instruction
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              const float2 a = make_float2(x[i], x[i + 1]), b = make_float2(x[i + 4], x[i + 5]);
              const float2 c2 = make_float2(cs[i], cs[i + 1]), s2 = make_float2(sn[i], sn[i + 1]);
              const float2 y = fma2(a, c2, mul2(b, make_float2(-s2.x, -s2.y))), z = fma2(b, c2, mul2(a, s2));
              x[i] = y.x;
              x[i + 1] = y.y;
              x[i + 4] = z.x;
              x[i + 5] = z.y;
            }
          }
        }
        if (r >= rows) continue;
        if (is_q) {
          uint8_t *at = to_q + r * (D * EB);
          put4(IN, at, 0, x);
          put4(IN, at, gap, x + 4);
        } else if (fmt >= 0) {
          uint8_t *at = (is_v ? to_v : to_k) + r * head_bytes;
          put4(fmt, at, 0, x);
          put4(fmt, at, gap, x + 4);
        }
      }
    }
  }
}

template <int IN, bool INTERLEAVED>
void launch_rope(const RopeParams &p, cudaStream_t s) {
  const int tokens = (p.num_tokens + p.per - 1) / p.per;
  if (p.c.D == 128)
    rope_kernel<IN, 128, INTERLEAVED><<<tokens, kRopeThreads, 0, s>>>(p);
  else
    rope_kernel<IN, 64, INTERLEAVED><<<tokens, kRopeThreads, 0, s>>>(p);
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
  p.num_tokens = num_tokens;
  // several tokens a CTA once that leaves every SM a CTA or two (17K tokens: 108 us with one, 95 with four; 1.5K fp32
  // tokens 15.6 and 14.3); a short step's few tokens get a CTA each
  p.per = num_tokens >= 1024 ? kRopeTokens : 1;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (in_fmt == CFR_FMT_F32)
    interleaved ? launch_rope<CFR_FMT_F32, true>(p, s) : launch_rope<CFR_FMT_F32, false>(p, s);
  else
    interleaved ? launch_rope<CFR_FMT_BF16, true>(p, s) : launch_rope<CFR_FMT_BF16, false>(p, s);
  return cudaGetLastError() == cudaSuccess ? CFR_OK : CFR_ERR_CUDA;
}

}  // extern "C"
