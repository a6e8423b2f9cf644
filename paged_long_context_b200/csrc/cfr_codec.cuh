// cfr_codec.cuh -- vectors of eight stored elements: reading them as fp32 values
// and encoding fp32 values into a storage format (demotion, cache writes and
// read-back share these, so the codes are the same whichever path stored them).
#pragma once

#include <cuda_bf16.h>

#include "cfr_common.cuh"

namespace cfr {

constexpr int kVec = 8;  // elements per vector access

// Raw stored bytes of kVec consecutive elements of a source format, loaded with
// one or two vector accesses and decoded later (so that every load of a thread
// is in flight before the first one is used).
template <int SRC>
struct RawVec {
  uint2 w;  // CFR_FMT_I8 and CFR_FMT_FP8: 8 one-byte codes
};
template <>
struct RawVec<CFR_FMT_F32> {
  uint4 a, b;
};
template <>
struct RawVec<CFR_FMT_BF16> {
  uint4 a;
};
template <>
struct RawVec<CFR_FMT_I4> {
  uint32_t w;
};

template <int SRC>
__device__ __forceinline__ RawVec<SRC> load_raw(const uint8_t *blk, long long v) {
  RawVec<SRC> r;
  if constexpr (SRC == CFR_FMT_F32) {
    const uint4 *p = reinterpret_cast<const uint4 *>(blk + 32 * v);
    r.a = p[0];
    r.b = p[1];
  } else if constexpr (SRC == CFR_FMT_BF16) {
    r.a = *reinterpret_cast<const uint4 *>(blk + 16 * v);
  } else if constexpr (SRC == CFR_FMT_I4) {
    r.w = *reinterpret_cast<const uint32_t *>(blk + 4 * v);
  } else {
    r.w = *reinterpret_cast<const uint2 *>(blk + 8 * v);
  }
  return r;
}

// the eight values of a raw vector as fp32 (quantised: code * scale, fp32 product)
template <int SRC>
__device__ __forceinline__ void decode_raw(const RawVec<SRC> &r, float scale, float (&x)[kVec]) {
  if constexpr (SRC == CFR_FMT_F32) {
    const uint32_t a[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(a[k]);
  } else if constexpr (SRC == CFR_FMT_BF16) {
    const uint32_t a[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = bf16_lo(a[k]);
      x[2 * k + 1] = bf16_hi(a[k]);
    }
  } else if constexpr (SRC == CFR_FMT_I8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = __fmul_rn(i8_at(k < 4 ? r.w.x : r.w.y, k & 3), scale);
  } else if constexpr (SRC == CFR_FMT_FP8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = __fmul_rn(e4m3_at(k < 4 ? r.w.x : r.w.y, k & 3), scale);
  } else {  // CFR_FMT_I4
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = __fmul_rn(i4_at(r.w, k), scale);
  }
}

__device__ __forceinline__ int int_code(float x, float scale, int q) {
  if (!(scale > 0.f)) return 0;
  const int c = __float2int_rn(__fdiv_rn(x, scale));  // NaN -> 0
  return min(max(c, -q), q);
}

__device__ __forceinline__ uint32_t fp8_code(float x, float scale) {
  if (!(scale > 0.f)) return 0u;
  const float q = __fdiv_rn(x, scale);
  if (q != q) return 0x7Fu;  // NaN: the positive E4M3 NaN code
  return static_cast<uint32_t>(__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3));
}

// encodes eight values and stores them at element e of the destination block
__device__ __forceinline__ void store8(int fmt, uint8_t *blk, long long e, float scale,
                                       const float (&x)[kVec]) {
  if (fmt == CFR_FMT_F32) {
    float4 *p = reinterpret_cast<float4 *>(blk + 4 * e);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else if (fmt == CFR_FMT_BF16) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = __bfloat16_as_ushort(__float2bfloat16_rn(x[2 * k]));
      const uint32_t hi = __bfloat16_as_ushort(__float2bfloat16_rn(x[2 * k + 1]));
      w[k] = lo | (hi << 16);
    }
    *reinterpret_cast<uint4 *>(blk + 2 * e) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if (fmt == CFR_FMT_I8) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k)
      w[k >> 2] |= (static_cast<uint32_t>(int_code(x[k], scale, 127)) & 0xFFu) << (8 * (k & 3));
    *reinterpret_cast<uint2 *>(blk + e) = make_uint2(w[0], w[1]);
  } else if (fmt == CFR_FMT_FP8) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k >> 2] |= fp8_code(x[k], scale) << (8 * (k & 3));
    *reinterpret_cast<uint2 *>(blk + e) = make_uint2(w[0], w[1]);
  } else {  // CFR_FMT_I4: element 2i in the low nibble of byte i
    uint32_t w = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) w |= (static_cast<uint32_t>(int_code(x[k], scale, 7)) & 0xFu) << (4 * k);
    *reinterpret_cast<uint32_t *>(blk + e / 2) = w;
  }
}

__device__ __forceinline__ void store_zero8(int fmt, uint8_t *blk, long long e) {
  if (fmt == CFR_FMT_F32) {
    float4 *p = reinterpret_cast<float4 *>(blk + 4 * e);
    p[0] = make_float4(0.f, 0.f, 0.f, 0.f);
    p[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  } else if (fmt == CFR_FMT_BF16) {
    *reinterpret_cast<uint4 *>(blk + 2 * e) = make_uint4(0u, 0u, 0u, 0u);
  } else if (fmt == CFR_FMT_I4) {
    *reinterpret_cast<uint32_t *>(blk + e / 2) = 0u;
  } else {
    *reinterpret_cast<uint2 *>(blk + e) = make_uint2(0u, 0u);
  }
}

__device__ __forceinline__ float qmax_of(int fmt) {
  return fmt == CFR_FMT_I8 ? 127.f : fmt == CFR_FMT_I4 ? 7.f : 448.f;
}

}  // namespace cfr
