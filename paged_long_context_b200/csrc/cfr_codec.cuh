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
    // (integer conversions run at an eighth of the rate of these: 2^23 + code + 128, exact, less 2^23 + 128)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t u = (k < 4 ? r.w.x : r.w.y) ^ 0x80808080u;
      x[k] = __fmul_rn(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540u | (k & 3))) - 8388736.f, scale);
    }
  } else if constexpr (SRC == CFR_FMT_FP8) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const uint32_t h = e4m3x2_to_h2(k < 4 ? r.w.x : r.w.y, (k & 3) >> 1);
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
      x[k] = __fmul_rn(f.x, scale);
      x[k + 1] = __fmul_rn(f.y, scale);
    }
  } else {  // CFR_FMT_I4: 2^23 + code + 8 less 2^23 + 8
    const uint32_t u = r.w ^ 0x88888888u, lo = u & 0x0F0F0F0Fu, hi = (u >> 4) & 0x0F0F0F0Fu;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      x[k] = __fmul_rn(__uint_as_float(__byte_perm(k & 1 ? hi : lo, 0x4B000000u, 0x7540u | (k >> 1))) - 8388616.f, scale);
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

// ---------------------------------------------------------------------------
// Codes without a division per element.
//
// The codes are the ones defined above, code = rint(fl(x / scale)) (or the
// E4M3 code of fl(x / scale)), reached without a division per element.  Let q = x / scale (exact) and f = fl(q).
// With a normal, finite scale and r = fl(1 / scale) (one correctly rounded
// reciprocal per block), take r- = fl(r * (1 - 2^-20)) and r+ = fl(r * (1 + 2^-20)).
// Each of r, r-, r+ and f carries a relative rounding error of at most 2^-24,
// so x*r- and x*r+ (exact products) lie on either side of f:
//   |x*r-| <= |q| (1 - 2^-20 + 2^-23) < |f|,   |x*r+| >= |q| (1 + 2^-20 - 2^-23) > |f|
// (for tiny |q| all three round to 0).  One fused multiply-add of each into
// the magic constant 1.5 * 2^23, whose unit in the last place is 1, rounds
// the exact product to the nearest integer (ties to even) and leaves it in
// the low bits of the sum.  Rounding to nearest is monotone, so when both
// sums agree they equal rint(f): that is the code, and |code| <= Q (the clamp
// cannot bind: |x| <= max|x| and scale >= max|x| / Q to within 2^-24).  When
// they differ (a half-integer within about |q| * 2^-20 of the product, and
// every NaN), the eight elements of the vector are encoded again with the
// IEEE division.  On bf16 blocks of N(0,1) values that is about one element in
// 600: a value that is a simple fraction of max|x| (max|x| / 2, say) puts
// x / scale within an ulp of a half-integer.  E4M3 destinations
// round the two products to fp32 and then to E4M3, both monotone, so equal
// codes of the two are the code of f.  A block whose maximum is infinite or
// whose scale is zero or subnormal (where the bounds above fail) is encoded
// with the division throughout.
// ---------------------------------------------------------------------------

constexpr float kRintMagic = 12582912.0f;         // 1.5 * 2^23
constexpr uint32_t kRintMagicBits = 0x4B400000u;  // its bit pattern

// Running max|x| of bf16 pairs: per half, max(|m|, |w|) (its sign bit left
// arbitrary).  The bf16 max returns the other operand when one is NaN, as
// fmaxf does.
__device__ __forceinline__ uint32_t absmax_acc(uint32_t m, uint32_t w) {
  uint32_t d;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(w));
  return d;
}

__device__ __forceinline__ float absmax_value(uint32_t m) {
  return fmaxf(bf16_lo(m & 0x7FFF7FFFu), bf16_hi(m & 0x7FFF7FFFu));
}

// stores eight codes (the low byte, or for int4 the low nibble, of each tb)
// as vector v of the block
template <int DST>
__device__ __forceinline__ void store_codes8(uint8_t *dst, int v, const uint32_t (&tb)[kVec]) {
  if constexpr (DST == CFR_FMT_I4) {  // element 2i in the low nibble of byte i
    uint32_t n[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) n[k] = (tb[2 * k] & 0x0Fu) | (tb[2 * k + 1] << 4);
    reinterpret_cast<uint32_t *>(dst)[v] =
        __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
  } else {  // int8 and E4M3: one byte each
    const uint32_t lo = __byte_perm(__byte_perm(tb[0], tb[1], 0x0040), __byte_perm(tb[2], tb[3], 0x0040), 0x5410);
    const uint32_t hi = __byte_perm(__byte_perm(tb[4], tb[5], 0x0040), __byte_perm(tb[6], tb[7], 0x0040), 0x5410);
    reinterpret_cast<uint2 *>(dst)[v] = make_uint2(lo, hi);
  }
}

// The eight codes of one vector of decoded values x, from the two bracketing
// products x * r_lo and x * r_hi; true when they disagree somewhere (or a
// value is NaN), and the vector must be encoded again with the division.
//  - int8 / int4: each as 0x4B400000 + code (the rounded sum with 1.5 * 2^23);
//  - E4M3: the code of each rounded product (rounding to fp32 and then to E4M3
//    are both monotone, so equal codes of the two products are the code of
//    fl(x / scale), which lies between them).
template <int DST>
__device__ __forceinline__ bool codes8_fast(const float (&x)[kVec], float r_lo, float r_hi,
                                            uint32_t (&tb)[kVec]) {
  bool near = false;
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    if constexpr (DST == CFR_FMT_FP8) {
      const uint32_t lo = __nv_cvt_float_to_fp8(__fmul_rn(x[k], r_lo), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float_to_fp8(__fmul_rn(x[k], r_hi), __NV_SATFINITE, __NV_E4M3);
      near |= (lo != hi) || (x[k] != x[k]);
      tb[k] = lo;
    } else {
      const float lo = __fmaf_rn(x[k], r_lo, kRintMagic);
      const float hi = __fmaf_rn(x[k], r_hi, kRintMagic);
      near |= lo != hi;
      tb[k] = __float_as_uint(lo);
    }
  }
  return near;
}

// the same codes with the IEEE division
template <int DST>
__device__ __forceinline__ void codes8_exact(const float (&x)[kVec], float scale, uint32_t (&tb)[kVec]) {
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    if constexpr (DST == CFR_FMT_FP8)
      tb[k] = fp8_code(x[k], scale);
    else
      tb[k] = kRintMagicBits + static_cast<uint32_t>(int_code(x[k], scale, DST == CFR_FMT_I8 ? 127 : 7));
  }
}

// The same codes from the quotients themselves, correctly rounded without a division: with r = fl(1 / scale),
//   q0 = fl(x r),  q1 = fl(q0 + r fl(x - q0 scale)),  f = fl(q1 + r (x - q1 scale)).
// q0 is within 1.5 ulp of x / scale and q1 within one, so the second remainder is exact (a
// multiple of ulp(q1) ulp(scale), below 2^24 of them) and f = fl(x / scale) (P. Markstein's theorem, for r
// correctly rounded).  No remainder that matters underflows while scale >= 2^-64 (a quotient below 2^-11 has
// code 0 in every format, however its last bits fall) and r is a normal number up to 2^64.
constexpr float kQuotientMin = 0x1p-64f, kQuotientMax = 0x1p64f;

__device__ __forceinline__ float2 quotients(float2 x, float2 r, float2 minus_scale) {
  const float2 q0 = mul2(x, r), q1 = fma2(fma2(q0, minus_scale, x), r, q0);
  return fma2(fma2(q1, minus_scale, x), r, q1);
}
__device__ __forceinline__ float with_sign(float f, float x) {   // (-0 comes out of the sums as +0)
  return __uint_as_float((__float_as_uint(f) & 0x7FFFFFFFu) | (__float_as_uint(x) & 0x80000000u));
}

// Stores the codes of eight values as vector v of the block.  Quotients below -Q, which only codes that no encoder writes
// lead to (-128, -8), are clamped where CLAMP says so.  Returns false, and what it stored is to be stored again,
// where an integer format meets a NaN.
template <int DST, bool CLAMP>
__device__ __forceinline__ bool store_quotients8(uint8_t *dst, int v, const float (&x)[kVec], float r, float scale) {
  const auto clamp = [](float2 q) {
    constexpr float least = DST == CFR_FMT_I8 ? -127.f : -7.f;
    return CLAMP ? make_float2(q.x < least ? least : q.x, q.y < least ? least : q.y) : q;
  };
  const float2 rr = make_float2(r, r), ms = make_float2(-scale, -scale);
  if constexpr (DST == CFR_FMT_FP8) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 q = quotients(make_float2(x[2 * k], x[2 * k + 1]), rr, ms);
      q.x = with_sign(q.x, x[2 * k]);
      q.y = with_sign(q.y, x[2 * k + 1]);
      w[k] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
    }
    reinterpret_cast<uint2 *>(dst)[v] = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    return true;
  } else if constexpr (DST == CFR_FMT_I4) {
    // of two elements, one sum: 1.5 * 2^23 + (c0 + 8) + 16 (c1 + 8), whose low byte with its signs
    // put back is the byte of both
    const float2 one = make_float2(kRintMagic, kRintMagic), both = make_float2(kRintMagic + 136.f, kRintMagic + 136.f);
    const float2 sixteen = make_float2(16.f, 16.f), minus = make_float2(-kRintMagic, -kRintMagic);
    uint32_t t[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {   // bytes 2 k and 2 k + 1
      const float2 e = add2(clamp(quotients(make_float2(x[4 * k], x[4 * k + 2]), rr, ms)), both);
      const float2 o = add2(add2(clamp(quotients(make_float2(x[4 * k + 1], x[4 * k + 3]), rr, ms)), one), minus);
      const float2 y = fma2(o, sixteen, e);
      t[2 * k] = __float_as_uint(y.x);
      t[2 * k + 1] = __float_as_uint(y.y);
    }
    reinterpret_cast<uint32_t *>(dst)[v] =
        __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410) ^ 0x88888888u;
    return !((t[0] | t[1] | t[2] | t[3]) & 0x30000000u);   // (of 0x4B4000xx or a NaN's 0x7FFFFFFF)
  } else {
    const float2 one = make_float2(kRintMagic, kRintMagic);
    uint32_t tb[kVec], any = 0u;
#pragma unroll
    for (int k = 0; k < kVec; k += 2) {
      const float2 q = add2(clamp(quotients(make_float2(x[k], x[k + 1]), rr, ms)), one);
      tb[k] = __float_as_uint(q.x);
      tb[k + 1] = __float_as_uint(q.y);
      any |= tb[k] | tb[k + 1];
    }
    store_codes8<DST>(dst, v, tb);
    return !(any & 0x30000000u);
  }
}

}  // namespace cfr
