// pagedkv_requant.cuh -- device helpers of the kernels that set the scales of
// 8-bit pools: the values of codes, a block's scale and the codes under it.
// A code c under scale s stands for the fp32 product c * s; a block's scale is
// the largest finite magnitude of its rows divided by the largest code value
// (127 or 448), in fp32; the code of x is the nearest to the fp32 quotient
// x / scale, ties to even (dev::quantize, dev::quantize_e4m3).
#pragma once

#include "pagedkv_device.cuh"

namespace pagedkv {
namespace dev {

template <bool kFp8>
constexpr float kCodeMax = kFp8 ? 448.0f : 127.0f;

constexpr float kLargestFinite = 3.402823466e38f;

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// |x| when finite, else 0 (an infinity or NaN never sets a scale).
__device__ __forceinline__ float finite_abs(float x) {
  const float m = fabsf(x);
  return m <= kLargestFinite ? m : 0.0f;
}

// The scale of a block whose largest finite magnitude is amax (0: all zero).
template <bool kFp8>
__device__ __forceinline__ float block_scale(float amax) {
  return __fdiv_rn(amax, kCodeMax<kFp8>);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The four code values of a 32-bit word, lowest byte first.  int8: each byte
// is placed under the exponent of 2^23, c + 128 + 2^23, and 2^23 + 128 taken
// off (exact; an integer conversion runs at an eighth of the add's rate).
template <bool kFp8>
__device__ __forceinline__ void code_values(uint32_t w, float (&v)[4]) {
  if constexpr (kFp8) {
    const uint32_t lo = codes_to_f16x2<true>(w, 0x4140u), hi = codes_to_f16x2<true>(w, 0x4342u);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
  } else {
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __uint_as_float(prmt(u, 0x4b000000u, 0x7440u + i)) - 8388736.0f;
  }
}

// Largest magnitude among 16 codes, as a code value (NaN codes passed over).
template <bool kFp8>
__device__ __forceinline__ float largest_code(uint4 x) {
  const uint32_t w[4] = {x.x ^ kCodeBias<kFp8>, x.y ^ kCodeBias<kFp8>, x.z ^ kCodeBias<kFp8>,
                         x.w ^ kCodeBias<kFp8>};
  __half2 m = __float2half2_rn(0.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = codes_to_f16x2<kFp8>(w[i], 0x4140u), hi = codes_to_f16x2<kFp8>(w[i], 0x4342u);
    m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&lo)));
    m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&hi)));
  }
  return fmaxf(__low2float(m), __high2float(m));
}

// Largest finite |c * s| of 16 codes, one by one (an overflowing or NaN scale).
template <bool kFp8>
__device__ __noinline__ float codes_amax_each(uint4 x, float s) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float m = 0.0f;
  for (int i = 0; i < 4; ++i) {
    float v[4];
    code_values<kFp8>(w[i], v);
    for (int k = 0; k < 4; ++k) m = fmaxf(m, finite_abs(__fmul_rn(v[k], s)));
  }
  return m;
}

// Codes without a division per element.  The code of the fp32 quotient q =
// x / s is wanted; q lies within a relative 2^-22 of x * r for the rounded
// r = 1 / s (or, for x = c * t under an old scale t, of c * (t r)), so between
// x * lo and x * hi with lo, hi = r (1 -+ 2^-21).  The code grows with the
// value: where both ends have the same code it is q's, and only the words
// where they differ (a border between two codes lies in between) are divided.
// An IEEE division per element bound these kernels at 21 % of the memory rate.
// s == 0 reads as 1; scales outside [2^-80, 2^80], whose products or
// remainders could lose bits, always divide, and so do ratios of two scales
// above 2^80: t r may be infinite, and 0 * infinity is no code.  (Any smaller
// ratio will do: below 2^-19 every product has the code 0, as its quotient.)
struct Interval {
  float lo, hi;
  bool on;
  float s, r;                                        // the scale (0 as 1), its reciprocal
};

__device__ __forceinline__ bool plain_size(float s) { return s >= 0x1p-80f && s <= 0x1p80f; }

__device__ __forceinline__ Interval interval(float factor, bool on, float s, float r) {
  return {factor * (1.0f - 0x1p-21f), factor * (1.0f + 0x1p-21f), on, s, r};
}

__device__ __forceinline__ float scale_or_one(float s) { return s == 0.0f ? 1.0f : s; }

// Interval of x / s for finite x with |x / s| at most the largest code.
__device__ __forceinline__ Interval quotients(float s) {
  s = scale_or_one(s);
  const float r = __frcp_rn(s);
  return interval(r, plain_size(s), s, r);
}
// Interval of (c * t) / s for codes c.
__device__ __forceinline__ Interval quotients(float t, float s) {
  s = scale_or_one(s);
  const float r = __frcp_rn(s);
  const float f = t * r;
  return interval(f, plain_size(s) && plain_size(t) && f <= 0x1p80f, s, r);
}

// The codes of x[k] * f, lowest byte first (int8: |x[k] * f| < 128).
template <bool kFp8>
__device__ __forceinline__ uint32_t code4_times(const float (&x)[4], float f) {
  if constexpr (kFp8) {
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1] * f), "f"(x[0] * f));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3] * f), "f"(x[2] * f));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  } else {
    // x f + 1.5 2^23, rounded once, holds the nearest integer in its low bits
    uint32_t t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = __float_as_uint(fmaf(x[k], f, 12582912.0f));
    return prmt(prmt(t[0], t[1], 0x0040u), prmt(t[2], t[3], 0x0040u), 0x5410u);
  }
}

// The bf16 values of two words.
__device__ __forceinline__ void bf16_values(uint32_t w0, uint32_t w1, float (&v)[4]) {
  v[0] = __uint_as_float(w0 << 16);
  v[1] = __uint_as_float(w0 & 0xffff0000u);
  v[2] = __uint_as_float(w1 << 16);
  v[3] = __uint_as_float(w1 & 0xffff0000u);
}

// The codes of four values by division.
template <bool kFp8>
__device__ __forceinline__ uint32_t code4_divided(const float (&x)[4], float s) {
  uint32_t o = 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) o |= (uint32_t)code8<kFp8>(x[k], s) << (8 * k);
  return o;
}

// 16 codes at both ends of an interval of factors: those of the lower end into
// `o`, and where they differ from the upper end's into `off` (the codes
// between are then not known).  One test per 16, so that the conversions of
// all four words run together.
template <bool kFp8>
__device__ __forceinline__ bool recode16_between(uint4 x, float lo, float hi, uint4& o, uint4& off) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4], d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[4];
    code_values<kFp8>(w[i], v);
    c[i] = code4_times<kFp8>(v, lo);
    d[i] = c[i] ^ code4_times<kFp8>(v, hi);
  }
  o = make_uint4(c[0], c[1], c[2], c[3]);
  off = make_uint4(d[0], d[1], d[2], d[3]);
  return (d[0] | d[1] | d[2] | d[3]) != 0u;
}

// `o` with the words marked in `off` (all of them with `every`) made by
// division: the codes of (code * t) / s.  Out of line: rare, and its code,
// repeated in every unrolled piece, would not fit the instruction cache.
template <bool kFp8>
__device__ __noinline__ uint4 divide_words(uint4 x, uint4 o, uint4 off, float t, float s, bool every) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w}, d[4] = {off.x, off.y, off.z, off.w};
  uint32_t r[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!every && d[i] == 0u) continue;
    float v[4];
    code_values<kFp8>(w[i], v);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __fmul_rn(v[k], t);
    r[i] = code4_divided<kFp8>(v, s);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// 16 codes under scale t as codes under scale s, with q = quotients(t, s).
// (A code -128, which this library never writes, may round to -128 again
// where the definition clamps to -127: such pieces divide.)
template <bool kFp8>
__device__ __forceinline__ uint4 recode16(uint4 x, const Interval& q, float t, float s) {
  const bool on = q.on && (kFp8 || largest_code<false>(x) <= 127.0f);
  uint4 o, off;
  return recode16_between<kFp8>(x, q.lo, q.hi, o, off) || !on ? divide_words<kFp8>(x, o, off, t, s, !on) : o;
}

// 16 bf16 values' codes under scale s by division.
template <bool kFp8>
__device__ __noinline__ uint4 code16_divided(uint4 a, uint4 b, float s) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[4];
    bf16_values(w[2 * i], w[2 * i + 1], v);
    o[i] = code4_divided<kFp8>(v, s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// 16 finite bf16 values under scale s, with q = quotients(s).  int8 goes by
// the interval as above.  For E4M3 a border is often met: both the values and
// the block's largest (448 s) have 8 significant bits, so x / s falls next to
// a midpoint of two codes in 0.5 % of N(0, 1) values and 43 % of warps had to
// divide.  There the quotient itself is made, by two of Markstein's correction
// steps (P. Markstein, IBM J. Res. Dev. 34, 1990) with r the correctly rounded
// reciprocal: q0 = x r is within 2 units in the last place, the first step
// brings it within one, from where the second rounds correctly.  The remainder
// is taken as y s - x, which is +0 for either zero: y - (+0) r then keeps the
// sign of a -0 (y + (+0) r, with the remainder x - y s, would lose it).
template <bool kFp8>
__device__ __forceinline__ uint4 code16(uint4 a, uint4 b, const Interval& q, float s) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t o[4], off = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[4];
    bf16_values(w[2 * i], w[2 * i + 1], v);
    if constexpr (kFp8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float y = v[k] * q.r;
        y = fmaf(fmaf(y, q.s, -v[k]), -q.r, y);
        v[k] = fmaf(fmaf(y, q.s, -v[k]), -q.r, y);
      }
      o[i] = code4_times<true>(v, 1.0f);
    } else {
      o[i] = code4_times<false>(v, q.lo);
      off |= o[i] ^ code4_times<false>(v, q.hi);
    }
  }
  if (q.on && off == 0u) return make_uint4(o[0], o[1], o[2], o[3]);
  return code16_divided<kFp8>(a, b, s);
}

}  // namespace dev
}  // namespace pagedkv
