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

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// |x| when finite, else 0 (an infinity or NaN never sets a scale).
__device__ __forceinline__ float finite_abs(float x) {
  const float m = fabsf(x);
  return m <= 3.402823466e38f ? m : 0.0f;
}

// The scale of a block whose largest finite magnitude is amax (0: all zero).
template <bool kFp8>
__device__ __forceinline__ float block_scale(float amax) {
  return __fdiv_rn(amax, kCodeMax<kFp8>);
}

// The four code values of a 32-bit word, lowest byte first.
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
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(w >> (8 * i));
  }
}

// Largest finite |c * s| of 16 codes.
template <bool kFp8>
__device__ __forceinline__ float codes_amax(uint4 x, float s) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[4];
    code_values<kFp8>(w[i], v);
#pragma unroll
    for (int k = 0; k < 4; ++k) m = fmaxf(m, finite_abs(__fmul_rn(v[k], s)));
  }
  return m;
}

// The codes of four values under scale s, lowest byte first.
template <bool kFp8>
__device__ __forceinline__ uint32_t code4(const float (&x)[4], float s) {
  uint32_t o = 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) o |= (uint32_t)code8<kFp8>(x[k], s) << (8 * k);
  return o;
}

// 16 codes under scale s as codes under scale ns.
template <bool kFp8>
__device__ __forceinline__ uint4 recode16(uint4 x, float s, float ns) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[4];
    code_values<kFp8>(w[i], v);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __fmul_rn(v[k], s);
    w[i] = code4<kFp8>(v, ns);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace dev
}  // namespace pagedkv
