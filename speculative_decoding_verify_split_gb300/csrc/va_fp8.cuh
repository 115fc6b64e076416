// e4m3 helpers of the FP8 tensor-core paths: packing, and the softmax weights as
// two e4m3 terms with block scales.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "va_split.cuh"

namespace va {

__device__ __forceinline__ uint32_t pack_fp8x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float2 unpack_fp8x2(uint32_t v) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)v, __NV_E4M3);
  return __half22float2(__half2(h));
}

// The weights of a block of 32 keys of one row as the tensor cores take them:
// p = 2^(s - e), with e the block's own exponent, so that the block's largest
// lies in [2^7, 2^8), as two e4m3 terms: hi = e4m3(p), lo = e4m3(32 (p - hi))
// (the remainder of a p below 2^8 is at most 8, so 32 times it stays under
// 448). The MMA's block scales bring them to the row's reference: 2^(e - m_ref)
// and 2^(e - m_ref - 5); m_ref is a whole number, so p does not depend on it. p
// keeps 8 bits down to 2^-7, 15 powers of two below the block's largest, and
// is rounded in steps of 2^-14 from there: what is lost of a row is at most 32
// keys' 2^-22 of the largest weight beside them, whatever the row's other
// blocks hold.
constexpr int kBlockTop = 7;  // floor(log2) of a block's largest p
constexpr int kLoShift = 5;   // the low terms' scale is 2^-kLoShift of the high terms'

// The exponent e of a block whose largest weight is 2^d, a whole number (finite
// for d = -inf or NaN, a block without weights), not below kMinScale of the
// reference: below that p falls under 2^7, down to 0 in O for weights under
// 2^-137 of 2^m_ref.
constexpr float kMinScale = -122.f;
__device__ __forceinline__ float block_exponent(float d, float m_ref) {
  return fmaxf(fmaxf(floorf(d), -1e30f) - (float)kBlockTop, m_ref + kMinScale);
}
// log2 of the block's scale: in [kMinScale, 100], so that the low terms' byte is
// at least 0 (m_ref = -inf: no visible key, p = 0).
__device__ __forceinline__ float block_scale(float e, float m_ref) { return fminf(e - m_ref, 100.f); }
__device__ __forceinline__ uint32_t scale_byte(float x) { return (uint32_t)((int)x + 127); }
__device__ __forceinline__ float exp2_int(float x) { return __uint_as_float(scale_byte(x) << 23); }
static_assert(kMinScale + 127 - kLoShift >= 0, "scale bytes");

// p (two fp32 values, a first) -> e4m3 hi and scaled lo bytes, via f16x2.
__device__ __forceinline__ void split_weights(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const __nv_fp8x2_storage_t h8 = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(h), __NV_SATFINITE, __NV_E4M3);
  const __half2 hh = __half2(__nv_cvt_fp8x2_to_halfraw2(h8, __NV_E4M3));
  const __half2 r = __hmul2(__hsub2(h, hh), __float2half2_rn((float)(1 << kLoShift)));
  const __nv_fp8x2_storage_t l8 = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(r), __NV_SATFINITE, __NV_E4M3);
  hi = (uint32_t)h8;
  lo = (uint32_t)l8;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  return (uint32_t)float_to_bf16_bits(lo) | ((uint32_t)float_to_bf16_bits(hi) << 16);
}

}  // namespace va
