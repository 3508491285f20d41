// Activations in 8 bits: e4m3 codes with one power-of-two scale per row and
// 32 consecutive columns.
//
// For a block of values x_0 .. x_31 with amax = max |x_j| over its finite
// ones, k is the smallest exponent in [-120, 120] with amax <= 448 * 2^k, the
// block's scale byte is k + 127, and code j is x_j * 2^-k rounded to e4m3 (to
// nearest, ties to even; 448 is e4m3's largest value, so none saturates).  A
// code stands for e4m3 * 2^k, which fp32 and bf16 both hold exactly (k >=
// -120 keeps e4m3's smallest step, 2^-9, above bf16's 2^-133): the relative
// error of a value in e4m3's normal range is at most 2^-4, that of a smaller
// one at most 2^-10 * 2^k.  Infinities and NaN become NaN.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"

namespace mlpk {

constexpr int kQ8Block = 32;   // columns that share a scale
__host__ __device__ inline int64_t q8_blocks(int64_t cols) { return (cols + kQ8Block - 1) / kQ8Block; }

// |x| as integer bits, 0 for infinities and NaN (the order of positive floats
// is that of their bits).
__device__ __forceinline__ uint32_t q8_mag(float x) {
  const uint32_t a = __float_as_uint(x) & 0x7fffffffu;
  return a < 0x7f800000u ? a : 0u;
}
// k from the bits of amax: 2^e * m <= 448 * 2^k = 1.75 * 2^(8 + k) with m in
// [1, 2) gives k = e - 8, or e - 7 where m > 1.75.
__device__ __forceinline__ int q8_exponent(uint32_t amax_bits) {
  const int k = (int)(amax_bits >> 23) - 135 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(k, -120);
}
__device__ __forceinline__ float q8_pow2(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// Four codes from four scaled values (x * 2^-k); NaN becomes NaN, but an
// infinity 448: values that may hold one go through q8_no_inf first.
__device__ __forceinline__ uint32_t q8_pack(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ float q8_no_inf(float x) {
  return (__float_as_uint(x) & 0x7fffffffu) == 0x7f800000u ? __uint_as_float(0x7fffffffu) : x;
}
// The values of four codes, times `scale` = 2^k.
__device__ __forceinline__ void q8_unpack(uint32_t w, float scale, float* v) {
  const __half2 lo(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3));
  const __half2 hi(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3));
  const float2 a = __half22float2(lo), b = __half22float2(hi);
  v[0] = a.x * scale; v[1] = a.y * scale; v[2] = b.x * scale; v[3] = b.y * scale;
}
// 2^(byte - 127) of a scale byte; a program may hand in ones that the encoder
// does not write: 0 stands for fp32's subnormal 2^-127, and 255 is NaN (as in the
// microscaling formats' scales), which makes every value of its block NaN.
__device__ __forceinline__ float q8_scale(uint32_t byte) {
  return __uint_as_float(byte << 23 | (((byte + 1u) & 0xfeu) == 0u ? 0x00400000u : 0u));
}
__device__ __forceinline__ float q8_value(uint32_t code, uint32_t byte) {
  float v[4];
  q8_unpack(code, q8_scale(byte), v);
  return v[0];
}

}  // namespace mlpk
