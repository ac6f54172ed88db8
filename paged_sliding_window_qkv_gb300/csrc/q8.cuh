// 8-bit rows: e4m3 codes under one power-of-two scale a row.
//
// A row y takes the least exponent e with max |y| <= 448 * 2^e (448: the largest e4m3 number), held
// to [-110, 120], and codes y * 2^-e rounded to nearest even. The multiplication is exact, so the
// code's rounding is the only one (at most 2^-4 of an element, 2^-10 * 2^e below 2^-6 * 2^e), and
// code * 2^e is exactly a bf16 number: its lowest bit is 2^(e-9) >= 2^-119, its significand 4 bits.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

namespace pg {
namespace {

constexpr int32_t kQ8Least = -110, kQ8Most = 120;

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float q8_pow2(int32_t e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// What a scale byte stands for: 2^(byte - 127), for byte 0 a subnormal number; 255 is NaN.
__device__ __forceinline__ float q8_scale(uint32_t byte) {
  return __uint_as_float(byte << 23 | (byte - 1u >= 254u ? 0x00400000u : 0u));
}

// The exponent of a row whose largest magnitude (finite, or 0) is m.
__device__ __forceinline__ int32_t q8_exponent_of(float m) {
  const uint32_t b = __float_as_uint(m);
  const int32_t e = (int32_t)(b >> 23) - 127 - ((b & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
  return min(max(e, kQ8Least), kQ8Most);
}

// The largest magnitude of a row spread over LPR consecutive lanes, N pairs a lane. Elements that are not
// finite become NaN (the conversion would turn an infinity into 448) and have no part in it. Every
// lane of the warp takes part.
template <int LPR, int N>
__device__ __forceinline__ float q8_largest(float2* y) {
  auto largest = [&]() {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) m = fmaxf(m, fmaxf(fabsf(y[k].x), fabsf(y[k].y)));  // (a NaN is passed over)
    return m;
  };
  auto reduced = [&]() {
    float m = largest();
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  };
  float m = reduced();
  if (__any_sync(0xffffffffu, m == INFINITY)) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (fabsf(y[k].x) == INFINITY) y[k].x = NAN;
      if (fabsf(y[k].y) == INFINITY) y[k].y = NAN;
    }
    m = reduced();
  }
  return m;
}

// Codes of four elements, the first in the low byte.
__device__ __forceinline__ uint32_t q8_codes(float2 a, float2 b, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a.x * inv, a.y * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(b.x * inv, b.y * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Values of two codes (the low 16 bits), unscaled; exact in 16 bits.
__device__ __forceinline__ __half2 q8_halves(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return *reinterpret_cast<const __half2*>(&h);
}
__device__ __forceinline__ float2 q8_values(uint32_t two) { return __half22float2(q8_halves(two)); }

}  // namespace
}  // namespace pg
