// e4m3 codes of the 8-bit K/V cache: conversions and the power-of-two scales.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "common.cuh"

namespace clsa {

// two codes (the low 16 bits of `codes`) -> two halves, exact (NaN stays NaN)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}
// four codes -> two half pairs (codes 0, 1 and 2, 3)
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi) : "r"(codes));
}
__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint16_t codes) {
  const uint32_t h = e4m3x2_to_f16x2(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// round to nearest even, beyond +-448 (infinities too) to +-448, NaN to NaN; x in the low byte
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}

// exponent of a block's scale: the smallest e >= -100 with amax 2^-e <= 448 = 1.75 * 2^8, at
// most 119 (448 * 2^119 is finite); amax_bits: the float's bits, finite and not negative
__device__ __forceinline__ int kv8_scale_exp(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127;
  const int r = (amax_bits & 0x7fffffu) > 0x600000u ? e - 7 : e - 8;
  return max(-100, min(119, r));
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127

}  // namespace clsa
