// fp4.cuh -- device conversions of the 4-bit formats (e2m1 codes, e4m3 and e8m0
// block scales).
#pragma once

#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace moe {

// two e2m1 codes (low nibble first) as floats
__device__ __forceinline__ float2 e2m1x2_to_f(uint32_t byte) {
  uint32_t h2;
  asm("{ .reg .b8 b, z; .reg .b16 w; cvt.u16.u32 w, %1; mov.b16 {b, z}, w; cvt.rn.f16x2.e2m1x2 %0, b; }"
      : "=r"(h2)
      : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}
// nearest e2m1 codes of two floats (a in the low nibble), ties to even,
// magnitudes beyond 6 saturate
__device__ __forceinline__ uint32_t f_to_e2m1x2(float a, float b) {
  uint32_t r;
  asm("{ .reg .b8 c; cvt.rn.satfinite.e2m1x2.f32 c, %2, %1; cvt.u32.u8 %0, c; }"
      : "=r"(r)
      : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float e4m3_to_f(uint32_t byte) {
  uint32_t h2;
  asm("{ .reg .b16 w; cvt.u16.u32 w, %1; cvt.rn.f16x2.e4m3x2 %0, w; }" : "=r"(h2) : "r"(byte));
  return __low2float(*reinterpret_cast<const __half2*>(&h2));
}
// nearest e4m3 code, ties to even, saturating at 448
__device__ __forceinline__ uint32_t f_to_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
  return r & 0xffu;
}
// 2^(byte - 127), NaN for 0xFF
__device__ __forceinline__ float e8m0_to_f(uint32_t byte) {
  if (byte == 0xffu) return __uint_as_float(0x7fffffffu);
  return byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);
}

}  // namespace moe
