// e4m3 helpers shared by the kernels of the 8-bit KV pool (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace kv8 {

// Two floats rounded to nearest e4m3 (magnitudes above 448 become 448),
// `lo` in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes (low 16 bits) as an f16 pair, exactly.
__device__ __forceinline__ uint32_t to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"(uint16_t(codes)));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  float2 f;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// The least e >= -126 with amax <= 448 * 2^e, for a finite amax >= 0.  448 =
// 1.75 * 2^8, so it follows from amax's exponent and whether its mantissa
// exceeds 1.75.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = int(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

}  // namespace kv8
