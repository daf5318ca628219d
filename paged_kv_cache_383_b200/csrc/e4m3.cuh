// e4m3 codes of the 8-bit cache: conversions and the scales' powers of two.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace pagedkv {
namespace dev {

// The two codes in the low 16 bits of w as packed fp16: exact (an e4m3 value,
// subnormals included, is an fp16 value).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
// The same for the two codes in the high 16 bits.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

// Four floats to four codes (element 0 in the low byte), each rounded once to
// nearest even; magnitudes past 448 become 448, NaN stays NaN.
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c,
                                                    float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// 2^e as a float, e in [-126, 127].
__device__ __forceinline__ float exp2_int(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// floor(log2(x)) of a positive normal x, from its exponent field.
__device__ __forceinline__ int floor_log2(float x) {
  return static_cast<int>((__float_as_uint(x) >> 23) & 0xffu) - 127;
}

}  // namespace dev
}  // namespace pagedkv
