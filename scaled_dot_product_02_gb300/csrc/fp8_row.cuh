// fp8_row.cuh -- rows of an 8-bit cache: E4M3 codes times one power of two.
//
// A row's exponent is the least e with max |x| <= 448 2^e (448: the largest
// code), kept as a byte e + 127; value i is code_i 2^e. E4M3 is a floating
// format, so a power of two costs no precision against a scale that fits the
// row exactly (at most one of its 15 binades), and code times scale is exact in
// the row's 16-bit type: reading back rounds nothing, and attention can apply
// the scales to whole scores. For that the exponent is kept within
//   fp16: -15 (2^-9, the least code, times 2^-15 is fp16's least value) to 7 (448 2^7 = 57344)
//   bf16: -80 to 80 (and 2^80 times what the attention sums stays within fp32).
// Larger rows saturate, smaller ones lose their low bits. NaN stays NaN.
#pragma once
#include <cstdint>

namespace sdpa {

template <bool BF16>
struct Fp8Row {
  static constexpr int LO = BF16 ? -80 : -15, HI = BF16 ? 80 : 7;
};

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// 2^(byte - 127): the scale a byte stands for. 0 and 255, which no row is given, are 2^-127 and 2^128: kept within
// fp32's numbers by a zero and an infinity.
__device__ __forceinline__ float exp2_byte(int byte) { return __int_as_float(byte << 23); }

// The exponent of a row whose largest magnitude is `top` (0 and infinity included): the scale 2^(x - 8) of
// top = m 2^x, or twice that where m > 1.75, 448 being 1.75 2^8.
template <bool BF16>
__device__ __forceinline__ int fp8_row_exponent(float top) {
  const int bits = __float_as_int(top);
  const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000);
  return min(max(e, Fp8Row<BF16>::LO), Fp8Row<BF16>::HI);
}

// Four fp32 values -> four E4M3 codes (round to nearest even, saturating), x0 in the lowest byte.
__device__ __forceinline__ uint32_t pack_e4m3x4(float x0, float x1, float x2, float x3) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1), "f"(x0));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3), "f"(x2));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Two E4M3 codes -> their values as two fp16 (exact).
__device__ __forceinline__ uint32_t unpack_e4m3x2(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return h;
}

}  // namespace sdpa
