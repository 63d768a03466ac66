// pa_quant.cuh -- codes of the 8-bit pools: a row's values times 127 / amax
// (int8) or 448 / amax (FP8 E4M3), rounded to nearest even.
#pragma once

#include "pa_device.cuh"

namespace pa {

// The int8 code of one value as the low byte of its result, inv = 127 / amax of its row.
// 1.5 * 2^23 added to a float of that size leaves its nearest integer, ties to even, in the
// lowest bits. (The conversion instructions, an eighth of the addition's rate, bound the
// int8 kernels: 53 us in the place of 43 for 16 x 4096 cached keys of 8 heads turned.)
__device__ __forceinline__ uint32_t int8_code(float x, float inv) {
  const float t = fminf(fmaxf(__fmul_rn(x, inv), -127.f), 127.f);
  return __float_as_uint(__fadd_rn(t, 12582912.f));
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The E4M3 codes of two scaled values, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}

// The values of two E4M3 codes (exact in f16, and so in fp32).
__device__ __forceinline__ float2 e4m3x2_values(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  float2 f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// A row's largest magnitude maps to this code value.
template <bool FP8>
__device__ __forceinline__ float code_range() {
  return FP8 ? 448.f : 127.f;
}

// The factor from a row's values to its codes. Of rows below 1.3e-36 (FP8) the quotient
// is infinite, and an infinity times a zero beside the largest value a NaN.
template <bool FP8>
__device__ __forceinline__ float code_factor(float amax) {
  return fminf(__fdiv_rn(code_range<FP8>(), amax), 3.402823466e38f);
}

// Codes of eight consecutive values of a row as eight bytes.
template <bool FP8>
__device__ __forceinline__ uint2 codes_of8(const float* x, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float* f = x + 4 * i;
    if constexpr (FP8)
      w[i] = e4m3x2_of(__fmul_rn(f[0], inv), __fmul_rn(f[1], inv)) |
             (e4m3x2_of(__fmul_rn(f[2], inv), __fmul_rn(f[3], inv)) << 16);
    else
      w[i] = low_bytes(int8_code(f[0], inv), int8_code(f[1], inv), int8_code(f[2], inv),
                       int8_code(f[3], inv));
  }
  return make_uint2(w[0], w[1]);
}

// Values of eight codes, without their row's scale.
template <bool FP8>
__device__ __forceinline__ void values_of8(uint2 c, float* x) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (FP8) {
      const float2 lo = e4m3x2_values(w[i] & 0xffffu), hi = e4m3x2_values(w[i] >> 16);
      x[4 * i] = lo.x;
      x[4 * i + 1] = lo.y;
      x[4 * i + 2] = hi.x;
      x[4 * i + 3] = hi.y;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // code + 128 as the lowest byte of 2^23's mantissa: exact
        const uint32_t bits = __byte_perm(w[i] ^ 0x80808080u, 0x4b000000u, 0x7440 | j);
        x[4 * i + j] = __fadd_rn(__uint_as_float(bits), -8388736.f);
      }
    }
  }
}

}  // namespace pa
