// Values of the cache in 8 bits: E4M3 codes, and one power of two for each token
// and group (each token of the index keys), kept as its exponent + 127 in a byte
// (E8M0). code * 2^e has four significant bits, so it is exact in bf16, and the
// code alone is exact in fp16, which one conversion of two codes gives.
//
// The power of two is the smallest that brings a vector's largest magnitude to
// 448, E4M3's largest, or below. A scale of any value (max / 448) would use the
// format's range up to its end, but codes are floating-point numbers: what their
// rounding loses (2^-4 of a value) is the same for both, and values of it would
// not be exact in bf16 or fp16.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "paged_math.cuh"

namespace msa {

// Exponents are kept in [-117, 120]: 448 * 2^120 is above every bf16, and the smallest code, 2^-9, times 2^-117 is the
// smallest normal number. (With 2^120, what rounds to 256 = 0x78 is 2^128: an infinity in bf16 and fp32.)
constexpr int kLeastExp = 10, kMostExp = 247;

// The byte of a vector whose largest finite magnitude is `most`.
__device__ __forceinline__ int exp_byte(float most) {
  const uint32_t u = __float_as_uint(most);
  const int b = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u);  // 448 = 1.75 * 2^8
  return min(kMostExp, max(kLeastExp, b));
}
// 2^(byte - 127); and its inverse, for bytes of exp_byte.
__device__ __forceinline__ float exp_value(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float exp_inverse(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

// Largest magnitude of the finite ones.
__device__ __forceinline__ float finite_max(float most, float x) {
  const float m = fabsf(x);
  return m < INFINITY ? fmaxf(most, m) : most;
}
// (a, b) *= m
__device__ __forceinline__ void mul2(float& a, float& b, float m) {
  asm("{\n\t.reg .b64 x, m;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 m, {%2, %2};\n\tmul.rn.f32x2 x, x, m;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(m));
}
// Four codes of x * scale (a power of two), rounded to nearest, ties to even; NaN stays NaN.
__device__ __forceinline__ uint32_t four_codes(float a, float b, float c, float d, float scale) {
  mul2(a, b, scale);
  mul2(c, d, scale);
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// The fp16 pair of the low two codes of `v`, and of the high two.
__device__ __forceinline__ uint32_t f16_lo(uint32_t v) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t f16_hi(uint32_t v) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// The bf16 pair of an fp16 pair of codes times 2^e, exactly (2^128: an infinity).
__device__ __forceinline__ uint32_t scaled_bf16(uint32_t f16x2, float pow2) {
  float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f16x2));
  mul2(f.x, f.y, pow2);
  return pack_bf16(f.x, f.y);
}
// Eight codes as eight bf16.
__device__ __forceinline__ uint4 eight_bf16(uint2 codes, float pow2) {
  return make_uint4(scaled_bf16(f16_lo(codes.x), pow2), scaled_bf16(f16_hi(codes.x), pow2),
                    scaled_bf16(f16_lo(codes.y), pow2), scaled_bf16(f16_hi(codes.y), pow2));
}
// Eight codes as eight fp16, times a pair of equal fp16 powers of two.
__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint4 eight_f16(uint2 codes, uint32_t pow2) {
  return make_uint4(mul_f16(f16_lo(codes.x), pow2), mul_f16(f16_hi(codes.x), pow2), mul_f16(f16_lo(codes.y), pow2),
                    mul_f16(f16_hi(codes.y), pow2));
}

// A query as fp16, for products with codes: times the power of two that brings its largest finite magnitude into
// [2^14, 2^15), so that its values are exact down to 2^-28 of that and off by 2^-39 of it at most below (magnitudes under
// 2^-100 are treated as if the largest were that). Returns the scale; its inverse is exp_value(254 - byte).
__device__ __forceinline__ uint32_t query_scale_byte(float most) {
  const int up = max(27, (int)(__float_as_uint(most) >> 23));  // exponent + 127
  return 254 - (up - 14);                                      // 2^(14 - exponent)
}
__device__ __forceinline__ uint32_t f16_of_bf16(uint32_t pair, float scale) {
  return pack_f16(lo_f(pair) * scale, hi_f(pair) * scale);
}
// Largest finite magnitude of a bf16 pair and `most`.
__device__ __forceinline__ float finite_max2(float most, uint32_t pair) {
  return finite_max(finite_max(most, lo_f(pair)), hi_f(pair));
}

}  // namespace msa
