// What the paged kernels' arithmetic has in common: exponentials, and pairs of bf16 in 32 bits.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace msa {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The low and the high value of a bf16 pair, and a pair of two rounded ones.
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// P = (p0, p1), not negative, as the sum of two bf16 pairs that are both above 0 where P is: P cut off, and the rest. Both
// times an infinity are then that infinity (a part of 0, or below, would make it NaN). The rest is exact but for 2^-23 P,
// which keeps it above 0, and at most a bf16 step (2^-7 P), so it rounds to bf16 with 2^-16 P at most.
__device__ __forceinline__ uint32_t bf16_cut(float p0, float p1) {
  return __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
}
__device__ __forceinline__ uint32_t bf16_rest(float p0, float p1, uint32_t cut) {
  constexpr float above = 1.f + 0x1p-23f;
  return pack_bf16(fmaf(p0, above, -lo_f(cut)), fmaf(p1, above, -hi_f(cut)));
}

}  // namespace msa
