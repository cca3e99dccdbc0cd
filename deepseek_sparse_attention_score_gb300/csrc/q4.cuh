// Codes of the 4-bit latent cache -> bf16, in registers.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

namespace dsa {

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Pair i (0..3) of a word of codes, dims 2i (nibble i) and 2i + 1 (nibble
// i + 4), as bf16 bit patterns: the sign at the top, the three magnitude bits
// over the lowest exponent bits and the first mantissa bit. Read as bf16 that
// is the e2m1 value times 2^-126, subnormal codes included (an exponent field
// of zero means the same in both formats).
template <int i>
__device__ __forceinline__ uint32_t q4_pair_bits(uint32_t w) {
  constexpr int up = 6 - 4 * i;
  const uint32_t mag = (up >= 0 ? w << (up >= 0 ? up : 0) : w >> (up < 0 ? -up : 0)) & 0x01c001c0u;
  return ((w << (12 - 4 * i)) & 0x80008000u) | mag;
}

// The values of one word times `s2` / 2^126 (both halves of s2 alike). Exact:
// at most 2 + 4 significant bits, bf16 has 8, and bf16 products keep
// subnormals.
__device__ __forceinline__ uint4 q4_scaled8(uint32_t w, uint32_t s2) {
  return make_uint4(mul_bf16x2(q4_pair_bits<0>(w), s2), mul_bf16x2(q4_pair_bits<1>(w), s2),
                    mul_bf16x2(q4_pair_bits<2>(w), s2), mul_bf16x2(q4_pair_bits<3>(w), s2));
}

// The values of one word: first back to e2m1 values (times 2^126, which with
// the scale in one factor would overflow bf16), then the scale.
__device__ __forceinline__ uint4 q4_values8(uint32_t w, uint32_t s2) {
  const uint4 v = q4_scaled8(w, 0x7e807e80u);  // 2^126 in both halves
  return make_uint4(mul_bf16x2(v.x, s2), mul_bf16x2(v.y, s2), mul_bf16x2(v.z, s2), mul_bf16x2(v.w, s2));
}

__device__ __forceinline__ float e4m3_value(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h));
  return f;
}
__device__ __forceinline__ uint32_t bf16x2_of(float x) {
  const __nv_bfloat162 v = __float2bfloat162_rn(x);
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace dsa
