// Codes of the 4-bit latent cache <-> bf16, in registers.
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

// code pair e2m1(hi) << 4 | e2m1(lo), to the nearest even, saturating
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_of(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}
// 8 bf16 (four words) and 1/s -> one word of codes: dims 0, 2, 4, 6 in
// nibbles 0..3, dims 1, 3, 5, 7 in nibbles 4..7.
//
// x * r with r = 1/s rounded is within 2^-22 of x / s. x has 8 significant
// bits, s 4 and a boundary between two codes 3, so x / s is either exactly a
// boundary or at least 2^-8 away from it: rounding the product to 16 bits
// puts the first kind back on the boundary and moves none of the second over
// it, as an exact division would, at a fraction of its cost.
__device__ __forceinline__ uint32_t quantise8(const uint32_t (&x)[4], float r) {
  float e[4], o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __uint_as_float(x[i] << 16) * r, b = __uint_as_float(x[i] & 0xffff0000u) * r;
    e[i] = __uint_as_float((__float_as_uint(a) + 0x80u) & 0xffffff00u);
    o[i] = __uint_as_float((__float_as_uint(b) + 0x80u) & 0xffffff00u);
  }
  return e2m1_pair(e[0], e[1]) | (e2m1_pair(e[2], e[3]) << 8) | (e2m1_pair(o[0], o[1]) << 16) |
         (e2m1_pair(o[2], o[3]) << 24);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
// A group of 16 dims: its codes, and its scale sb (e4m3 bits).
__device__ __forceinline__ uint2 quantise16(const uint32_t (&x0)[4], const uint32_t (&x1)[4], uint32_t& sb) {
  // the largest magnitude as an integer of the bf16 bits: the order of the
  // values, with infinities and NaN on top
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_u16x2(m, max_u16x2(x0[i] & 0x7fff7fffu, x1[i] & 0x7fff7fffu));
  const uint32_t top = max(m & 0xffffu, m >> 16);
  sb = 0x7fu;  // NaN, with zero codes
  uint2 code = make_uint2(0u, 0u);
  if (top < 0x7f80u) {
    sb = e4m3_of(__fdiv_rn(__uint_as_float(top << 16), 6.f));
    const float sc = e4m3_value(sb);
    const float r = sc > 0.f ? __frcp_rn(sc) : 0.f;
    code = make_uint2(quantise8(x0, r), quantise8(x1, r));
  }
  return code;
}

}  // namespace dsa
