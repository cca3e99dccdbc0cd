// Device pieces of the rotary positions that rope.cu and append.cu share: what
// a launch rotates, how a warp moves its share of a token, and the turn of a
// run of pairs (the mathematics is at the top of rope.cu).
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"
#include "steps.cuh"

namespace dsa {

constexpr int kRopeWarps = 4;
constexpr int kUnitsPerLane = 16;  // units a lane moves when tokens abound
constexpr size_t kRopeSmem = kRopeWarps * (kRopeMaxDim / 2) * sizeof(float2);

struct RopeTarget {
  const void* x;
  void* y;
  long long xt, xh, yt, yh;  // strides in elements
  int H, D, rot_off;
  int rot_units, units;  // per head: units that rotate, all units
  int half, fp32;        // layout, type
  int first;             // units of the targets before
  unsigned long long inv_units;  // ceil(2^40 / units): v * inv_units >> 40 is v / units
  float scale;
};
struct RopeParams {
  RopeTarget tg[kRopeMaxTargets];
  int n, rot_dim, T;
  int parts, chunk;  // warps per token, units per warp
  const int32_t* positions;
  const double* freqs;
  float sign;  // -1: turn back
};

__device__ __forceinline__ void turn1(float& a, float& b, float2 c, float scale) {
  const float co = c.x * scale, si = c.y * scale, x = a;
  a = x * co - b * si;
  b = b * co + x * si;
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The pairs of two 16-byte runs, from pair 0 of cs (16-byte aligned) on:
// halves hold a[k], b[k]; interleaved elements run on from a to b.
__device__ __forceinline__ void rotate_bf16(uint32_t (&a)[4], uint32_t (&b)[4], bool half, float scale,
                                            const float2* cs) {
  const float4* c4 = reinterpret_cast<const float4*>(cs);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (half) {  // pairs 2j, 2j + 1
      const float4 c = c4[j];
      float a0 = lo_f(a[j]), a1 = hi_f(a[j]), b0 = lo_f(b[j]), b1 = hi_f(b[j]);
      turn1(a0, b0, make_float2(c.x, c.y), scale);
      turn1(a1, b1, make_float2(c.z, c.w), scale);
      a[j] = pack_bf16(a0, a1);
      b[j] = pack_bf16(b0, b1);
    } else {  // pairs 2j, 2j + 1 of the eight: words 2j, 2j + 1 of a then b
      const float4 c = c4[j];
      uint32_t& w0 = j < 2 ? a[2 * j % 4] : b[2 * j % 4];
      uint32_t& w1 = j < 2 ? a[(2 * j + 1) % 4] : b[(2 * j + 1) % 4];
      float x0 = lo_f(w0), y0 = hi_f(w0), x1 = lo_f(w1), y1 = hi_f(w1);
      turn1(x0, y0, make_float2(c.x, c.y), scale);
      turn1(x1, y1, make_float2(c.z, c.w), scale);
      w0 = pack_bf16(x0, y0);
      w1 = pack_bf16(x1, y1);
    }
  }
}
__device__ __forceinline__ void rotate_f32(uint32_t (&a)[4], uint32_t (&b)[4], bool half, float scale,
                                           const float2* cs) {
  const float4* c4 = reinterpret_cast<const float4*>(cs);
#pragma unroll
  for (int j = 0; j < 2; ++j) {  // pairs 2j, 2j + 1 of the four
    const float4 c = c4[j];
    uint32_t* x[4] = {&a[2 * j], &b[2 * j], &a[2 * j + 1], &b[2 * j + 1]};
    uint32_t(&v)[4] = j ? b : a;
    float f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(half ? *x[k] : v[k]);
    turn1(f[0], f[1], make_float2(c.x, c.y), scale);
    turn1(f[2], f[3], make_float2(c.z, c.w), scale);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (half) *x[k] = __float_as_uint(f[k]);
      else v[k] = __float_as_uint(f[k]);
    }
  }
}

// One unit of a token: where its two runs of V elements are read and written.
// kBytes: 16, or 0 for single elements (V = 1).
struct Unit {
  const uint8_t* xa;
  const uint8_t* xb;
  uint8_t* ya;
  uint8_t* yb;  // null: the unit has one run only
  int target;   // -1: no unit
  int pair0;    // first pair, -1: passes through
};
template <int kBytes>
__device__ __forceinline__ Unit unit_of(const RopeParams& p, int t, int u, int end) {
  Unit m;
  m.target = -1;
  if (u >= end) return m;
  int k = 0;
  while (k + 1 < p.n && u >= p.tg[k + 1].first) ++k;
  const RopeTarget& g = p.tg[k];
  const int es = g.fp32 ? 4 : 2, V = kBytes ? kBytes / es : 1;
  const int v = u - g.first, h = (int)((unsigned)v * g.inv_units >> 40), r = v - h * g.units;
  int ca, cb;
  bool two = true;
  if (r < g.rot_units) {
    m.pair0 = r * V;
    ca = g.rot_off + (g.half ? r * V : 2 * r * V);
    cb = ca + (g.half ? p.rot_dim / 2 : V);
  } else {  // runs before the rotated columns, then those after
    m.pair0 = -1;
    const int run = 2 * (r - g.rot_units);
    ca = run * V;
    cb = ca + V;
    two = (run + 1) * V < g.D - p.rot_dim;
    if (ca >= g.rot_off) ca += p.rot_dim;
    if (cb >= g.rot_off) cb += p.rot_dim;
  }
  m.target = k;
  const uint8_t* x = static_cast<const uint8_t*>(g.x) + (t * g.xt + h * g.xh) * es;
  uint8_t* y = static_cast<uint8_t*>(g.y) + (t * g.yt + h * g.yh) * es;
  m.xa = x + ca * es;
  m.xb = two ? x + cb * es : m.xa;
  m.ya = y + ca * es;
  m.yb = two ? y + cb * es : nullptr;
  return m;
}

// One pair, or two elements that pass through.
__device__ __forceinline__ void move_elements(const Unit& m, const RopeTarget& g, const float2* cs) {
  if (g.fp32) {
    float a = *reinterpret_cast<const float*>(m.xa), b = *reinterpret_cast<const float*>(m.xb);
    if (m.pair0 >= 0) turn1(a, b, cs[m.pair0], g.scale);
    *reinterpret_cast<float*>(m.ya) = a;
    if (m.yb) *reinterpret_cast<float*>(m.yb) = b;
  } else {
    __nv_bfloat16 a = *reinterpret_cast<const __nv_bfloat16*>(m.xa), b = *reinterpret_cast<const __nv_bfloat16*>(m.xb);
    if (m.pair0 >= 0) {
      float fa = __bfloat162float(a), fb = __bfloat162float(b);
      turn1(fa, fb, cs[m.pair0], g.scale);
      a = __float2bfloat16_rn(fa);
      b = __float2bfloat16_rn(fb);
    }
    *reinterpret_cast<__nv_bfloat16*>(m.ya) = a;
    if (m.yb) *reinterpret_cast<__nv_bfloat16*>(m.yb) = b;
  }
}

// Warp w of the T * p.parts warps of a launch: its share of a token's units.
// cs: room for the token's cosines and sines, this warp's own.
template <int kBytes>
__device__ __forceinline__ void rope_warp(const RopeParams& p, long long w, float2* cs) {
  const int lane = lane_id();
  const int t = (int)(w / p.parts);
  if (t >= p.T) return;
  const int pos = __ldg(p.positions + t);
  if (pos < 0) return;  // a padding row: left as it is
  const RopeTarget& last = p.tg[p.n - 1];
  const int begin = (int)(w % p.parts) * p.chunk, end = min(begin + p.chunk, last.first + last.H * last.units);
  for (int i = lane; i < p.rot_dim / 2; i += 32) {
    const double turns = (double)pos * (__ldg(p.freqs + i) * 0.15915494309189533577);  // 1 / (2 pi)
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cs[i] = make_float2(c, s * p.sign);
  }
  __syncwarp();
#pragma unroll 1
  for (int u = begin + lane; u < end; u += 64) {
    const Unit m[2] = {unit_of<kBytes>(p, t, u, end), unit_of<kBytes>(p, t, u + 32, end)};
    if constexpr (kBytes == 16) {
      uint32_t a[2][4], b[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (m[k].target >= 0) {
          *reinterpret_cast<uint4*>(a[k]) = *reinterpret_cast<const uint4*>(m[k].xa);
          *reinterpret_cast<uint4*>(b[k]) = *reinterpret_cast<const uint4*>(m[k].xb);
        }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (m[k].target >= 0) {
          const RopeTarget& g = p.tg[m[k].target];
          if (m[k].pair0 >= 0) {
            if (g.fp32) rotate_f32(a[k], b[k], g.half, g.scale, cs + m[k].pair0);
            else rotate_bf16(a[k], b[k], g.half, g.scale, cs + m[k].pair0);
          }
          *reinterpret_cast<uint4*>(m[k].ya) = *reinterpret_cast<const uint4*>(a[k]);
          if (m[k].yb) *reinterpret_cast<uint4*>(m[k].yb) = *reinterpret_cast<const uint4*>(b[k]);
        }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (m[k].target >= 0) move_elements(m[k], p.tg[m[k].target], cs);
    }
  }
}

// Sorts a call's targets into those that move 16 bytes at a time (group 0) and
// those that go element by element (group 1), with the CTAs of kRopeWarps warps
// that each takes (0: it has no targets). Returns DSA_OK or an error.
int plan_rope(const dsa_rope_target* targets, int n, int T, int rot_dim, const int32_t* positions, const double* freqs,
              bool inverse, RopeParams (&group)[2], unsigned (&grid)[2]);
// Launches group 1.
int run_rope_elements(cudaStream_t stream, const RopeParams& p, unsigned grid);

}  // namespace dsa
