// Rotary positions. Pair i of a row at position p, (a, b) = elements
// (2i, 2i + 1) of the rotated columns (interleaved) or (i, i + R/2) (halves),
// becomes scale * (a cos - b sin, b cos + a sin) with the angle p * freqs[i];
// `inverse` turns by the negative angle, which is the transpose of the turn:
// the gradient with respect to x.
//
// The angle of a far position needs more bits than fp32 has (position 10^6
// at one radian each is off by 0.06 in fp32), so it is formed in turns in
// fp64, reduced to (-1/2, 1/2] there, and only the fraction goes to fp32 and
// sincospi. That is a few fp64 operations per (token, pair), shared by all
// heads of all targets through shared memory.
//
// What bounds it is memory: each rotated element is read and written once. A
// warp takes a run of one token's units: it forms the token's cosines and
// sines (one pair per lane and step), then moves units of two 16-byte runs,
// the two halves of a run of pairs or two runs that only pass through, two
// units in flight per lane. Warps share nothing, so the trigonometry of some
// hides behind the copies of others (with one block per token and a barrier
// between the two, 8192 tokens of the four tensors of a layer took 100 us).
// Targets whose rows do not lie on 16 bytes go element by element, in a launch
// of their own (queries of 128 heads beside one unaligned key head: 55 us for
// 8192 tokens, 204 with all targets element by element; 4.8 and 4.4 for 32).
#include <cuda_bf16.h>

#include "common.cuh"
#include "steps.cuh"

namespace dsa {

namespace {
constexpr int kRopeWarps = 4;
constexpr int kUnitsPerLane = 16;  // units a lane moves when tokens abound

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

template <int kBytes>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const __grid_constant__ RopeParams p) {
  griddep_launch_dependents();
  griddep_wait();
  extern __shared__ __align__(16) float2 cs_all[];
  const int lane = lane_id();
  float2* cs = cs_all + warp_id() * kRopeMaxDim / 2;
  const long long w = (long long)blockIdx.x * kRopeWarps + warp_id();
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
}  // namespace

namespace {
// Whether a target moves 16 bytes at a time: all of its runs start and end on
// 16 bytes.
bool in_runs(const dsa_rope_target& a, int rot_dim) {
  const int v = a.dtype == DSA_DTYPE_F32 ? 4 : 8;
  auto mult = [&](long long k) { return k % v == 0; };
  return mult(a.x_stride_t) && mult(a.x_stride_h) && mult(a.y_stride_t) && mult(a.y_stride_h) && mult(a.rot_off) &&
         mult(rot_dim / 2) && mult(a.D) && ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y)) & 15u) == 0;
}
}  // namespace

int run_rope(cudaStream_t stream, const dsa_rope_target* targets, int n, int T, int rot_dim, const int32_t* positions,
             const double* freqs, bool inverse) {
  // the targets that move 16 bytes at a time in one launch, those that go
  // element by element in another
  RopeParams group[2] = {};
  unsigned grid[2] = {};
  for (int e = 0; e < 2; ++e) {
    RopeParams& p = group[e];
    long long units = 0;
    for (int i = 0; i < n; ++i) {
      const dsa_rope_target& a = targets[i];
      if (a.H == 0 || in_runs(a, rot_dim) == (e == 1)) continue;
      const int run = e ? 1 : a.dtype == DSA_DTYPE_F32 ? 4 : 8;
      const int rot_units = rot_dim / 2 / run;
      const int copied = a.x != a.y ? ((a.D - rot_dim) / run + 1) / 2 : 0;  // in place the other columns stay
      p.tg[p.n++] = {a.x, a.y, a.x_stride_t, a.x_stride_h, a.y_stride_t, a.y_stride_h, a.H, a.D, a.rot_off, rot_units,
                     rot_units + copied, a.layout == DSA_ROPE_HALF, a.dtype == DSA_DTYPE_F32, (int)units,
                     ((1ULL << 40) + rot_units + copied - 1) / (rot_units + copied), a.scale};
      units += (long long)a.H * (rot_units + copied);
      if (units >= (1LL << 30)) return DSA_ERR_UNSUPPORTED;
    }
    if (p.n == 0) continue;
    p.rot_dim = rot_dim;
    p.T = T;
    p.positions = positions;
    p.freqs = freqs;
    p.sign = inverse ? -1.f : 1.f;
    // units per warp: sixteen per lane, fewer while there are fewer warps than
    // the GPU holds (64 per SM)
    int per_lane = kUnitsPerLane;
    while (per_lane > 1 && (long long)T * ((units + 32 * per_lane - 1) / (32 * per_lane)) < 64LL * sm_count())
      per_lane /= 2;
    p.chunk = 32 * per_lane;
    p.parts = (int)((units + p.chunk - 1) / p.chunk);
    const long long ctas = ((long long)T * p.parts + kRopeWarps - 1) / kRopeWarps;
    if (ctas >= (1LL << 31)) return DSA_ERR_UNSUPPORTED;
    grid[e] = (unsigned)ctas;
  }
  const size_t smem = kRopeWarps * (kRopeMaxDim / 2) * sizeof(float2);
  if (group[0].n) DSA_LAUNCH_PDL(rope_kernel<16>, dim3(grid[0]), dim3(kRopeWarps * 32), smem, stream, group[0]);
  if (group[1].n) DSA_LAUNCH_PDL(rope_kernel<0>, dim3(grid[1]), dim3(kRopeWarps * 32), smem, stream, group[1]);
  return DSA_OK;
}

}  // namespace dsa
