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
// What bounds it is memory: each rotated element is read and written once.
// A CTA takes one token (of all targets) or, when there are few tokens, a
// part of its heads, and a thread moves 16 bytes from each half of a pair
// run; columns that only pass through (out of place) move as 16-byte copies.
#include <cuda_bf16.h>

#include "common.cuh"
#include "steps.cuh"

namespace dsa {

namespace {
constexpr int kRopeThreads = 256;

struct RopeTarget {
  const void* x;
  void* y;
  long long xt, xh, yt, yh;  // strides in elements
  int H, rot_off;
  int rot_units, units;  // per head: units that rotate, all units
  int half, fp32, vec;   // layout, type, 16-byte path
  int copy;              // y is not x: the other columns are copied
  float scale;
};
struct RopeParams {
  RopeTarget tg[kRopeMaxTargets];
  int n, rot_dim;
  const int32_t* positions;
  const double* freqs;
  float sign;  // -1: turn back
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

// Units u = part * threads + tid, ... of one token's row of target g. A unit
// that rotates covers V pairs (two runs of V elements), one that copies V
// elements.
template <typename T, int V>
__device__ __forceinline__ void rope_rows(const RopeTarget& g, int t, int rot_dim, const float2* cs) {
  using P = Pack<T, V>;
  const T* x = static_cast<const T*>(g.x) + t * g.xt;
  T* y = static_cast<T*>(g.y) + t * g.yt;
  const int total = g.H * g.units, step = gridDim.y * kRopeThreads;
  for (int u = blockIdx.y * kRopeThreads + threadIdx.x; u < total; u += step) {
    const int h = u / g.units, r = u - h * g.units;
    const T* xr = x + h * g.xh;
    T* yr = y + h * g.yh;
    if (r < g.rot_units) {
      const int i0 = r * V;  // first pair
      const int ca = g.rot_off + (g.half ? i0 : 2 * i0), cb = ca + (g.half ? rot_dim / 2 : V);
      const P a = *reinterpret_cast<const P*>(xr + ca), b = *reinterpret_cast<const P*>(xr + cb);
      P oa, ob;
      if (g.half) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float2 c = cs[i0 + k];
          const float fa = to_f(a.v[k]), fb = to_f(b.v[k]), co = c.x * g.scale, si = c.y * g.scale;
          from_f(oa.v[k], fa * co - fb * si);
          from_f(ob.v[k], fb * co + fa * si);
        }
      } else {
        T in[2 * V], out[2 * V];
#pragma unroll
        for (int k = 0; k < V; ++k) in[k] = a.v[k], in[V + k] = b.v[k];
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float2 c = cs[i0 + k];
          const float fa = to_f(in[2 * k]), fb = to_f(in[2 * k + 1]), co = c.x * g.scale, si = c.y * g.scale;
          from_f(out[2 * k], fa * co - fb * si);
          from_f(out[2 * k + 1], fb * co + fa * si);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) oa.v[k] = out[k], ob.v[k] = out[V + k];
      }
      *reinterpret_cast<P*>(yr + ca) = oa;
      *reinterpret_cast<P*>(yr + cb) = ob;
    } else {
      int c = (r - g.rot_units) * V;  // columns before the rotated ones, then those after
      if (c >= g.rot_off) c += rot_dim;
      *reinterpret_cast<P*>(yr + c) = *reinterpret_cast<const P*>(xr + c);
    }
  }
}

__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float2 cs[kRopeMaxDim / 2];
  const int t = blockIdx.x;
  const int pos = __ldg(p.positions + t);
  if (pos < 0) return;  // a padding row: left as it is
  for (int i = threadIdx.x; i < p.rot_dim / 2; i += kRopeThreads) {
    const double turns = (double)pos * (__ldg(p.freqs + i) * 0.15915494309189533577);  // 1 / (2 pi)
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cs[i] = make_float2(c, s * p.sign);
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < p.n; ++k) {
    const RopeTarget& g = p.tg[k];
    if (g.fp32) {
      if (g.vec) rope_rows<float, 4>(g, t, p.rot_dim, cs);
      else rope_rows<float, 1>(g, t, p.rot_dim, cs);
    } else {
      if (g.vec) rope_rows<__nv_bfloat16, 8>(g, t, p.rot_dim, cs);
      else rope_rows<__nv_bfloat16, 1>(g, t, p.rot_dim, cs);
    }
  }
}
}  // namespace

int run_rope(cudaStream_t stream, const dsa_rope_target* targets, int n, int T, int rot_dim, const int32_t* positions,
             const double* freqs, bool inverse) {
  RopeParams p{};
  long long units = 0;
  for (int i = 0; i < n; ++i) {
    const dsa_rope_target& a = targets[i];
    if (a.H == 0) continue;
    RopeTarget& g = p.tg[p.n++];
    g = {a.x, a.y, a.x_stride_t, a.x_stride_h, a.y_stride_t, a.y_stride_h, a.H, a.rot_off, 0, 0,
         a.layout == DSA_ROPE_HALF, a.dtype == DSA_DTYPE_F32, 0, a.x != a.y, a.scale};
    // 16 bytes at a time where every run of a pair and every copied run
    // starts and ends on 16 bytes
    const int es = g.fp32 ? 4 : 2, v = 16 / es;
    auto mult = [&](long long k) { return k % v == 0; };
    g.vec = mult(g.xt) && mult(g.xh) && mult(g.yt) && mult(g.yh) && mult(a.rot_off) && mult(rot_dim / 2) &&
            mult(a.D) && ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y)) & 15u) == 0;
    const int run = g.vec ? v : 1;
    g.rot_units = rot_dim / 2 / run;
    g.units = g.rot_units + (g.copy ? (a.D - rot_dim) / run : 0);
    units += (long long)g.H * g.units;
  }
  if (p.n == 0) return DSA_OK;
  p.rot_dim = rot_dim;
  p.positions = positions;
  p.freqs = freqs;
  p.sign = inverse ? -1.f : 1.f;
  // few tokens: several CTAs share a token's heads, until the GPU is full
  const long long full = 4LL * sm_count();
  const long long parts = std::min<long long>((units + kRopeThreads - 1) / kRopeThreads, (full + T - 1) / T);
  DSA_LAUNCH_PDL(rope_kernel, dim3(T, (unsigned)std::min<long long>(std::max<long long>(parts, 1), 65535)),
                 dim3(kRopeThreads), 0, stream, p);
  return DSA_OK;
}

}  // namespace dsa
