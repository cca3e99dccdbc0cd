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
#include "rope.cuh"

namespace dsa {

namespace {
template <int kBytes>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const __grid_constant__ RopeParams p) {
  griddep_launch_dependents();
  griddep_wait();
  extern __shared__ __align__(16) float2 cs_all[];
  rope_warp<kBytes>(p, (long long)blockIdx.x * kRopeWarps + warp_id(), cs_all + warp_id() * kRopeMaxDim / 2);
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

int plan_rope(const dsa_rope_target* targets, int n, int T, int rot_dim, const int32_t* positions, const double* freqs,
              bool inverse, RopeParams (&group)[2], unsigned (&grid)[2]) {
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
  return DSA_OK;
}

int run_rope(cudaStream_t stream, const dsa_rope_target* targets, int n, int T, int rot_dim, const int32_t* positions,
             const double* freqs, bool inverse) {
  RopeParams group[2] = {};
  unsigned grid[2] = {};
  const int rc = plan_rope(targets, n, T, rot_dim, positions, freqs, inverse, group, grid);
  if (rc != DSA_OK) return rc;
  if (group[0].n)
    DSA_LAUNCH_PDL(rope_kernel<16>, dim3(grid[0]), dim3(kRopeWarps * 32), kRopeSmem, stream, group[0]);
  return group[1].n ? run_rope_elements(stream, group[1], grid[1]) : DSA_OK;
}

int run_rope_elements(cudaStream_t stream, const RopeParams& p, unsigned grid) {
  DSA_LAUNCH_PDL(rope_kernel<0>, dim3(grid), dim3(kRopeWarps * 32), kRopeSmem, stream, p);
  return DSA_OK;
}

}  // namespace dsa
