// Appending rows to the paged caches with the rotary positions applied on the
// way, so that neither the rotated copy of the rows nor a second pass over them
// is needed: row t of a target goes to cache row slots[t], its rotated columns
// turned by positions[t] (the mathematics is at the top of rope.cu), the others
// copied, or quantised into a 4-bit row (cache4.cu). Queries and other targets
// of dsa_rope may turn in the same launch, in CTAs of their own.
//
// What bounds it is memory: each row is read once and written once. A warp
// takes one token and moves all of its targets' units, two 16-byte runs each
// (the halves of a run of pairs, or two runs that only pass), two units in
// flight per lane; a 4-bit row's latent dims are one group of 16 per lane.
#include "append.cuh"
#include "q4.cuh"
#include "rope.cuh"

namespace dsa {

namespace {
struct Unit16 {
  const uint8_t* xa;
  const uint8_t* xb;
  uint8_t* ya;
  uint8_t* yb;  // null: the unit has one run only
  int target, pair0;  // -1: no unit; passes through
};

// Unit u of token t, whose cache row is `slot`.
__device__ __forceinline__ Unit16 append_unit(const AppendParams& p, int t, long long slot, int u) {
  Unit16 m;
  m.target = -1;
  if (u >= p.units) return m;
  int k = 0;
  while (k + 1 < p.n && u >= p.tg[k + 1].first) ++k;
  const AppendTarget& g = p.tg[k];
  const int v = u - g.first;
  uint8_t* y = g.cache + slot * g.cache_stride;
  m.target = k;
  if (v < g.rot_units) {
    m.pair0 = v * 8;
    const int ca = g.half ? v * 8 : v * 16, cb = ca + (g.half ? p.rot_dim / 2 : 8);
    const uint16_t* x = g.xr + t * g.xr_stride;
    m.xa = reinterpret_cast<const uint8_t*>(x + ca);
    m.xb = reinterpret_cast<const uint8_t*>(x + cb);
    m.ya = y + g.rot_at + 2 * ca;
    m.yb = y + g.rot_at + 2 * cb;
  } else {  // columns that pass: those before the rotated ones, then those after
    m.pair0 = -1;
    const int ca = (v - g.rot_units) * 16, cb = ca + 8;  // of the passing columns
    const bool two = cb < g.pass;
    const int skip = p.rot_dim, da = ca >= g.rot_off ? skip : 0, db = cb >= g.rot_off ? skip : 0;
    const uint16_t* x = g.x + t * g.x_stride;
    m.xa = reinterpret_cast<const uint8_t*>(x + ca + (g.split ? 0 : da));
    m.xb = two ? reinterpret_cast<const uint8_t*>(x + cb + (g.split ? 0 : db)) : m.xa;
    m.ya = y + 2 * (ca + da);
    m.yb = two ? y + 2 * (cb + db) : nullptr;
  }
  return m;
}

__device__ __forceinline__ void append_token(const AppendParams& p, int t, float2* cs) {
  const int lane = lane_id();
  const int slot = __ldg(p.slots + t), pos = __ldg(p.positions + t);
  if (slot < 0 || pos < 0) return;  // a padding row: nothing is written
  if (slot >= p.rows) {
    if (lane == 0) set_status(p.dev_status, DSA_STATUS_BAD_INDEX);
    return;
  }
  for (int i = lane; i < p.rot_dim / 2; i += 32) {
    const double turns = (double)pos * (__ldg(p.freqs + i) * 0.15915494309189533577);  // 1 / (2 pi)
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cs[i] = make_float2(c, s);
  }
  __syncwarp();
#pragma unroll 1
  for (int u = lane; u < p.units; u += 64) {
    const Unit16 m[2] = {append_unit(p, t, slot, u), append_unit(p, t, slot, u + 32)};
    uint32_t a[2][4], b[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (m[k].target >= 0) {
        *reinterpret_cast<uint4*>(a[k]) = __ldg(reinterpret_cast<const uint4*>(m[k].xa));
        *reinterpret_cast<uint4*>(b[k]) = __ldg(reinterpret_cast<const uint4*>(m[k].xb));
      }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (m[k].target >= 0) {
        const AppendTarget& g = p.tg[m[k].target];
        if (m[k].pair0 >= 0) rotate_bf16(a[k], b[k], g.half, g.scale, cs + m[k].pair0);
        *reinterpret_cast<uint4*>(m[k].ya) = *reinterpret_cast<const uint4*>(a[k]);
        if (m[k].yb) *reinterpret_cast<uint4*>(m[k].yb) = *reinterpret_cast<const uint4*>(b[k]);
      }
  }
#pragma unroll 1
  for (int k = 0; k < p.n; ++k) {
    const AppendTarget& g = p.tg[k];
    if (!g.q4) continue;
    // one group of 16 latent dims per lane
    const uint4* src = reinterpret_cast<const uint4*>(g.x + t * g.x_stride) + 2 * lane;
    const uint4 u = __ldg(src), v = __ldg(src + 1);
    const uint32_t x0[4] = {u.x, u.y, u.z, u.w}, x1[4] = {v.x, v.y, v.z, v.w};
    uint32_t sb;
    const uint2 code = quantise16(x0, x1, sb);
    uint8_t* dst = g.cache + slot * g.cache_stride;
    reinterpret_cast<uint2*>(dst)[lane] = code;
    dst[kRow4Codes + lane] = (uint8_t)sb;
  }
}

// The first `append_ctas` CTAs append, the others turn the targets of r.
__global__ void __launch_bounds__(kRopeWarps * 32)
    append_kernel(const __grid_constant__ AppendParams p, const __grid_constant__ RopeParams r) {
  griddep_launch_dependents();
  griddep_wait();
  extern __shared__ __align__(16) float2 cs_all[];
  float2* cs = cs_all + warp_id() * kRopeMaxDim / 2;
  if (blockIdx.x < p.append_ctas) {
    const long long t = (long long)blockIdx.x * kRopeWarps + warp_id();
    if (t < p.T) append_token(p, (int)t, cs);
  } else {
    rope_warp<16>(r, (long long)(blockIdx.x - p.append_ctas) * kRopeWarps + warp_id(), cs);
  }
}
}  // namespace

int run_rope_append(cudaStream_t stream, const dsa_rope_target* rot, int n_rot, const dsa_append_target* app, int n_app,
                    int T, int rot_dim, const int32_t* positions, const int32_t* slots, const double* freqs,
                    long long rows, int32_t* dev_status) {
  AppendParams p{};
  for (int i = 0; i < n_app; ++i) {
    const dsa_append_target& a = app[i];
    AppendTarget& g = p.tg[p.n++];
    const bool q4 = a.format == DSA_CACHE_Q4;
    g.x = static_cast<const uint16_t*>(a.x);
    g.x_stride = a.x_stride;
    g.split = a.x_rot != nullptr;
    g.xr = g.split ? static_cast<const uint16_t*>(a.x_rot) : g.x + a.rot_off;
    g.xr_stride = g.split ? a.x_rot_stride : a.x_stride;
    g.cache = static_cast<uint8_t*>(a.cache);
    g.cache_stride = q4 ? kRow4Bytes : 2 * a.cache_stride;
    g.rot_at = q4 ? kRow4Codes + kRow4Scales : 2 * a.rot_off;
    g.rot_off = a.rot_off;
    g.pass = q4 ? 0 : a.D - rot_dim;
    g.rot_units = rot_dim / 16;
    g.first = p.units;
    g.half = a.layout == DSA_ROPE_HALF;
    g.scale = a.scale;
    g.q4 = q4;
    p.units += g.rot_units + (g.pass + 15) / 16;
  }
  p.rot_dim = rot_dim;
  p.T = T;
  p.rows = rows;
  p.positions = positions;
  p.slots = slots;
  p.freqs = freqs;
  p.dev_status = dev_status;
  p.append_ctas = (unsigned)((T + (long long)kRopeWarps - 1) / kRopeWarps);
  RopeParams group[2] = {};
  unsigned grid[2] = {};
  if (n_rot) {
    const int rc = plan_rope(rot, n_rot, T, rot_dim, positions, freqs, false, group, grid);
    if (rc != DSA_OK) return rc;
  }
  if ((long long)p.append_ctas + grid[0] >= (1LL << 31)) return DSA_ERR_UNSUPPORTED;
  DSA_LAUNCH_PDL(append_kernel, dim3(p.append_ctas + grid[0]), dim3(kRopeWarps * 32), kRopeSmem, stream, p, group[0]);
  return group[1].n ? run_rope_elements(stream, group[1], grid[1]) : DSA_OK;
}

}  // namespace dsa
