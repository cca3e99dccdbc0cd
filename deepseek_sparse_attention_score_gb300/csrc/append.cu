// Appending rows to the paged caches with the rotary positions applied on the
// way, so that neither the rotated copy of the rows nor a second pass over them
// is needed: row t of a target goes to cache row slots[t], its rotated columns
// turned by positions[t] (the mathematics is at the top of rope.cu), the others
// copied, or quantised into a 4-bit row (cache4.cu). Queries and other targets
// of dsa_rope may turn in the same launch, in CTAs of their own.
//
// What bounds it is memory: each row is read once and written once. A unit is
// two 16-byte runs of a row: the two halves of a run of pairs, or two runs that
// only pass, half a row apart so that the lanes of a warp cover whole lines. A
// lane keeps two units' places and walks over its warp's tokens with them; the
// loads of a token are issued before its angles are formed. A 4-bit row's latent
// dims are one group of 16 per lane.
//
// A pair's frequency is held as the 64-bit fraction of a turn per position, so
// that position times frequency, wrapped at 2^64, is the angle's fraction of a
// turn, exact to the frequency's 53 bits: integer products in the place of the
// five fp64 operations per token and pair of rope.cu, which are shared by all
// heads there but by two rows here.
#include "append.cuh"
#include "q4.cuh"
#include "rope.cuh"

namespace dsa {

namespace {
// A lane's unit: where its runs lie in row 0 of the source and of the cache.
struct RowUnit {
  const uint8_t* x;
  uint8_t* y;
  long long xs, ys;  // bytes from row to row
  int xb, yb;        // the second run's distance; yb 0: there is none
  int pair0;         // first pair, -1: passes
  bool some, half;
  float scale;
};

__device__ __forceinline__ RowUnit row_unit(const AppendParams& p, int u) {
  RowUnit m{};
  m.some = u < p.units;
  if (!m.some) return m;
  int k = 0;
  while (k + 1 < p.n && u >= p.tg[k + 1].first) ++k;
  const AppendTarget& g = p.tg[k];
  const int v = u - g.first, runs = g.pass / 8, pass_units = (runs + 1) / 2;
  m.ys = g.cache_stride;
  if (v < pass_units) {  // columns that pass: those before the rotated ones, then those after
    const int ca = v * 8, cb = ca + pass_units * 8;
    const int da = ca >= g.rot_off ? p.rot_dim : 0, db = cb >= g.rot_off ? p.rot_dim : 0;
    m.pair0 = -1;
    m.xs = 2 * g.x_stride;
    m.x = reinterpret_cast<const uint8_t*>(g.x + ca + (g.split ? 0 : da));
    m.y = g.cache + 2 * (ca + da);
    if (cb < g.pass) {
      m.yb = 2 * (cb + db - ca - da);
      m.xb = g.split ? 2 * (cb - ca) : m.yb;
    }
  } else {
    const int r = v - pass_units, ca = g.half ? r * 8 : r * 16;
    m.pair0 = r * 8;
    m.xb = m.yb = g.half ? p.rot_dim : 16;
    m.xs = 2 * g.xr_stride;
    m.x = reinterpret_cast<const uint8_t*>(g.xr + ca);
    m.y = g.cache + g.rot_at + 2 * ca;
    m.half = g.half;
    m.scale = g.scale;
  }
  return m;
}

// The tokens of one warp, t0 .. t1 - 1. turns: the pairs' frequencies; cs: room
// for a token's cosines and sines, this warp's own.
__device__ __forceinline__ void append_tokens(const AppendParams& p, int t0, int t1, const unsigned long long* turns,
                                              float2* cs) {
  const int lane = lane_id();
#pragma unroll 1
  for (int u0 = 0; u0 < p.units; u0 += 64) {  // 64 units at a time: all of them, unless rows are very wide
    const RowUnit m[2] = {row_unit(p, u0 + lane), row_unit(p, u0 + 32 + lane)};
    const bool quantise = u0 == 0 && p.n_q4 > 0;
#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
      const int slot = __ldg(p.slots + t), pos = __ldg(p.positions + t);
      uint32_t a[2][4], b[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (m[k].some) {
          const uint8_t* x = m[k].x + t * m[k].xs;
          *reinterpret_cast<uint4*>(a[k]) = __ldg(reinterpret_cast<const uint4*>(x));
          *reinterpret_cast<uint4*>(b[k]) = __ldg(reinterpret_cast<const uint4*>(x + m[k].xb));
        }
      uint4 q0, q1;
      auto load_group = [&](const AppendTarget& g) {
        const uint4* x = reinterpret_cast<const uint4*>(g.x + t * g.x_stride) + 2 * lane;
        q0 = __ldg(x);
        q1 = __ldg(x + 1);
      };
      if (quantise) load_group(p.tg[p.q4[0]]);
      if (slot < 0 || pos < 0) continue;  // a padding row: nothing is written
      if (slot >= p.rows) {
        if (lane == 0) set_status(p.dev_status, DSA_STATUS_BAD_INDEX);
        continue;
      }
      __syncwarp();  // the last token's have been read
      for (int i = lane; i < p.rot_dim / 2; i += 32) {
        float s, c;  // of the nearer way round: -1/2 .. 1/2 of a turn
        sincospif((float)(int)((turns[i] * (unsigned)pos) >> 32) * 0x1p-31f, &s, &c);
        cs[i] = make_float2(c, s);
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (m[k].some) {
          if (m[k].pair0 >= 0) rotate_bf16(a[k], b[k], m[k].half, m[k].scale, cs + m[k].pair0);
          uint8_t* y = m[k].y + slot * m[k].ys;
          *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(a[k]);
          if (m[k].yb) *reinterpret_cast<uint4*>(y + m[k].yb) = *reinterpret_cast<const uint4*>(b[k]);
        }
      if (quantise) {
#pragma unroll 1
        for (int k = 0; k < p.n_q4; ++k) {
          const AppendTarget& g = p.tg[p.q4[k]];
          if (k) load_group(g);
          const uint32_t x0[4] = {q0.x, q0.y, q0.z, q0.w}, x1[4] = {q1.x, q1.y, q1.z, q1.w};
          uint32_t sb;
          const uint2 code = quantise16(x0, x1, sb);
          uint8_t* y = g.cache + slot * g.cache_stride;
          reinterpret_cast<uint2*>(y)[lane] = code;
          y[kRow4Codes + lane] = (uint8_t)sb;
        }
      }
    }
  }
}

// The first `append_ctas` CTAs append, the others turn the targets of r.
__global__ void __launch_bounds__(kRopeWarps * 32)
    append_kernel(const __grid_constant__ AppendParams p, const __grid_constant__ RopeParams r) {
  griddep_launch_dependents();
  griddep_wait();
  extern __shared__ __align__(16) float2 cs_all[];
  __shared__ unsigned long long turns[kRopeMaxDim / 2];
  float2* cs = cs_all + warp_id() * kRopeMaxDim / 2;
  if (blockIdx.x >= p.append_ctas) {
    rope_warp<16>(r, (long long)(blockIdx.x - p.append_ctas) * kRopeWarps + warp_id(), cs);
    return;
  }
  for (int i = threadIdx.x; i < p.rot_dim / 2; i += kRopeWarps * 32) {
    const double f = __ldg(p.freqs + i) * 0.15915494309189533577;  // 1 / (2 pi)
    turns[i] = __double2ull_rn((f - floor(f)) * 0x1p64);
  }
  __syncthreads();
  const long long t0 = ((long long)blockIdx.x * kRopeWarps + warp_id()) * p.tokens;
  if (t0 < p.T) append_tokens(p, (int)t0, (int)min((long long)p.T, t0 + p.tokens), turns, cs);
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
    if (q4) p.q4[p.n_q4++] = i;
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
    g.first = p.units;
    g.half = a.layout == DSA_ROPE_HALF;
    g.scale = a.scale;
    p.units += rot_dim / 16 + (g.pass + 15) / 16;
  }
  p.rot_dim = rot_dim;
  p.T = T;
  p.rows = rows;
  p.positions = positions;
  p.slots = slots;
  p.freqs = freqs;
  p.dev_status = dev_status;
  // a token per warp while there are fewer warps than the GPU holds (32 per SM)
  p.tokens = (int)std::min<long long>(kAppendTokens, (T - 1) / (32LL * sm_count()) + 1);
  const long long per = (long long)kRopeWarps * p.tokens;
  p.append_ctas = (unsigned)((T + per - 1) / per);
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
