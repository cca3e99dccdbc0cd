// Appending rows to the paged caches with the rotary positions applied on the
// way, so that neither the rotated copy of the rows nor a second pass over them
// is needed: row t of a target goes to cache row slots[t], its rotated columns
// turned by positions[t] (the mathematics is at the top of rope.cu), the others
// copied, or quantised into a 4-bit row (cache4.cu). Queries and other targets
// of dsa_rope may turn in the same launch, in CTAs of their own.
//
// What bounds it is memory: each row is read once and written once. The rotated
// columns go a pair per lane, which has formed that pair's cosine and sine
// itself, once for all targets; a 4-bit row's latent dims one group of 16 per lane.
//  - Rows by themselves: bulk copies bring them to shared memory, a few tokens ahead,
//    and take them from there to their slots, so that the bytes in flight cost no
//    registers, and few tokens no chain of loads.
//  - With queries, or too wide for that: a token per warp, whose rows go through
//    registers.
//
// A pair's frequency is held as the 64-bit fraction of a turn per position, off
// by 2^-65 of a turn at most, so that position times frequency, wrapped at 2^64, is
// the angle's fraction of a turn: integer products in the place of the
// five fp64 operations per token and pair of rope.cu, which are shared by all
// heads there but by two rows here. The whole product goes to fp32, signed, so that
// small angles keep fp32's relative precision as they do there (its upper half alone
// leaves steps of 2^-32 turns, which at 10^-9 radians is all of the angle).
#include "append.cuh"
#include "q4.cuh"
#include "rope.cuh"

namespace dsa {

namespace {
constexpr int kRunsPerLane = 3;  // a latent row and an indexer key: 72 runs

// Cosine and sine of a pair that turns by `turn` 2^-64 turns per position.
__device__ __forceinline__ float2 cos_sin(unsigned long long turn, int pos) {
  float s, c;  // of the nearer way round: -1/2 .. 1/2 of a turn
  sincospif((float)(long long)(turn * (unsigned)pos) * 0x1p-63f, &s, &c);
  return make_float2(c, s);
}
__device__ __forceinline__ unsigned long long turn_of(double radians) {
  const double f = fabs(radians) * 0.15915494309189533577;  // 1 / (2 pi)
  const unsigned long long turn = __double2ull_rn((f - floor(f)) * 0x1p64);
  return radians < 0.0 ? 0ull - turn : turn;  // 1 - f would round a small f
}
// Pair i of bf16 columns x, turned into columns y; R columns in all. x and y may
// be global or shared memory, and the same.
__device__ __forceinline__ void turn_pair(const uint16_t* x, uint16_t* y, int i, int R, bool half, float2 cs,
                                          float scale) {
  const uint32_t w = half ? x[i] | (uint32_t)x[R / 2 + i] << 16 : reinterpret_cast<const uint32_t*>(x)[i];
  float a = lo_f(w), b = hi_f(w);
  turn1(a, b, cs, scale);
  const uint32_t v = pack_bf16(a, b);
  if (half) {
    y[i] = (uint16_t)v;
    y[R / 2 + i] = (uint16_t)(v >> 16);
  } else {
    reinterpret_cast<uint32_t*>(y)[i] = v;
  }
}
// Group `lane` of 16 latent dims (u, v) into a 4-bit row.
__device__ __forceinline__ void put_group(const uint4& u, const uint4& v, uint8_t* row) {
  const uint32_t x0[4] = {u.x, u.y, u.z, u.w}, x1[4] = {v.x, v.y, v.z, v.w};
  uint32_t sb;
  const uint2 code = quantise16(x0, x1, sb);
  reinterpret_cast<uint2*>(row)[lane_id()] = code;
  row[kRow4Codes + lane_id()] = (uint8_t)sb;
}

// A token's slot, -1 if nothing is written: a negative slot or position is a padding
// row.
__device__ __forceinline__ int checked_slot(const AppendParams& p, int slot, int pos) {
  if (pos < 0 || slot < 0) return -1;
  if (slot >= p.rows) {
    set_status(p.dev_status, DSA_STATUS_BAD_INDEX);
    return -1;
  }
  return slot;
}

// 16 bytes that pass: run u of all targets' of token t.
struct Run {
  const uint4* x;
  long long at;  // byte of the target's cache row `slot`
  int target;
};
__device__ __forceinline__ Run run_of(const AppendParams& p, long long t, int u) {
  int k = 0;
  while (k + 1 < p.n && u >= p.tg[k + 1].first) ++k;
  const AppendTarget& g = p.tg[k];
  const int col = (u - g.first) * 8, gap = col >= g.rot_off ? p.rot_dim : 0;  // before the rotated columns, or after
  return {reinterpret_cast<const uint4*>(g.x + t * g.x_stride + col + (g.split ? 0 : gap)), 2 * (col + gap), k};
}

// One token, through registers.
__device__ __forceinline__ void append_token(const AppendParams& p, int t) {
  const int lane = lane_id(), pairs = p.rot_dim / 2;
  // all loads that do not depend on others first
  uint4 v[kRunsPerLane], q0, q1;
#pragma unroll
  for (int i = 0; i < kRunsPerLane; ++i)
    if (32 * i + lane < p.runs) v[i] = __ldg(run_of(p, t, 32 * i + lane).x);
  if (p.n_q4) {
    const AppendTarget& g = p.tg[p.q4[0]];
    const uint4* x = reinterpret_cast<const uint4*>(g.x + t * g.x_stride) + 2 * lane;
    q0 = __ldg(x);
    q1 = __ldg(x + 1);
  }
  const double freq = lane < pairs ? __ldg(p.freqs + lane) : 0.0;
  const int pos = __ldg(p.positions + t), slot = checked_slot(p, __ldg(p.slots + t), pos);
  if (slot < 0) return;
  auto row = [&](int k) { return p.tg[k].cache + slot * p.tg[k].cache_stride; };
#pragma unroll
  for (int i = 0; i < kRunsPerLane; ++i)
    if (32 * i + lane < p.runs) {
      const Run w = run_of(p, t, 32 * i + lane);
      *reinterpret_cast<uint4*>(row(w.target) + w.at) = v[i];
    }
  for (int u = 32 * kRunsPerLane + lane; u < p.runs; u += 32) {  // the rest of wide rows
    const Run w = run_of(p, t, u);
    *reinterpret_cast<uint4*>(row(w.target) + w.at) = __ldg(w.x);
  }
  for (int i = lane; i < pairs; i += 32) {
    const float2 cs = cos_sin(turn_of(i == lane ? freq : __ldg(p.freqs + i)), pos);
#pragma unroll 1
    for (int k = 0; k < p.n; ++k) {
      const AppendTarget& g = p.tg[k];
      turn_pair(g.xr + t * g.xr_stride, reinterpret_cast<uint16_t*>(row(k) + g.rot_at), i, p.rot_dim, g.half, cs,
                g.scale);
    }
  }
#pragma unroll 1
  for (int j = 0; j < p.n_q4; ++j) {
    if (j) {
      const AppendTarget& g = p.tg[p.q4[j]];
      const uint4* x = reinterpret_cast<const uint4*>(g.x + t * g.x_stride) + 2 * lane;
      q0 = __ldg(x);
      q1 = __ldg(x + 1);
    }
    put_group(q0, q1, row(p.q4[j]));
  }
}

// The first `append_ctas` CTAs append, the others turn the targets of r.
__global__ void __launch_bounds__(kRopeWarps * 32)
    append_kernel(const __grid_constant__ AppendParams p, const __grid_constant__ RopeParams r) {
  griddep_launch_dependents();
  griddep_wait();
  extern __shared__ __align__(16) float2 cs_all[];
  if (blockIdx.x >= p.append_ctas) {
    rope_warp<16>(r, (long long)(blockIdx.x - p.append_ctas) * kRopeWarps + warp_id(),
                  cs_all + warp_id() * kRopeMaxDim / 2);
    return;
  }
  const long long t = (long long)blockIdx.x * kRopeWarps + warp_id();
  if (t < p.T) append_token(p, (int)t);
}

// Several tokens per warp, through shared memory. A warp has p.stages places of
// p.stage bytes for a token's rows: of each target the source row, laid out as
// the cache row, and behind a 4-bit target's the row of codes.
__global__ void __launch_bounds__(kRopeWarps * 32) append_bulk_kernel(const __grid_constant__ AppendParams p) {
  if (p.next_early) griddep_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kRopeWarps][kAppendStages];
  __shared__ unsigned long long turns[kRopeMaxDim / 2];
  __shared__ int gave_up;
  const int lane = lane_id(), warp = warp_id(), pairs = p.rot_dim / 2;
  volatile int* abort_flag = &gave_up;
  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&bars[warp][s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  // tokens t0, t0 + step, ...: at any time the warps work on neighbouring rows
  const int t0 = blockIdx.x * kRopeWarps + warp, step = gridDim.x * kRopeWarps;
  const int n = t0 < p.T ? (p.T - 1 - t0) / step + 1 : 0;
  const uint32_t ring = smem_u32(smem) + warp * p.stages * p.stage, bar0 = smem_u32(&bars[warp][0]);
  // A lane's copy in: piece lane % 3 of target lane / 3, the columns before the
  // rotated ones, those, the ones after; or the whole row. And its copy out: the
  // row of target `lane`.
  const uint8_t* in = nullptr;
  long long in_stride = 0;
  int in_bytes = 0, in_at = 0;
  if (lane < 3 * p.n) {
    const AppendTarget& g = p.tg[lane / 3];
    const int piece = lane % 3, before = 2 * g.rot_off, rot = 2 * p.rot_dim;
    in = reinterpret_cast<const uint8_t*>(g.split && piece == 1 ? g.xr : g.x) + (g.split && piece == 2 ? before : 0);
    in_stride = 2 * (g.split && piece == 1 ? g.xr_stride : g.x_stride);
    in_at = g.stage_at + (g.split ? piece == 0 ? 0 : piece == 1 ? before : before + rot : 0);
    in_bytes = g.split ? piece == 0 ? before : piece == 1 ? rot : 2 * g.D - before - rot : piece ? 0 : 2 * g.D;
    in += t0 * in_stride;
    in_stride *= step;
  }
  uint8_t* out = nullptr;
  long long out_stride = 0;
  int out_bytes = 0, out_at = 0;
  if (lane < p.n) {
    const AppendTarget& g = p.tg[lane];
    out = g.cache;
    out_stride = g.cache_stride;
    out_bytes = g.q4 ? kRow4Bytes : 2 * g.D;
    out_at = g.stage_at + (g.q4 ? 2 * g.D : 0);
  }
  griddep_wait();
  int slots = -1, positions = 0;  // of 32 tokens, one per lane
  int fill = 0;                   // the place that is filled next, with the next token's rows
  auto load = [&]() {
    if (lane == 0) mbar_arrive_expect_tx(&bars[warp][fill], p.row_bytes);
    __syncwarp();
    if (in_bytes) bulk_load(ring + fill * p.stage + in_at, in, in_bytes, bar0 + fill * 8);
    in += in_stride;
    if (++fill == p.stages) fill = 0;
  };
  // a place is filled again two tokens after its last user's, whose copies out
  // have been read by then but for the last one's
  int loaded = min(n, p.stages - 2);
#pragma unroll 1
  for (int j = 0; j < loaded; ++j) load();
  // the first tokens' slots and the pairs' turns while the first rows are on their way
  auto lookup = [&](int j) {
    if (j + lane >= n) return;
    const long long t = t0 + (long long)(j + lane) * step;
    slots = __ldg(p.slots + t);
    positions = __ldg(p.positions + t);
  };
  lookup(0);
  for (int i = threadIdx.x; i < pairs; i += kRopeWarps * 32) turns[i] = turn_of(__ldg(p.freqs + i));
  __syncthreads();
  bool ok = true;
  int j = 0, place = 0, phase = 0;
#pragma unroll 1
  for (; j < n; ++j) {
    if (j % 32 == 0) {
      if (j) lookup(j);
      slots = checked_slot(p, slots, positions);
    }
    const int slot = __shfl_sync(0xffffffffu, slots, j % 32), pos = __shfl_sync(0xffffffffu, positions, j % 32);
    if (loaded < n) {
      bulk_wait_read<1>();  // all but the last token's
      load();
      ++loaded;
    }
    if (!(ok = mbar_wait_warp(&bars[warp][place], phase, abort_flag))) break;
    const int at = warp * p.stages * p.stage + place * p.stage;
    uint8_t* rows = smem + at;
    if (++place == p.stages) place = 0, phase ^= 1;
    if (slot < 0) {
      bulk_commit();  // a group per token, empty or not
      continue;
    }
    for (int i = lane; i < pairs; i += 32) {
      const float2 cs = cos_sin(turns[i], pos);
#pragma unroll
      for (int k = 0; k < kAppendMaxTargets; ++k) {
        if (k >= p.n) break;
        const AppendTarget& g = p.tg[k];
        uint16_t* x = reinterpret_cast<uint16_t*>(rows + g.stage_at) + g.rot_off;
        turn_pair(x, g.q4 ? reinterpret_cast<uint16_t*>(rows + g.stage_at + 2 * g.D + g.rot_at) : x, i, p.rot_dim,
                  g.half, cs, g.scale);
      }
    }
#pragma unroll 1
    for (int k = 0; k < p.n_q4; ++k) {
      const AppendTarget& g = p.tg[p.q4[k]];
      const uint4* x = reinterpret_cast<const uint4*>(rows + g.stage_at) + 2 * lane;
      put_group(x[0], x[1], rows + g.stage_at + 2 * g.D);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane < p.n) bulk_store(out + slot * out_stride, rows + out_at, out_bytes);
    bulk_commit();
    __syncwarp();
  }
  if (!ok) {
    if (lane == 0) {
      set_status(p.dev_status, DSA_STATUS_TIMEOUT);
      for (int i = j; i < loaded; ++i)  // no copy may land after the CTA has gone
        mbar_wait_drain(&bars[warp][i % p.stages], (i / p.stages) & 1);
    }
    __syncwarp();
  }
  bulk_wait_read<0>();
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
    g.D = a.D;
    g.first = p.runs;
    g.q4 = q4;
    g.half = a.layout == DSA_ROPE_HALF;
    g.scale = a.scale;
    g.stage_at = p.stage;
    if (q4) p.q4[p.n_q4++] = i;
    p.runs += q4 ? 0 : (a.D - rot_dim) / 8;
    p.stage += 2 * a.D + (q4 ? kRow4Bytes : 0);
    p.row_bytes += 2 * a.D;
  }
  p.rot_dim = rot_dim;
  p.T = T;
  p.rows = rows;
  p.positions = positions;
  p.slots = slots;
  p.freqs = freqs;
  p.dev_status = dev_status;
  RopeParams group[2] = {};
  unsigned grid[2] = {};
  if (n_rot) {
    const int rc = plan_rope(rot, n_rot, T, rot_dim, positions, freqs, false, group, grid);
    if (rc != DSA_OK) return rc;
  }
  // Rows by themselves go through shared memory, with targets of dsa_rope beside them
  // through registers, in one launch with those. Measured, latent rows and indexer
  // keys by themselves, registers / shared memory: 16 bits, 8 tokens 2.9 / 2.4 us, 512
  // 3.1 / 2.6, 8192 9.9 / 7.7, 65537 50 / 33 (a plain copy of as many bytes 29.3); 4 bits,
  // 8 tokens 2.8 / 2.5, 4096 5.4 / 4.6, 65537 48 / 36. With 128 heads' queries, one launch
  // / two: 64 tokens 4.1 / 6.1, 1024 15.3 / 18.0, 4096 42 / 46. CTAs per SM: 65537 tokens,
  // 3 / 4 / 5 / 6 CTAs 38.2 / 32.7 / 40.0 / 38.7 us (fewer leave the memory idle, more
  // spread over more rows at a time); 4 bits 49.8 / 39.5 / 41.1 / 36.3.
  p.stages = std::min(kAppendStages, kAppendRing / p.stage);
  if (p.stages >= 3 && !group[0].n) {
    const long long ctas = std::min<long long>((p.n_q4 ? 6 : 4) * sm_count(), (T + kRopeWarps - 1LL) / kRopeWarps);
    // The next kernel's CTAs may come early where they find most of the GPU idle. CTAs
    // that come to SMs whose shared memory these hold keep the little L1 that is left
    // for as long as that kernel runs: dsa_rope of 128 heads behind 1024, 4096, 8192 rows
    // 21, 56, 99 us the two, 18, 46, 86 if it starts when these have ended; behind 64
    // rows 6.1, and 6.7.
    p.next_early = ctas <= sm_count();
    set_smem_attr_once(reinterpret_cast<const void*>(append_bulk_kernel), kRopeWarps * kAppendRing);
    DSA_LAUNCH_PDL(append_bulk_kernel, dim3((unsigned)ctas), dim3(kRopeWarps * 32), kRopeWarps * p.stages * p.stage,
                   stream, p);
  } else {
    p.append_ctas = (unsigned)((T + (long long)kRopeWarps - 1) / kRopeWarps);
    if ((long long)p.append_ctas + grid[0] >= (1LL << 31)) return DSA_ERR_UNSUPPORTED;
    DSA_LAUNCH_PDL(append_kernel, dim3(p.append_ctas + grid[0]), dim3(kRopeWarps * 32), kRopeSmem, stream, p, group[0]);
  }
  return group[1].n ? run_rope_elements(stream, group[1], grid[1]) : DSA_OK;
}

}  // namespace dsa
