// Rows of the 4-bit latent cache: quantising write-back and read.
//
// Group g of 16 latent dims x: scale s = e4m3(max|x| / 6), code = e2m1(x / s)
// (both to the nearest, ties to even), value = code * s. e2m1 has 2
// significant bits and e4m3 4, so a value has at most 6 and is exact in bf16.
// The 64 rotary dims stay bf16: they carry positions, one eighth of the row.
// A group with an infinity or a NaN gets the NaN scale and reads back as NaN;
// one whose maximum is below 2^-10 * 6 reads back as zeros; one above
// 448 * 6 saturates.
//
// One warp per row, one group per lane: a lane reads 32 contiguous bytes and
// writes 8 (codes) + 1 (scale), so every access of the warp is one contiguous
// run; eight lanes copy the rotary part. Memory bound: 1152 bytes in, 416 out
// (or the reverse).
#include "common.cuh"
#include "q4.cuh"
#include "steps.cuh"

namespace dsa {

namespace {
constexpr int kRowThreads = 128;  // 4 rows per CTA
constexpr int kRowsPerCta = kRowThreads / 32;

__global__ void __launch_bounds__(kRowThreads) q4_write_back_kernel(
    const uint16_t* __restrict__ rows, long long src_stride, uint8_t* __restrict__ cache,
    const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ cu_q_lens,
    const int32_t* __restrict__ cu_kv_lens, const int32_t* __restrict__ page_indices, int T, int S, int P, int PTW,
    int ps, int32_t* dev_status) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = lane_id();
  const long long row = (long long)blockIdx.x * kRowsPerCta + warp_id();
  if (row >= min(T, __ldg(cu_q_lens + S))) return;  // past the end, or a padding row behind the last request
  const int t = (int)row;
  // the row's loads do not depend on where it goes: issue them first
  const uint4* src = reinterpret_cast<const uint4*>(rows + (size_t)t * src_stride);
  const uint4 u = __ldg(src + 2 * lane), v = __ldg(src + 2 * lane + 1);
  uint4 rp = make_uint4(0, 0, 0, 0);
  if (lane < kRow4Rope / 16) rp = __ldg(src + 64 + lane);
  const int s = seq_of_token_warp(cu_q_lens, S, t);
  const int q0 = __ldg(cu_q_lens + s), q1 = __ldg(cu_q_lens + s + 1);
  const int kv = __ldg(seq_lens + s);
  const long long pos = (long long)kv - (q1 - q0) + (t - q0);
  const long long ent = (long long)(__ldg(cu_kv_lens + s) / ps) + pos / ps;
  if (t < q0 || t >= q1 || pos < 0 || q1 - q0 > kv || ent < 0 || ent >= PTW) {
    if (lane == 0) set_status(dev_status, DSA_STATUS_BAD_METADATA);
    return;
  }
  const int pg = __ldg(page_indices + ent);
  if (pg < 0 || pg >= P) {
    if (lane == 0) set_status(dev_status, DSA_STATUS_BAD_METADATA);
    return;
  }
  uint8_t* dst = cache + ((size_t)pg * ps + (size_t)(pos % ps)) * kRow4Bytes;
  const uint32_t x0[4] = {u.x, u.y, u.z, u.w}, x1[4] = {v.x, v.y, v.z, v.w};
  uint32_t sb;
  const uint2 code = quantise16(x0, x1, sb);
  reinterpret_cast<uint2*>(dst)[lane] = code;
  dst[kRow4Codes + lane] = (uint8_t)sb;
  if (lane < kRow4Rope / 16) reinterpret_cast<uint4*>(dst + kRow4Codes + kRow4Scales)[lane] = rp;
}

__global__ void __launch_bounds__(kRowThreads) q4_read_rows_kernel(
    const uint8_t* __restrict__ cache, long long total_rows, const int32_t* __restrict__ slots, int N,
    uint16_t* __restrict__ rows, long long dst_stride, int32_t* dev_status) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = lane_id();
  const long long i = (long long)blockIdx.x * kRowsPerCta + warp_id();
  if (i >= N) return;
  const int slot = __ldg(slots + i);
  uint4 o[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}, rp = make_uint4(0, 0, 0, 0);
  if (slot >= 0 && slot < total_rows) {
    const uint8_t* src = cache + (size_t)slot * kRow4Bytes;
    const uint2 c = *(reinterpret_cast<const uint2*>(src) + lane);
    const float s = e4m3_value(src[kRow4Codes + lane]);
    if (lane < kRow4Rope / 16) rp = *(reinterpret_cast<const uint4*>(src + kRow4Codes + kRow4Scales) + lane);
    const uint32_t s2 = bf16x2_of(s);
    o[0] = q4_values8(c.x, s2);
    o[1] = q4_values8(c.y, s2);
  } else if (slot >= 0 && lane == 0) {
    set_status(dev_status, DSA_STATUS_BAD_INDEX);
  }
  uint4* dst = reinterpret_cast<uint4*>(rows + (size_t)i * dst_stride);
  dst[2 * lane] = o[0];
  dst[2 * lane + 1] = o[1];
  if (lane < kRow4Rope / 16) dst[64 + lane] = rp;
}
}  // namespace

int run_q4_write_back(cudaStream_t stream, const uint16_t* rows, long long src_stride, uint8_t* cache,
                      const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                      const int32_t* page_indices, int T, int S, int P, int PTW, int ps, int32_t* dev_status) {
  DSA_LAUNCH_PDL(q4_write_back_kernel, dim3((T - 1) / kRowsPerCta + 1), dim3(kRowThreads), 0, stream, rows, src_stride,
                 cache, seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps, dev_status);
  return DSA_OK;
}

int run_q4_read_rows(cudaStream_t stream, const uint8_t* cache, long long total_rows, const int32_t* slots, int N,
                     uint16_t* rows, long long dst_stride, int32_t* dev_status) {
  DSA_LAUNCH_PDL(q4_read_rows_kernel, dim3((N - 1) / kRowsPerCta + 1), dim3(kRowThreads), 0, stream, cache, total_rows,
                 slots, N, rows, dst_stride, dev_status);
  return DSA_OK;
}

}  // namespace dsa
