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
  // the largest magnitude as an integer of the bf16 bits: the order of the
  // values, with infinities and NaN on top
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_u16x2(m, max_u16x2(x0[i] & 0x7fff7fffu, x1[i] & 0x7fff7fffu));
  const uint32_t top = max(m & 0xffffu, m >> 16);
  uint32_t sb = 0x7fu;  // NaN, with zero codes
  uint2 code = make_uint2(0u, 0u);
  if (top < 0x7f80u) {
    sb = e4m3_of(__fdiv_rn(__uint_as_float(top << 16), 6.f));
    const float sc = e4m3_value(sb);
    const float r = sc > 0.f ? __frcp_rn(sc) : 0.f;
    code = make_uint2(quantise8(x0, r), quantise8(x1, r));
  }
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
