// Rows on their way into the paged caches, rotary positions applied (append.cu).
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/dsa.h"

namespace dsa {

constexpr int kAppendMaxTargets = 4;
constexpr int kAppendRing = 12 * 1024, kAppendStages = 4;  // a warp's places in shared memory: bytes, and how many

struct AppendTarget {
  const uint16_t* x;   // columns that pass, and with !split the rotated ones among them
  const uint16_t* xr;  // rotated columns
  long long x_stride, xr_stride;  // elements
  uint8_t* cache;
  long long cache_stride;  // bytes of a cache row
  int D, rot_off;
  int rot_at;    // byte of a cache row where the rotated columns start
  int first;     // runs of 16 bytes that pass of the targets before (of 4-bit rows none: they are quantised)
  int stage_at;  // byte of a token's place in shared memory
  int half, split, q4;
  float scale;
};
struct AppendParams {
  AppendTarget tg[kAppendMaxTargets];
  int q4[kAppendMaxTargets], n_q4;  // targets that are quantised
  int n, runs, rot_dim, T;
  int stages, stage, row_bytes;  // a warp's places in shared memory; bytes of one, and of a token's source rows
  unsigned append_ctas;
  bool next_early;  // append_bulk_kernel lets the stream's next kernel launch at once
  long long rows;  // of each cache: pages * page size
  const int32_t* positions;
  const int32_t* slots;
  const double* freqs;
  int32_t* dev_status;
};
// Targets are checked by the entry point.
int run_rope_append(cudaStream_t stream, const dsa_rope_target* rot, int n_rot, const dsa_append_target* app, int n_app,
                    int T, int rot_dim, const int32_t* positions, const int32_t* slots, const double* freqs,
                    long long rows, int32_t* dev_status);

}  // namespace dsa
