// Rows on their way into the paged caches, rotary positions applied (append.cu).
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/dsa.h"

namespace dsa {

constexpr int kAppendMaxTargets = 4;
constexpr int kAppendTokens = 8;  // of one warp, at most

struct AppendTarget {
  const uint16_t* x;   // columns that pass, and with !split the rotated ones among them
  const uint16_t* xr;  // rotated columns
  long long x_stride, xr_stride;  // elements
  uint8_t* cache;
  long long cache_stride;  // bytes of a cache row
  int rot_at;              // byte of a cache row where the rotated columns start
  int rot_off, pass;       // first rotated column; columns that pass (4 bits: none, they are quantised)
  int first;               // units of the targets before
  int half, split;
  float scale;
};
struct AppendParams {
  AppendTarget tg[kAppendMaxTargets];
  int q4[kAppendMaxTargets], n_q4;  // targets that are quantised
  int n, units, rot_dim, T;
  int tokens;  // of a warp
  unsigned append_ctas;
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
