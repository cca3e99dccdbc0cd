// The steps around the attention: a step's page tables (tables.cu), rotary
// positions (rope.cu) and the 4-bit latent cache's rows (cache4.cu).
#pragma once
#include <algorithm>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/dsa.h"

namespace dsa {

constexpr int kTablesMaxRequests = 16384;  // three sums per request fit shared memory

struct TablesParams {
  const int32_t* q_lens;
  const int32_t* seq_lens;
  int32_t* block_table;  // [S, bt_stride], `width` entries of a row used
  long long bt_stride;
  int width;
  const int32_t* free_pages;
  int32_t* free_state;  // [3 + 2 S], or null: the list is used from its start
  int F, S, T, PTW, ps;
  int32_t* cu_q_lens;
  int32_t* cu_kv_lens;
  int32_t* page_indices;
  int32_t* token_seq;
  int32_t* positions;
  int32_t* slots;
  int32_t* n_taken;
  int32_t* dev_status;
  bool vec_out;  // page_indices is 16-byte aligned (set by run_page_tables)
};
int run_page_tables(cudaStream_t stream, TablesParams p);

constexpr int kRopeMaxTargets = 8;
constexpr int kRopeMaxDim = 512;
// a target's heads and columns: the kernel's division by reciprocal is exact
// while H * (units of a head)^2 < 2^40, and a head of 4096 columns has at most
// 2049 units
constexpr int kRopeMaxHeads = 65536, kRopeMaxColumns = 4096;
// Rotates every target's rows; the targets are checked by the entry point.
int run_rope(cudaStream_t stream, const dsa_rope_target* targets, int n, int T, int rot_dim, const int32_t* positions,
             const double* freqs, bool inverse);

// One row of the 4-bit latent cache: 512 e2m1 codes, 32 e4m3 scales, 64 bf16
// rotary dims.
constexpr int kRow4Codes = 256, kRow4Scales = 32, kRow4Rope = 128;
constexpr int kRow4Bytes = kRow4Codes + kRow4Scales + kRow4Rope;
static_assert(kRow4Bytes == DSA_Q4_ROW_BYTES, "include/dsa.h states the row size");
int run_q4_write_back(cudaStream_t stream, const uint16_t* rows, long long src_stride, uint8_t* cache,
                      const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                      const int32_t* page_indices, int T, int S, int P, int PTW, int ps, int32_t* dev_status);
int run_q4_read_rows(cudaStream_t stream, const uint8_t* cache, long long total_rows, const int32_t* slots, int N,
                     uint16_t* rows, long long dst_stride, int32_t* dev_status);

}  // namespace dsa
