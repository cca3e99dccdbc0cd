// Attention of requests that share a prefix (prefix.cu).
#pragma once
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace dsa {

constexpr long long kPrefixMaxRows = (1LL << 31) - (1 << 16);  // T * H: a tile ends past them
constexpr int kPrefixMaxGroups = 1 << 20;

// A row tile: 256 rows or fewer of one group.
struct alignas(16) PrefixTile {
  int row0, rows;      // of [T * H]
  int s0, s1, last;    // first request, end of the group's, last token
  int prefix;          // positions read through the group's first request, whole boxes of keys
  int page_base;       // and where its page-table entries start
  int begin, end;      // its units, of all tiles' in a row
};
// What a cluster works on: units [begin, end), from row tile `tile` on, of which it
// has a copy; and the list that its end is the first to cut.
struct alignas(16) PrefixShare {
  int begin, end;
  int tile;
  int last;                // last share that works on the list that is cut
  int first_slot;          // place of this share's part (share k's is 2k)
  int cut_row0, cut_rows;  // the list's rows, 0: none is cut here first
  int pad;
  PrefixTile first;
};

struct PrefixParams {
  const uint16_t* q;   // bf16 [T, H, 576]
  const uint16_t* kv;  // bf16 [P, ps, row_stride]
  int row_stride;
  const int32_t* seq_lens;
  const int32_t* cu_q_lens;
  const int32_t* cu_kv_lens;
  const int32_t* page_indices;
  const int32_t* prefix_lens;    // [G]
  const int32_t* group_offsets;  // [G + 1], or null: one group of all requests
  int G, max_kv, T, S, P, PTW, ps, H;
  float scale_log2;  // sm_scale * log2(e)
  uint16_t* o;       // bf16 [T, H, 512]
  float* lse;        // [T, H] or null
  int32_t* dev_status;
  // workspace (set by run_prefix_mla)
  int32_t* tile_base;    // [G + 1] tiles of the groups before
  PrefixTile* tiles;
  int* unit_base;        // [tiles + 1] key tiles of the tiles before, where shared memory is too small
  PrefixShare* share;    // [shares], those past the work empty
  float* part_o;    // [2 * shares][256][512]
  float* part_lse;  // [2 * shares][256], log2
  int max_tiles, max_units, shares;  // max_units: key tiles of one row tile
};

// Whether all key tiles of a call, at most, can be counted in 31 bits.
bool prefix_units_fit(int T, int H, int G, int max_kv);
size_t prefix_workspace_bytes(int T, int H, int G);
// ws: at least that many bytes.
int run_prefix_mla(cudaStream_t stream, PrefixParams prm, void* ws);

}  // namespace dsa
