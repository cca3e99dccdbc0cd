// extern "C" entry points of include/dsa.h: host-side argument checks,
// workspace carving, and the kernel launches of each operation.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include <nvtx3/nvToolsExt.h>

#include "append.cuh"
#include "attend.cuh"
#include "common.cuh"
#include "indexer.cuh"
#include "prefix.cuh"
#include "rows.h"
#include "steps.cuh"

namespace dsa {

static std::atomic<long long> g_launches{0};
void note_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

int sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 0 || dev >= 64) dev = 0;
  if (!cached[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cached[dev] = n;
  }
  return cached[dev];
}

void set_smem_attr_once(const void* func, int bytes) {
  struct Entry {
    const void* f;
    int dev;
  };
  static Entry done[64];
  static int ndone = 0;
  static std::mutex lock;  // calls may come from several threads at once
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> hold(lock);
  for (int i = 0; i < ndone; ++i)
    if (done[i].f == func && done[i].dev == dev) return;
  cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (ndone < 64) done[ndone++] = {func, dev};
}

static PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

bool encode_bf16_2d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t row_elems, uint32_t box_rows,
                    uint64_t used_cols) {
  auto fn = get_encode();
  if (!fn) return false;
  cuuint64_t dims[2] = {used_cols, rows};
  cuuint64_t strides[1] = {row_elems * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_bf16_3d(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t groups,
                    uint32_t box_rows) {
  auto fn = get_encode();
  if (!fn) return false;
  cuuint64_t dims[3] = {cols, rows, groups};
  cuuint64_t strides[2] = {cols * 2, cols * rows * 2};
  cuuint32_t box[3] = {64, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool ps_supported(int ps) { return ps == 32 || ps == 64 || ps == 128; }

static int check_meta(const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                      const int32_t* page_indices, int T, int S, int P, int PTW, int ps) {
  if (T < 0 || S < 0 || P < 0 || PTW < 0) return DSA_ERR_INVALID_ARGUMENT;
  if (T > 0 && (S < 1 || P < 1 || PTW < 1)) return DSA_ERR_INVALID_ARGUMENT;
  if (T > 0 && (!seq_lens || !cu_q_lens || !cu_kv_lens || !page_indices)) return DSA_ERR_INVALID_ARGUMENT;
  if (!ps_supported(ps)) return DSA_ERR_UNSUPPORTED;
  if ((long long)P * ps >= (1LL << 31)) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

static int indexer_common(cudaStream_t stream, const uint16_t* q, const float* w, const uint16_t* kcache,
                          const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                          const int32_t* page_indices, int T, int S, int P, int PTW, int ps, int Hi, int Di,
                          int max_kv, int k_pages, int32_t* topk_pages, int k, int32_t* topk, float* topk_scores,
                          void* ws, size_t ws_bytes, int32_t* dev_status) {
  int rc = check_meta(seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps);
  if (rc) return rc;
  if (Hi != 32 || Di != 128) return DSA_ERR_UNSUPPORTED;
  if (max_kv < 1) return DSA_ERR_INVALID_ARGUMENT;
  if (topk && k < 1) return DSA_ERR_INVALID_ARGUMENT;
  if (topk_pages && k_pages < 1) return DSA_ERR_INVALID_ARGUMENT;
  if (!topk && !topk_pages) return DSA_ERR_INVALID_ARGUMENT;
  if (T == 0) return DSA_OK;
  if (!q || !w || !kcache) return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(w) || !aligned16(kcache)) return DSA_ERR_ALIGNMENT;
  if (T >= (1 << 24) || S >= (1 << 24)) return DSA_ERR_UNSUPPORTED;
  const IndexerLayout L = indexer_layout(T, S, max_kv, ps);
  if (!ws || ws_bytes < L.total || !aligned16(ws)) return DSA_ERR_WORKSPACE;
  IndexerMeta m{w, seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps, max_kv, dev_status, 0, 0};
  IndexerPlan pl;
  IndexerOut out;
  rc = run_indexer(stream, m, q, kcache, ws, L, topk != nullptr, topk_pages != nullptr, &pl, &out);
  if (rc) return rc;
  if (topk) {
    rc = run_topk(stream, out.tok_scores, out.ld_tok, pl.nvis, T, 1, k, topk, topk_scores, max_kv);
    if (rc) return rc;
  }
  if (topk_pages) {
    rc = run_page_topk(stream, out.gran_scores, out.ld_gr, pl.nvis, T, ps, k_pages, topk_pages,
                       reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + L.page_scores), (long long)L.ld_pg,
                       (max_kv + ps - 1) / ps);
    if (rc) return rc;
  }
  return DSA_OK;
}

static int attend_check(const uint16_t* q, const uint16_t* kv, int row_stride, int T, int H, int Dk, int Dv,
                        uint16_t* o) {
  if (H < 0) return DSA_ERR_INVALID_ARGUMENT;
  if (Dk != 576 || Dv != 512) return DSA_ERR_UNSUPPORTED;
  if (row_stride != 576 && row_stride != 640) return DSA_ERR_UNSUPPORTED;
  if (T > 0 && H > 0 && (!q || !kv || !o)) return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(kv) || !aligned16(o)) return DSA_ERR_ALIGNMENT;
  if (T > 65535) return DSA_ERR_UNSUPPORTED;  // grid.y of the sparse, dense and window kernels; one bound for all
  return DSA_OK;
}

}  // namespace dsa

using namespace dsa;

namespace {
// One NVTX range per device entry point, so a timeline tool shows the ABI
// calls around their kernels (header-only NVTX: free unless a tool attaches).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};
}  // namespace

extern "C" {

int dsa_device_sm_count(void) { return sm_count(); }

int dsa_selftest_wait_timeout(dsa_stream_t stream, long long limit_clocks, int32_t* dev_status) {
  if (!dev_status || limit_clocks < 1 || limit_clocks > 10000000000LL) return DSA_ERR_INVALID_ARGUMENT;
  return run_wait_timeout_selftest(static_cast<cudaStream_t>(stream), limit_clocks, dev_status);
}

int dsa_topk_pages_from_tokens(dsa_stream_t stream, const int32_t* topk, int T, int K, int ps, int max_pages,
                               int cap, int32_t* pages, int32_t* counts, int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_topk_pages_from_tokens");
  if (T < 0 || K < 0 || ps < 1 || cap < 1) return DSA_ERR_INVALID_ARGUMENT;
  if (max_pages < 1 || max_pages > topk_pages_max_pages()) return DSA_ERR_UNSUPPORTED;
  if (T == 0) return DSA_OK;
  if (!pages || (K > 0 && !topk)) return DSA_ERR_INVALID_ARGUMENT;
  return run_topk_pages(static_cast<cudaStream_t>(stream), topk, T, K, ps, max_pages, cap, pages, counts,
                        dev_status);
}

int dsa_paged_write_back(dsa_stream_t stream, const uint16_t* rows, int src_stride, int D, uint16_t* cache,
                         int cache_stride, const int32_t* seq_lens, const int32_t* cu_q_lens,
                         const int32_t* cu_kv_lens, const int32_t* page_indices, int T, int S, int P, int PTW,
                         int ps, int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_paged_write_back");
  return dsa_paged_write_back_pair(stream, rows, src_stride, D, cache, cache_stride, nullptr, 0, 0, nullptr, 0,
                                   seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps, dev_status);
}

static int write_back_target_check(const uint16_t* rows, int src_stride, int D, uint16_t* cache, int cache_stride) {
  if (D < 0) return DSA_ERR_INVALID_ARGUMENT;
  if (D == 0) return DSA_OK;
  if (!rows || !cache) return DSA_ERR_INVALID_ARGUMENT;
  if (D % 8 || src_stride % 8 || cache_stride % 8 || D > src_stride || D > cache_stride) return DSA_ERR_UNSUPPORTED;
  if (!aligned16(rows) || !aligned16(cache)) return DSA_ERR_ALIGNMENT;
  return DSA_OK;
}

int dsa_paged_write_back_pair(dsa_stream_t stream, const uint16_t* rows0, int src_stride0, int D0, uint16_t* cache0,
                              int cache_stride0, const uint16_t* rows1, int src_stride1, int D1, uint16_t* cache1,
                              int cache_stride1, const int32_t* seq_lens, const int32_t* cu_q_lens,
                              const int32_t* cu_kv_lens, const int32_t* page_indices, int T, int S, int P, int PTW,
                              int ps, int32_t* dev_status) {
  if (T < 0 || S < 0 || P < 0 || PTW < 0) return DSA_ERR_INVALID_ARGUMENT;
  int rc = write_back_target_check(rows0, src_stride0, D0, cache0, cache_stride0);
  if (rc) return rc;
  if (rows1 || cache1 || D1) {
    rc = write_back_target_check(rows1, src_stride1, D1, cache1, cache_stride1);
    if (rc) return rc;
  }
  if (T == 0 || D0 == 0) {
    if (D1 == 0 || T == 0) return DSA_OK;
    // only the second cache: write it as the first
    rows0 = rows1, src_stride0 = src_stride1, D0 = D1, cache0 = cache1, cache_stride0 = cache_stride1;
    rows1 = nullptr, cache1 = nullptr, D1 = 0;
  }
  if (S < 1 || P < 1 || PTW < 1 || ps < 1) return DSA_ERR_INVALID_ARGUMENT;
  if (!seq_lens || !cu_q_lens || !cu_kv_lens || !page_indices) return DSA_ERR_INVALID_ARGUMENT;
  return run_paged_write_back(static_cast<cudaStream_t>(stream), rows0, src_stride0, D0, cache0, cache_stride0, rows1,
                              src_stride1, D1, cache1, cache_stride1, seq_lens, cu_q_lens, cu_kv_lens, page_indices,
                              T, S, P, PTW, ps, dev_status);
}
long long dsa_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int dsa_index_build_share_map(const int32_t* types, int num_layers, int skip_offset, int32_t* full_slot,
                              int32_t* src_slot, int32_t* num_full) {
  (void)skip_offset;  // accepted and unused, as in the reference map builder
  if (num_layers < 0 || !full_slot || !src_slot || !num_full) return DSA_ERR_INVALID_ARGUMENT;
  int last = -1, nfull = 0;
  for (int l = 0; l < num_layers; ++l) {
    const int ty = types ? types[l] : 0;
    if (ty == 0) {
      last = nfull++;
      full_slot[l] = last;
      src_slot[l] = last;
    } else if (ty == 1) {
      if (last < 0) return DSA_ERR_SHARED_BEFORE_FULL;
      full_slot[l] = -1;
      src_slot[l] = last;
    } else {
      return DSA_ERR_BAD_INDEXER_TYPE;
    }
  }
  *num_full = nfull;
  return DSA_OK;
}

size_t dsa_indexer_workspace_size(int T, int S, int max_kv, int ps) {
  if (T < 0 || S < 0 || max_kv < 1 || !ps_supported(ps)) return 0;
  return indexer_layout(T, S, max_kv, ps).total;
}

// workspace of the approximate top-k: the indexer's, then bin maxima and
// their positions [T, B], bin counts [T] and the selected bins [T, k]
static size_t approx_bins(int k, int over, int max_kv) {
  const long long kb = (long long)k * over;
  const size_t b = (size_t)(kb < max_kv ? kb : max_kv);
  return (b + 3) & ~(size_t)3;  // the row stride of the bin maxima: a multiple of four
}
static size_t approx_extra(int T, int k, int over, int max_kv) {
  const size_t B = approx_bins(k, over, max_kv);
  return 2 * align_up((size_t)T * B * 4, 256) + align_up((size_t)T * 4, 256) + align_up((size_t)T * k * 4, 256);
}

size_t dsa_indexer_topk_approx_workspace_size(int T, int S, int max_kv, int ps, int k, int over) {
  if (T < 0 || S < 0 || max_kv < 1 || !ps_supported(ps) || k < 1 || over < 1) return 0;
  return indexer_layout(T, S, max_kv, ps).total + approx_extra(T, k, over, max_kv);
}

int dsa_indexer_topk_approx(dsa_stream_t stream, const uint16_t* q, const float* w, const uint16_t* kcache,
                            const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                            const int32_t* page_indices, int T, int S, int P, int PTW, int ps, int Hi, int Di,
                            int max_kv, int k, int over, int32_t* topk, void* ws, size_t ws_bytes,
                            int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_indexer_topk_approx");
  int rc = check_meta(seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps);
  if (rc) return rc;
  if (Hi != 32 || Di != 128) return DSA_ERR_UNSUPPORTED;
  if (!topk || k < 1 || over < 1 || max_kv < 1) return DSA_ERR_INVALID_ARGUMENT;
  if (k > approx_max_k()) return DSA_ERR_UNSUPPORTED;
  if (T == 0) return DSA_OK;
  if (!q || !w || !kcache) return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(w) || !aligned16(kcache)) return DSA_ERR_ALIGNMENT;
  if (T >= (1 << 24) || S >= (1 << 24)) return DSA_ERR_UNSUPPORTED;
  const IndexerLayout L = indexer_layout(T, S, max_kv, ps);
  if (!ws || ws_bytes < L.total + approx_extra(T, k, over, max_kv) || !aligned16(ws)) return DSA_ERR_WORKSPACE;
  IndexerMeta m{w, seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps, max_kv, dev_status, 0, 0};
  IndexerPlan pl;
  IndexerOut out;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = run_indexer(st, m, q, kcache, ws, L, true, false, &pl, &out);
  if (rc) return rc;
  const size_t B = approx_bins(k, over, max_kv);
  uint8_t* x = static_cast<uint8_t*>(ws) + L.total;
  float* vals = reinterpret_cast<float*>(x);
  x += align_up((size_t)T * B * 4, 256);
  int* pos = reinterpret_cast<int*>(x);
  x += align_up((size_t)T * B * 4, 256);
  int* nb = reinterpret_cast<int*>(x);
  x += align_up((size_t)T * 4, 256);
  int32_t* cand = reinterpret_cast<int32_t*>(x);
  return run_topk_approx(st, out.tok_scores, out.ld_tok, pl.nvis, T, k, over, max_kv, vals, pos, nb, cand, topk);
}

int dsa_indexer_topk(dsa_stream_t stream, const uint16_t* q, const float* w, const uint16_t* kcache,
                     const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                     const int32_t* page_indices, int T, int S, int P, int PTW, int ps, int Hi, int Di, int max_kv,
                     int k, int32_t* topk, float* topk_scores, void* ws, size_t ws_bytes, int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_indexer_topk");
  if (!topk) return DSA_ERR_INVALID_ARGUMENT;
  return indexer_common(static_cast<cudaStream_t>(stream), q, w, kcache, seq_lens, cu_q_lens, cu_kv_lens,
                        page_indices, T, S, P, PTW, ps, Hi, Di, max_kv, 0, nullptr, k, topk, topk_scores, ws,
                        ws_bytes, dev_status);
}

int dsa_indexer_page_topk(dsa_stream_t stream, const uint16_t* q, const float* w, const uint16_t* kcache,
                          const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                          const int32_t* page_indices, int T, int S, int P, int PTW, int ps, int Hi, int Di,
                          int max_kv, int k_pages, int32_t* topk_pages, int k, int32_t* topk, float* topk_scores,
                          void* ws, size_t ws_bytes, int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_indexer_page_topk");
  if (!topk_pages) return DSA_ERR_INVALID_ARGUMENT;
  return indexer_common(static_cast<cudaStream_t>(stream), q, w, kcache, seq_lens, cu_q_lens, cu_kv_lens,
                        page_indices, T, S, P, PTW, ps, Hi, Di, max_kv, k_pages, topk_pages, k, topk, topk_scores,
                        ws, ws_bytes, dev_status);
}

int dsa_build_block_union(dsa_stream_t stream, const int32_t* topk_units, int T, int K, int QB, int u_max,
                          const int32_t* cu_q_lens, const int32_t* cu_kv_lens, int S, int ps, int PTW,
                          int32_t* units, uint32_t* member, int32_t* counts, int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_build_block_union");
  if (T < 0 || K < 1 || QB < 32 || QB % 32 != 0 || QB > 1024 || PTW < 1) return DSA_ERR_INVALID_ARGUMENT;
  if (cu_q_lens && (!cu_kv_lens || S < 1 || ps < 1)) return DSA_ERR_INVALID_ARGUMENT;
  if (u_max <= 0) u_max = (int)std::min<long long>((long long)QB * K, PTW);
  if (T == 0) return DSA_OK;
  if (!topk_units || !units || !member || !counts) return DSA_ERR_INVALID_ARGUMENT;
  return run_block_union(static_cast<cudaStream_t>(stream), topk_units, T, K, QB, u_max, cu_q_lens, cu_kv_lens, S,
                         ps, PTW, units, member, counts, dev_status);
}

size_t dsa_sparse_mla_decode_workspace_size(int T, int H, int Dv) {
  if (T <= 0 || H <= 0 || Dv != 512) return 0;
  const int z = attend_num_splits(T, H, 1 << 30, kModeToken);
  return attend_workspace_bytes(T, H, z);
}

int dsa_sparse_mla_decode(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv, int row_stride,
                          const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                          const int32_t* page_indices, const int32_t* sel, int K, int unit, int T, int S, int P,
                          int PTW, int ps, int H, int Dk, int Dv, float sm_scale, uint16_t* o, float* lse,
                          void* ws, size_t ws_bytes, int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_sparse_mla_decode");
  int rc = check_meta(seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps);
  if (rc) return rc;
  rc = attend_check(q, kv, row_stride, T, H, Dk, Dv, o);
  if (rc) return rc;
  if (K < 1 || (T > 0 && !sel)) return DSA_ERR_INVALID_ARGUMENT;
  if (unit != 1 && unit != ps) return DSA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(sm_scale)) return DSA_ERR_INVALID_ARGUMENT;
  if (T == 0 || H == 0) return DSA_OK;
  AttendParams prm{};
  prm.q = q;
  prm.kv = kv;
  prm.row_stride = row_stride;
  prm.seq_lens = seq_lens;
  prm.cu_q_lens = cu_q_lens;
  prm.cu_kv_lens = cu_kv_lens;
  prm.page_indices = page_indices;
  prm.T = T;
  prm.S = S;
  prm.P = P;
  prm.PTW = PTW;
  prm.ps = ps;
  prm.H = H;
  prm.scale_log2 = sm_scale * 1.4426950408889634f;
  prm.mode = unit == 1 ? kModeToken : kModePage;
  prm.sel = sel;
  prm.K = K;
  prm.o = o;
  prm.lse = lse;
  prm.dev_status = dev_status;
  int z = attend_num_splits(T, H, K, prm.mode);
  if (z > 1 && (!ws || ws_bytes < attend_workspace_bytes(T, H, z) || !aligned16(ws))) z = 1;
  prm.nsplit = z;
  return run_attend(static_cast<cudaStream_t>(stream), prm, ws, ws_bytes);
}

int dsa_dense_mla(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv, int row_stride, const int32_t* seq_lens,
                  const int32_t* cu_q_lens, const int32_t* cu_kv_lens, const int32_t* page_indices, int max_kv,
                  int T, int S, int P, int PTW, int ps, int H, int Dk, int Dv, float sm_scale, int sliding_window,
                  float soft_cap, uint16_t* o, float* lse, void* ws, size_t ws_bytes, int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_dense_mla");
  int rc = check_meta(seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps);
  if (rc) return rc;
  rc = attend_check(q, kv, row_stride, T, H, Dk, Dv, o);
  if (rc) return rc;
  if (max_kv < 1 || sliding_window < 0) return DSA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(sm_scale) || !std::isfinite(soft_cap) || soft_cap < 0.f) return DSA_ERR_INVALID_ARGUMENT;
  if (T == 0 || H == 0) return DSA_OK;
  AttendParams prm{};
  prm.q = q;
  prm.kv = kv;
  prm.row_stride = row_stride;
  prm.seq_lens = seq_lens;
  prm.cu_q_lens = cu_q_lens;
  prm.cu_kv_lens = cu_kv_lens;
  prm.page_indices = page_indices;
  prm.T = T;
  prm.S = S;
  prm.P = P;
  prm.PTW = PTW;
  prm.ps = ps;
  prm.H = H;
  prm.scale_log2 = sm_scale * 1.4426950408889634f;
  prm.mode = kModeDense;
  prm.window = sliding_window;
  if (soft_cap > 0.f) {
    prm.soft_cap_on = 1;
    prm.inv_cap_scale = sm_scale / soft_cap;
    prm.cap_log2 = soft_cap * 1.4426950408889634f;
  }
  prm.K = (max_kv + ps - 1) / ps;  // pages of the longest request: the split unit
  prm.o = o;
  prm.lse = lse;
  prm.dev_status = dev_status;
  int z = attend_num_splits(T, H, prm.K, prm.mode);
  if (z > 1 && (!ws || ws_bytes < attend_workspace_bytes(T, H, z) || !aligned16(ws))) z = 1;
  prm.nsplit = z;
  return run_attend(static_cast<cudaStream_t>(stream), prm, ws, ws_bytes);
}

int dsa_window_mla(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv, int row_stride, const int32_t* seq_lens,
                   const int32_t* cu_q_lens, const int32_t* cu_kv_lens, const int32_t* page_indices, int max_kv,
                   int T, int S, int P, int PTW, int ps, int H, int Dk, int Dv, float sm_scale, int sliding_window,
                   int num_sinks, float soft_cap, uint16_t* o, float* lse, void* ws, size_t ws_bytes,
                   int32_t* dev_status) {
  (void)ws, (void)ws_bytes;  // taken as dsa_dense_mla takes them; this form needs none
  NvtxRange nvtx_range("dsa_window_mla");
  int rc = check_meta(seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps);
  if (rc) return rc;
  rc = attend_check(q, kv, row_stride, T, H, Dk, Dv, o);
  if (rc) return rc;
  if (max_kv < 1 || sliding_window < 0 || num_sinks < 0) return DSA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(sm_scale) || !std::isfinite(soft_cap) || soft_cap < 0.f) return DSA_ERR_INVALID_ARGUMENT;
  if ((long long)T * H >= (1LL << 31)) return DSA_ERR_UNSUPPORTED;
  if (!std::isfinite(sm_scale * 1.4426950408889634f)) return DSA_ERR_INVALID_ARGUMENT;  // the kernel's logit factor
  if (T == 0 || H == 0) return DSA_OK;
  AttendParams prm{};
  prm.q = q;
  prm.kv = kv;
  prm.row_stride = row_stride;
  prm.seq_lens = seq_lens;
  prm.cu_q_lens = cu_q_lens;
  prm.cu_kv_lens = cu_kv_lens;
  prm.page_indices = page_indices;
  prm.T = T;
  prm.S = S;
  prm.P = P;
  prm.PTW = PTW;
  prm.ps = ps;
  prm.H = H;
  prm.scale_log2 = sm_scale * 1.4426950408889634f;
  prm.mode = kModeDense;
  prm.window = sliding_window > 0 ? sliding_window : INT_MAX;
  prm.sinks = num_sinks;
  // c tanh(l / c) is l to fp32 accuracy where |l| < 2^-12 c; from 2^60 on that
  // is every logit that a softmax can tell apart, and l / c would underflow.
  // A tiny cap's factor stops at the largest number, so that 0 stays 0.
  if (soft_cap > 0.f && soft_cap < 0x1p60f) {
    prm.soft_cap_on = 1;
    prm.inv_cap_scale = std::min(std::max(sm_scale / soft_cap, -FLT_MAX), FLT_MAX);
    prm.cap_log2 = soft_cap * 1.4426950408889634f;
  }
  // pages of the longest list, the split unit: at most the request's, or the
  // sinks' and the window's, which may start inside one
  const long long pages = ((long long)max_kv + ps - 1) / ps;
  const long long most = ((long long)num_sinks + ps - 1) / ps + ((long long)prm.window + ps - 1) / ps + 1;
  prm.K = (int)std::min(pages, most);
  prm.o = o;
  prm.lse = lse;
  prm.dev_status = dev_status;
  return run_attend_cache(static_cast<cudaStream_t>(stream), prm);
}

size_t dsa_prefix_mla_workspace_size(int T, int H, int G) {
  if (T <= 0 || H <= 0 || G <= 0 || (long long)T * H >= kPrefixMaxRows || G > kPrefixMaxGroups) return 0;
  return prefix_workspace_bytes(T, H, G);
}

int dsa_prefix_mla(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv, int row_stride, const int32_t* seq_lens,
                   const int32_t* cu_q_lens, const int32_t* cu_kv_lens, const int32_t* page_indices,
                   const int32_t* prefix_lens, const int32_t* group_offsets, int G, int max_kv, int T, int S, int P,
                   int PTW, int ps, int H, int Dk, int Dv, float sm_scale, uint16_t* o, float* lse, void* ws,
                   size_t ws_bytes, int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_prefix_mla");
  int rc = check_meta(seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps);
  if (rc) return rc;
  rc = attend_check(q, kv, row_stride, T, H, Dk, Dv, o);
  if (rc) return rc;
  if (G < 1 || max_kv < 1 || (G > 1 && !group_offsets)) return DSA_ERR_INVALID_ARGUMENT;
  if (G > kPrefixMaxGroups || max_kv > (1 << 30) || (long long)T * H >= kPrefixMaxRows) return DSA_ERR_UNSUPPORTED;
  if (!std::isfinite(sm_scale * 1.4426950408889634f)) return DSA_ERR_INVALID_ARGUMENT;  // the kernel's logit factor
  if (T == 0 || H == 0) return DSA_OK;
  if (!prefix_units_fit(T, H, G, max_kv)) return DSA_ERR_UNSUPPORTED;
  if (!prefix_lens) return DSA_ERR_INVALID_ARGUMENT;
  if (!ws || ws_bytes < prefix_workspace_bytes(T, H, G)) return DSA_ERR_WORKSPACE;
  if (!aligned16(ws)) return DSA_ERR_ALIGNMENT;
  PrefixParams prm{};
  prm.q = q;
  prm.kv = kv;
  prm.row_stride = row_stride;
  prm.seq_lens = seq_lens;
  prm.cu_q_lens = cu_q_lens;
  prm.cu_kv_lens = cu_kv_lens;
  prm.page_indices = page_indices;
  prm.prefix_lens = prefix_lens;
  prm.group_offsets = group_offsets;
  prm.G = G;
  prm.max_kv = max_kv;
  prm.T = T;
  prm.S = S;
  prm.P = P;
  prm.PTW = PTW;
  prm.ps = ps;
  prm.H = H;
  prm.scale_log2 = sm_scale * 1.4426950408889634f;
  prm.o = o;
  prm.lse = lse;
  prm.dev_status = dev_status;
  return run_prefix_mla(static_cast<cudaStream_t>(stream), prm, ws);
}

int dsa_sparse_mla_decode_q4(dsa_stream_t stream, const uint16_t* q, const uint8_t* cache, const int32_t* seq_lens,
                             const int32_t* cu_q_lens, const int32_t* cu_kv_lens, const int32_t* page_indices,
                             const int32_t* sel, int K, int unit, int T, int S, int P, int PTW, int ps, int H, int Dk,
                             int Dv, float sm_scale, uint16_t* o, float* lse, void* ws, size_t ws_bytes,
                             int32_t* dev_status) {
  (void)ws, (void)ws_bytes;  // taken as dsa_sparse_mla_decode takes them; this form needs none
  NvtxRange nvtx_range("dsa_sparse_mla_decode_q4");
  int rc = check_meta(seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps);
  if (rc) return rc;
  rc = attend_check(q, reinterpret_cast<const uint16_t*>(cache), 576, T, H, Dk, Dv, o);
  if (rc) return rc;
  if (K < 1 || (T > 0 && !sel)) return DSA_ERR_INVALID_ARGUMENT;
  if (unit != 1 && unit != ps) return DSA_ERR_INVALID_ARGUMENT;
  if (K > (1 << 30) || (long long)T * H >= (1LL << 31)) return DSA_ERR_UNSUPPORTED;
  AttendParams prm{};
  prm.scale_log2 = sm_scale * 1.4426950408889634f;
  if (!std::isfinite(prm.scale_log2 * 128.f)) return DSA_ERR_INVALID_ARGUMENT;  // the kernel's logit factor
  if (T == 0 || H == 0) return DSA_OK;
  prm.q = q;
  prm.kv4 = cache;
  prm.seq_lens = seq_lens;
  prm.cu_q_lens = cu_q_lens;
  prm.cu_kv_lens = cu_kv_lens;
  prm.page_indices = page_indices;
  prm.T = T;
  prm.S = S;
  prm.P = P;
  prm.PTW = PTW;
  prm.ps = ps;
  prm.H = H;
  prm.mode = unit == 1 ? kModeToken : kModePage;
  prm.sel = sel;
  prm.K = K;
  prm.o = o;
  prm.lse = lse;
  prm.dev_status = dev_status;
  return run_attend_cache(static_cast<cudaStream_t>(stream), prm);
}

int dsa_build_page_tables(dsa_stream_t stream, const int32_t* q_lens, const int32_t* seq_lens, int32_t* block_table,
                          int64_t bt_stride, int width, const int32_t* free_pages, int F, int S, int T, int PTW,
                          int ps, int32_t* cu_q_lens, int32_t* cu_kv_lens, int32_t* page_indices, int32_t* token_seq,
                          int32_t* positions, int32_t* slots, int32_t* n_taken, int32_t* dev_status) {
  return dsa_build_page_tables_next(stream, q_lens, seq_lens, block_table, bt_stride, width, free_pages, F, nullptr, S,
                                    T, PTW, ps, cu_q_lens, cu_kv_lens, page_indices, token_seq, positions, slots,
                                    n_taken, dev_status);
}

int dsa_build_page_tables_next(dsa_stream_t stream, const int32_t* q_lens, const int32_t* seq_lens,
                               int32_t* block_table, int64_t bt_stride, int width, const int32_t* free_pages, int F,
                               int32_t* free_state, int S, int T, int PTW, int ps, int32_t* cu_q_lens,
                               int32_t* cu_kv_lens, int32_t* page_indices, int32_t* token_seq, int32_t* positions,
                               int32_t* slots, int32_t* n_taken, int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_build_page_tables");
  if (S < 0 || T < 0 || PTW < 0 || F < 0 || width < 0 || bt_stride < width) return DSA_ERR_INVALID_ARGUMENT;
  if (!ps_supported(ps) || S > kTablesMaxRequests || (long long)width * ps >= (1LL << 31)) return DSA_ERR_UNSUPPORTED;
  if (T > (1 << 30) || PTW > (1 << 30)) return DSA_ERR_UNSUPPORTED;
  if (!cu_q_lens || !cu_kv_lens || !n_taken) return DSA_ERR_INVALID_ARGUMENT;
  if ((S > 0 && (!q_lens || !seq_lens)) || (S > 0 && width > 0 && !block_table) || (F > 0 && !free_pages) ||
      (PTW > 0 && !page_indices) || (T > 0 && (!token_seq || !positions || !slots)))
    return DSA_ERR_INVALID_ARGUMENT;
  TablesParams p{q_lens, seq_lens, block_table, bt_stride, width, free_pages, free_state, F, S, T, PTW, ps, cu_q_lens,
                 cu_kv_lens, page_indices, token_seq, positions, slots, n_taken, dev_status, false};
  return run_page_tables(static_cast<cudaStream_t>(stream), p);
}

// Whether n0 x n1 rows of D elements, s0 and s1 elements apart, are disjoint.
static bool rows_apart(long long n0, long long s0, long long n1, long long s1, long long D) {
  s0 = s0 < 0 ? -s0 : s0;
  s1 = s1 < 0 ? -s1 : s1;
  if (n0 <= 1) return n1 <= 1 || s1 >= D;
  if (n1 <= 1) return s0 >= D;
  if (s0 < s1) std::swap(n0, n1), std::swap(s0, s1);  // s1: the inner rows
  return s1 >= D && (s0 - D) / (n1 - 1) >= s1 && s0 >= D;
}

static int rope_check(const dsa_rope_target* targets, int n_targets, int T, int rot_dim) {
  if (n_targets > kRopeMaxTargets) return DSA_ERR_UNSUPPORTED;
  if (rot_dim < 2 || rot_dim % 2) return DSA_ERR_INVALID_ARGUMENT;
  if (rot_dim > kRopeMaxDim) return DSA_ERR_UNSUPPORTED;
  for (int i = 0; i < n_targets; ++i) {
    const dsa_rope_target& g = targets[i];
    if (g.H < 0 || g.D < 0 || g.rot_off < 0 || (long long)g.rot_off + rot_dim > g.D) return DSA_ERR_INVALID_ARGUMENT;
    if ((g.layout != DSA_ROPE_INTERLEAVED && g.layout != DSA_ROPE_HALF) || !std::isfinite(g.scale))
      return DSA_ERR_INVALID_ARGUMENT;
    if (g.dtype != DSA_DTYPE_BF16 && g.dtype != DSA_DTYPE_F32) return DSA_ERR_UNSUPPORTED;
    if (g.H > kRopeMaxHeads || g.D > kRopeMaxColumns) return DSA_ERR_UNSUPPORTED;
    if (T == 0 || g.H == 0) continue;
    if (!g.x || !g.y) return DSA_ERR_INVALID_ARGUMENT;
    if (g.x == g.y && (g.x_stride_t != g.y_stride_t || g.x_stride_h != g.y_stride_h)) return DSA_ERR_INVALID_ARGUMENT;
    if (!rows_apart(T, g.y_stride_t, g.H, g.y_stride_h, g.D)) return DSA_ERR_INVALID_ARGUMENT;
    const uintptr_t es = g.dtype == DSA_DTYPE_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(g.x) % es || reinterpret_cast<uintptr_t>(g.y) % es) return DSA_ERR_ALIGNMENT;
  }
  return DSA_OK;
}

int dsa_rope(dsa_stream_t stream, const dsa_rope_target* targets, int n_targets, int T, int rot_dim,
             const int32_t* positions, const double* freqs, int inverse) {
  NvtxRange nvtx_range("dsa_rope");
  if (T < 0 || !targets || n_targets < 1) return DSA_ERR_INVALID_ARGUMENT;
  const int rc = rope_check(targets, n_targets, T, rot_dim);
  if (rc) return rc;
  if (T == 0) return DSA_OK;
  if (!positions || !freqs) return DSA_ERR_INVALID_ARGUMENT;
  return run_rope(static_cast<cudaStream_t>(stream), targets, n_targets, T, rot_dim, positions, freqs, inverse != 0);
}

// Whether a part of the call writes what another reads or writes, in rows that its
// strides step over: the columns between a tensor's rows may be others'.
static bool append_parts_meet(const dsa_append_target* append, int n_append, const dsa_rope_target* rotate,
                              int n_rotate, int T, int rot_dim, long long cache_rows) {
  auto address = [](const void* p) { return (long long)reinterpret_cast<uintptr_t>(p); };
  auto cache_of = [&](const dsa_append_target& g) -> Rows {
    const bool q4 = g.format == DSA_CACHE_Q4;
    return {address(g.cache), cache_rows, q4 ? DSA_Q4_ROW_BYTES : 2 * g.cache_stride, q4 ? DSA_Q4_ROW_BYTES : 2 * g.D};
  };
  auto meets_target = [&](const Rows& r, const void* base, long long st, long long sh, const dsa_rope_target& g) {
    const long long es = g.dtype == DSA_DTYPE_F32 ? 4 : 2;
    const bool place = g.x == g.y;  // touches the rotated columns only
    return rows_meet(r, {address(base) + (place ? g.rot_off * es : 0), T, st * es, (place ? rot_dim : g.D) * es}, g.H,
                     sh * es);
  };
  for (int i = 0; i < n_append; ++i) {
    const dsa_append_target& g = append[i];
    const Rows cache = cache_of(g);
    for (int j = 0; j < i; ++j)
      if (rows_meet(cache, cache_of(append[j]))) return true;
    const bool split = g.x_rot != nullptr;
    const Rows source[2] = {{address(g.x), T, 2 * g.x_stride, 2 * (split ? g.D - rot_dim : g.D)},
                            {address(g.x_rot), split ? T : 0, 2 * g.x_rot_stride, 2 * rot_dim}};
    for (const Rows& x : source) {
      for (int j = 0; j < n_append; ++j)
        if (rows_meet(x, cache_of(append[j]))) return true;
      for (int j = 0; j < n_rotate; ++j)
        if (meets_target(x, rotate[j].y, rotate[j].y_stride_t, rotate[j].y_stride_h, rotate[j])) return true;
    }
    for (int j = 0; j < n_rotate; ++j) {
      const dsa_rope_target& r = rotate[j];
      if (meets_target(cache, r.x, r.x_stride_t, r.x_stride_h, r) || meets_target(cache, r.y, r.y_stride_t, r.y_stride_h, r))
        return true;
    }
  }
  return false;
}

int dsa_rope_append(dsa_stream_t stream, const dsa_append_target* append, int n_append, const dsa_rope_target* rotate,
                    int n_rotate, int T, int rot_dim, const int32_t* positions, const int32_t* slots,
                    const double* freqs, int P, int ps, int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_rope_append");
  if (T < 0 || P < 0 || !append || n_append < 1 || n_rotate < 0 || (n_rotate > 0 && !rotate))
    return DSA_ERR_INVALID_ARGUMENT;
  if (n_append > kAppendMaxTargets || !ps_supported(ps) || (long long)P * ps >= (1LL << 31)) return DSA_ERR_UNSUPPORTED;
  const int rc = rope_check(rotate, n_rotate, T, rot_dim);
  if (rc) return rc;
  if (rot_dim % 16) return DSA_ERR_UNSUPPORTED;
  for (int i = 0; i < n_append; ++i) {
    const dsa_append_target& g = append[i];
    if (g.rot_off < 0 || (long long)g.rot_off + rot_dim > g.D) return DSA_ERR_INVALID_ARGUMENT;
    if ((g.layout != DSA_ROPE_INTERLEAVED && g.layout != DSA_ROPE_HALF) || !std::isfinite(g.scale))
      return DSA_ERR_INVALID_ARGUMENT;
    if (g.format != DSA_CACHE_BF16 && g.format != DSA_CACHE_Q4) return DSA_ERR_UNSUPPORTED;
    const bool q4 = g.format == DSA_CACHE_Q4, split = g.x_rot != nullptr;
    if (q4 && (g.D != 576 || g.rot_off != 512 || rot_dim != 64)) return DSA_ERR_UNSUPPORTED;
    if (g.D > kRopeMaxColumns || g.D % 8 || g.rot_off % 8) return DSA_ERR_UNSUPPORTED;
    if (T == 0) continue;
    const int pass = g.D - rot_dim;
    const bool reads_x = !split || pass > 0;
    if ((reads_x && !g.x) || (P > 0 && !g.cache)) return DSA_ERR_INVALID_ARGUMENT;
    // a single row's strides are never stepped over
    if (T > 1 && ((reads_x && g.x_stride < (split ? pass : g.D)) || (split && g.x_rot_stride < rot_dim)))
      return DSA_ERR_INVALID_ARGUMENT;
    if (!q4 && g.cache_stride < g.D) return DSA_ERR_INVALID_ARGUMENT;
    if ((reads_x && g.x_stride % 8) || (split && g.x_rot_stride % 8) || (!q4 && g.cache_stride % 8))
      return DSA_ERR_UNSUPPORTED;
    if ((reads_x && !aligned16(g.x)) || !aligned16(g.x_rot) || !aligned16(g.cache)) return DSA_ERR_ALIGNMENT;
  }
  if (T == 0) return DSA_OK;
  if (!positions || !slots || !freqs) return DSA_ERR_INVALID_ARGUMENT;
  if (append_parts_meet(append, n_append, rotate, n_rotate, T, rot_dim, (long long)P * ps))
    return DSA_ERR_INVALID_ARGUMENT;
  return run_rope_append(static_cast<cudaStream_t>(stream), rotate, n_rotate, append, n_append, T, rot_dim, positions,
                         slots, freqs, (long long)P * ps, dev_status);
}

int dsa_rope_freqs(int rot_dim, double base, int scaling, double factor, int orig_max_pos, double beta_fast,
                   double beta_slow, double* freqs, double* mscale) {
  if (rot_dim < 2 || rot_dim % 2 || !freqs || !std::isfinite(base) || base <= 1.0) return DSA_ERR_INVALID_ARGUMENT;
  if (scaling < DSA_ROPE_SCALE_NONE || scaling > DSA_ROPE_SCALE_YARN) return DSA_ERR_UNSUPPORTED;
  const bool yarn = scaling == DSA_ROPE_SCALE_YARN;
  if (scaling != DSA_ROPE_SCALE_NONE && (!std::isfinite(factor) || factor < 1.0)) return DSA_ERR_INVALID_ARGUMENT;
  if (yarn && (orig_max_pos < 1 || !std::isfinite(beta_fast) || !(beta_slow > 0.0) || !(beta_fast >= beta_slow)))
    return DSA_ERR_INVALID_ARGUMENT;
  double lo = 0, hi = 0;
  if (yarn) {
    // pair index at which a frequency makes `turns` turns over orig_max_pos
    auto at = [&](double turns) {
      return rot_dim * std::log(orig_max_pos / (turns * 2.0 * 3.14159265358979323846)) / (2.0 * std::log(base));
    };
    lo = std::max(std::floor(at(beta_fast)), 0.0);
    hi = std::min(std::ceil(at(beta_slow)), (double)rot_dim - 1);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot_dim);
    double keep = scaling == DSA_ROPE_SCALE_NONE ? 1.0 : 0.0;
    if (yarn) keep = 1.0 - std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
    freqs[i] = keep == 1.0 ? f : f * keep + f / factor * (1.0 - keep);
  }
  if (mscale) *mscale = yarn ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return DSA_OK;
}

int dsa_rope_attention_scales(double factor, double mscale, double mscale_all_dim, double* rotated, double* logits) {
  if (!rotated || !logits || !std::isfinite(factor) || factor < 1.0) return DSA_ERR_INVALID_ARGUMENT;
  const double m = 0.1 * mscale * std::log(factor) + 1.0, all = 0.1 * mscale_all_dim * std::log(factor) + 1.0;
  if (!std::isfinite(m) || !std::isfinite(all) || !(all > 0.0)) return DSA_ERR_INVALID_ARGUMENT;
  *rotated = m / all;
  *logits = all * all;
  return DSA_OK;
}

int dsa_q4_write_back(dsa_stream_t stream, const uint16_t* rows, int src_stride, uint8_t* cache,
                      const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                      const int32_t* page_indices, int T, int S, int P, int PTW, int ps, int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_q4_write_back");
  int rc = check_meta(seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps);
  if (rc) return rc;
  if (src_stride < 576 || src_stride % 8) return DSA_ERR_UNSUPPORTED;
  if (T == 0) return DSA_OK;
  if (!rows || !cache) return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned16(rows) || !aligned16(cache)) return DSA_ERR_ALIGNMENT;
  return run_q4_write_back(static_cast<cudaStream_t>(stream), rows, src_stride, cache, seq_lens, cu_q_lens, cu_kv_lens,
                           page_indices, T, S, P, PTW, ps, dev_status);
}

int dsa_q4_read_rows(dsa_stream_t stream, const uint8_t* cache, int P, int ps, const int32_t* slots, int N,
                     uint16_t* rows, int dst_stride, int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_q4_read_rows");
  if (P < 0 || N < 0) return DSA_ERR_INVALID_ARGUMENT;
  if (!ps_supported(ps) || (long long)P * ps >= (1LL << 31)) return DSA_ERR_UNSUPPORTED;
  if (dst_stride < 576 || dst_stride % 8) return DSA_ERR_UNSUPPORTED;
  if (N == 0) return DSA_OK;
  if ((P > 0 && !cache) || !slots || !rows) return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned16(cache) || !aligned16(rows)) return DSA_ERR_ALIGNMENT;
  return run_q4_read_rows(static_cast<cudaStream_t>(stream), cache, (long long)P * ps, slots, N, rows, dst_stride,
                          dev_status);
}

// No-allocation variant of dsa_sparse_mla_decode: the same checks and split
// choice; the split scratch is the library's built-in device array instead of
// a caller workspace.
int dsa_sparse_mla_decode_noalloc(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv, int row_stride,
                                  const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                                  const int32_t* page_indices, const int32_t* sel, int K, int unit, int T, int S,
                                  int P, int PTW, int ps, int H, int Dk, int Dv, float sm_scale, uint16_t* o,
                                  float* lse, int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_sparse_mla_decode_noalloc");
  int rc = check_meta(seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps);
  if (rc) return rc;
  rc = attend_check(q, kv, row_stride, T, H, Dk, Dv, o);
  if (rc) return rc;
  if (K < 1 || (T > 0 && !sel)) return DSA_ERR_INVALID_ARGUMENT;
  if (unit != 1 && unit != ps) return DSA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(sm_scale)) return DSA_ERR_INVALID_ARGUMENT;
  if (T == 0 || H == 0) return DSA_OK;
  AttendParams prm{};
  prm.q = q;
  prm.kv = kv;
  prm.row_stride = row_stride;
  prm.seq_lens = seq_lens;
  prm.cu_q_lens = cu_q_lens;
  prm.cu_kv_lens = cu_kv_lens;
  prm.page_indices = page_indices;
  prm.T = T;
  prm.S = S;
  prm.P = P;
  prm.PTW = PTW;
  prm.ps = ps;
  prm.H = H;
  prm.scale_log2 = sm_scale * 1.4426950408889634f;
  prm.mode = unit == 1 ? kModeToken : kModePage;
  prm.sel = sel;
  prm.K = K;
  prm.o = o;
  prm.lse = lse;
  prm.dev_status = dev_status;
  prm.nsplit = attend_num_splits(T, H, K, prm.mode);
  return run_attend_static_scratch(static_cast<cudaStream_t>(stream), prm);
}

static int qblock_common(cudaStream_t stream, const uint16_t* q, const uint16_t* kv, int row_stride,
                         const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                         const int32_t* page_indices, const int32_t* units, const uint32_t* member,
                         const int32_t* counts, int QB, int u_max, int T, int S, int P, int PTW, int ps, int H, int Dk,
                         int Dv, float sm_scale, int t_begin, int t_end, uint16_t* o, float* lse,
                         int32_t* dev_status) {
  int rc = check_meta(seq_lens, cu_q_lens, cu_kv_lens, page_indices, T, S, P, PTW, ps);
  if (rc) return rc;
  rc = attend_check(q, kv, row_stride, T, H, Dk, Dv, o);
  if (rc) return rc;
  if (QB < 32 || QB % 32 != 0 || u_max < 1) return DSA_ERR_INVALID_ARGUMENT;
  if (t_begin < 0 || t_end < t_begin || t_end > T) return DSA_ERR_INVALID_ARGUMENT;
  if (T > 0 && (!units || !member || !counts)) return DSA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(sm_scale)) return DSA_ERR_INVALID_ARGUMENT;
  if (t_end == t_begin || H == 0) return DSA_OK;
  AttendParams prm{};
  prm.q = q;
  prm.kv = kv;
  prm.row_stride = row_stride;
  prm.seq_lens = seq_lens;
  prm.cu_q_lens = cu_q_lens;
  prm.cu_kv_lens = cu_kv_lens;
  prm.page_indices = page_indices;
  prm.T = T;
  prm.S = S;
  prm.P = P;
  prm.PTW = PTW;
  prm.ps = ps;
  prm.H = H;
  prm.scale_log2 = sm_scale * 1.4426950408889634f;
  prm.mode = kModeQblock;
  prm.units = units;
  prm.member = member;
  prm.counts = counts;
  prm.QB = QB;
  prm.u_max = u_max;
  prm.K = 1;
  prm.nsplit = 1;
  prm.t0 = t_begin;
  prm.tn = t_end - t_begin;
  prm.o = o;
  prm.lse = lse;
  prm.dev_status = dev_status;
  return run_attend(stream, prm, nullptr, 0);
}

int dsa_sparse_mla_prefill_qblock(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv, int row_stride,
                                  const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                                  const int32_t* page_indices, const int32_t* units, const uint32_t* member,
                                  const int32_t* counts, int QB, int u_max, int T, int S, int P, int PTW, int ps,
                                  int H, int Dk, int Dv, float sm_scale, uint16_t* o, float* lse,
                                  int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_sparse_mla_prefill_qblock");
  return qblock_common(static_cast<cudaStream_t>(stream), q, kv, row_stride, seq_lens, cu_q_lens, cu_kv_lens,
                       page_indices, units, member, counts, QB, u_max, T, S, P, PTW, ps, H, Dk, Dv, sm_scale, 0,
                       T < 0 ? 0 : T, o, lse, dev_status);
}

int dsa_sparse_mla_prefill_qblock_range(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv, int row_stride,
                                        const int32_t* seq_lens, const int32_t* cu_q_lens,
                                        const int32_t* cu_kv_lens, const int32_t* page_indices,
                                        const int32_t* units, const uint32_t* member, const int32_t* counts, int QB,
                                        int u_max, int T, int S, int P, int PTW, int ps, int H, int Dk, int Dv,
                                        float sm_scale, int t_begin, int t_end, uint16_t* o, float* lse,
                                        int32_t* dev_status) {
  NvtxRange nvtx_range("dsa_sparse_mla_prefill_qblock_range");
  return qblock_common(static_cast<cudaStream_t>(stream), q, kv, row_stride, seq_lens, cu_q_lens, cu_kv_lens,
                       page_indices, units, member, counts, QB, u_max, T, S, P, PTW, ps, H, Dk, Dv, sm_scale,
                       t_begin, t_end, o, lse, dev_status);
}

}  // extern "C"
