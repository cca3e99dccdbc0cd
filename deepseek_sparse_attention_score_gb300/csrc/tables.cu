// A serving step's metadata from its requests' lengths: cumulative offsets,
// the packed page table, block-table growth from a free list, and per query
// token its request, position and cache slot.
//
// With q = q_lens[s], n = seq_lens[s], had = ceil((n - q) / ps) and
// need = ceil(n / ps):
//   cu_q_lens[s] = sum_{r<s} q_r        cu_kv_lens[s] = ps * sum_{r<s} need_r
//   block_table[s][had + i] = free_pages[sum_{r<s} (need_r - had_r) + i]
//   page_indices[cu_kv_lens[s] / ps + j] = block_table[s][j],  j < need
//   token t = cu_q_lens[s] + i:  pos = n - q + i,
//   slot = block_table[s][pos / ps] * ps + pos % ps
//
// One launch. Every CTA scans all S lengths by itself (three sums at once,
// into shared memory), so no CTA waits for another; then the CTAs
// share the tokens and the page entries, each found by a binary search of
// the sums. A page taken from the free list is read from there, never from
// the block table, whose new entries other CTAs may still be writing. What
// bounds it is latency: the launch, one round trip for the lengths, the scan,
// one for the pages.
//
// With a free_state the list goes on where the last step stopped. A step with
// the last one's lengths is that step again and takes its pages again, so a
// call can be repeated; any other starts behind them. Every CTA reads the
// state and finds the same start; the CTA that arrives last, when no other
// will read it any more, writes the new one behind its other work (64 requests
// 4.1 us without a state, 4.9 with one; 2047 requests 6.4 and 8.2).
#include <climits>

#include "common.cuh"
#include "steps.cuh"

namespace dsa {

namespace {
constexpr int kTbThreads = 1024;
constexpr int kTbWarps = kTbThreads / 32;
static_assert(kTbWarps == 32, "one warp scans the warps' sums");
constexpr int kEntriesPerThread = 4;  // page entries a thread resolves with one search

// Sums of the requests before, each stopping at INT_MAX (a sum that stops is
// past every size that a call may have; adding that way is associative).
struct Sums {
  int q, need, grow;
};
__device__ __forceinline__ int add_sat(int a, int b) { return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)INT_MAX); }
__device__ __forceinline__ Sums operator+(Sums a, Sums b) {
  return {add_sat(a.q, b.q), add_sat(a.need, b.need), add_sat(a.grow, b.grow)};
}
__device__ __forceinline__ Sums shfl_up(Sums a, int d) {
  return {__shfl_up_sync(0xffffffffu, a.q, d), __shfl_up_sync(0xffffffffu, a.need, d),
          __shfl_up_sync(0xffffffffu, a.grow, d)};
}

// free_state: CTAs that have read it, list entries that the steps before the
// last one used and that the last one used, its q_lens and its seq_lens
enum : int { kStateArrived = 0, kStateUsed = 1, kStateTaken = 2, kStateLens = 3 };

// Lengths of request s; one that cannot be right counts as empty.
__device__ __forceinline__ bool lens_of(const TablesParams& p, int s, int& q, int& n) {
  q = __ldg(p.q_lens + s);
  n = __ldg(p.seq_lens + s);
  const bool ok = q >= 0 && n >= q && n <= p.width * (long long)p.ps;
  if (!ok) q = n = 0;
  return ok;
}

__device__ __forceinline__ int pages_of(int n, int ps, int lg) { return (int)(((uint32_t)n + (uint32_t)ps - 1u) >> lg); }

// largest s with a[s] <= x, a[0] == 0 and x < a[S] (skips empty requests)
__device__ __forceinline__ int find(const int* a, int S, int x) {
  int lo = 0, hi = S;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTbThreads) page_tables_kernel(const TablesParams p) {
  griddep_launch_dependents();
  griddep_wait();
  extern __shared__ int sums[];  // cumulative tokens, pages and taken pages, S + 1 each
  __shared__ Sums s_warp[kTbWarps];
  int* cq = sums;
  int* cp = cq + p.S + 1;
  int* cg = cp + p.S + 1;
  const int tid = threadIdx.x, lane = lane_id(), w = warp_id();
  const int lg = 31 - __clz(p.ps), top_pages = INT_MAX >> lg;
  int used = 0, last_took = 0;
  if (p.free_state) used = __ldcg(p.free_state + kStateUsed), last_took = __ldcg(p.free_state + kStateTaken);
  // each thread sums a contiguous run of requests
  const int per = (p.S + kTbThreads - 1) / kTbThreads;
  const int s0 = min(p.S, tid * per), s1 = min(p.S, s0 + per);
  Sums mine = {0, 0, 0};
  bool bad = false, moved = false;
  for (int s = s0; s < s1; ++s) {
    int q, n;
    bad |= !lens_of(p, s, q, n);
    if (p.free_state) {
      const int* last = p.free_state + kStateLens + s;
      moved |= (__ldcg(last) != __ldg(p.q_lens + s)) | (__ldcg(last + p.S) != __ldg(p.seq_lens + s));
    }
    const int need = pages_of(n, p.ps, lg);
    mine = mine + Sums{q, need, need - pages_of(n - q, p.ps, lg)};
  }
  Sums x = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums y = shfl_up(x, d);
    if (lane >= d) x = x + y;
  }
  if (lane == 31) s_warp[w] = x;
  Sums run = shfl_up(x, 1);
  if (lane == 0) run = {0, 0, 0};
  __syncthreads();
  if (w == 0) {  // the sums of the warps before each warp
    Sums v = s_warp[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums y = shfl_up(v, d);
      if (lane >= d) v = v + y;
    }
    s_warp[lane] = v;
  }
  __syncthreads();
  if (w > 0) run = s_warp[w - 1] + run;
  for (int s = s0; s < s1; ++s) {
    int q, n;
    lens_of(p, s, q, n);
    const int need = pages_of(n, p.ps, lg);
    cq[s] = run.q;
    cp[s] = min(run.need, top_pages);
    cg[s] = run.grow;
    run = run + Sums{q, need, need - pages_of(n - q, p.ps, lg)};
  }
  const Sums all = s_warp[kTbWarps - 1];
  if (tid == 0) {
    cq[p.S] = all.q;
    cp[p.S] = min(all.need, top_pages);
    cg[p.S] = all.grow;
  }
  int start = 0;          // list entries used before this step
  bool last_cta = false;  // thread 0: its CTA is the last to have read the state
  if (p.free_state) {
    moved = __syncthreads_or(moved);  // every thread has its part of the state
    start = max(0, min(p.F, moved ? add_sat(max(used, 0), max(last_took, 0)) : used));
    if (tid == 0) {
      __threadfence();
      last_cta = atomicAdd(p.free_state + kStateArrived, 1) == (int)gridDim.x - 1;
    }
  } else {
    __syncthreads();
  }
  const int total_q = cq[p.S], total_p = cp[p.S];
  if (blockIdx.x == 0) {
    for (int s = tid; s <= p.S; s += kTbThreads) {
      p.cu_q_lens[s] = cq[s];
      p.cu_kv_lens[s] = cp[s] << lg;
    }
    if (tid == 0) {
      *p.n_taken = cg[p.S];
      if (all.q > p.T || all.need > p.PTW) set_status(p.dev_status, DSA_STATUS_BAD_METADATA);
      if (all.grow > p.F - start) set_status(p.dev_status, DSA_STATUS_NO_PAGES);
    }
    if (bad) set_status(p.dev_status, DSA_STATUS_BAD_METADATA);
  }
  auto taken = [&](int s, int i) {  // page i of those that request s takes
    const long long k = (long long)start + cg[s] + i;
    return k < p.F ? __ldg(p.free_pages + k) : -1;
  };

  const int step = gridDim.x * kTbThreads, first = blockIdx.x * kTbThreads + tid;
  // tokens
  for (int t = first; t < p.T; t += step) {
    int s = -1, pos = -1, slot = -1;
    if (t < total_q) {
      s = find(cq, p.S, t);
      int q, n;
      lens_of(p, s, q, n);
      pos = n - q + (t - cq[s]);
      const int j = pos >> lg, had = pages_of(n - q, p.ps, lg);
      const int pg = j < had ? p.block_table[(size_t)s * p.bt_stride + j] : taken(s, j - had);
      if (pg >= 0 && pg <= (INT_MAX >> lg) - 1) slot = (pg << lg) + (pos & (p.ps - 1));
    }
    p.token_seq[t] = s;
    p.positions[t] = pos;
    p.slots[t] = slot;
  }
  // page-table entries, a few consecutive ones per thread
  const int groups = (p.PTW + kEntriesPerThread - 1) / kEntriesPerThread;
  for (int g = first; g < groups; g += step) {
    const int e0 = g * kEntriesPerThread;
    int out[kEntriesPerThread];
    int s = 0, had = 0, end = 0;
    if (e0 < total_p) {
      s = find(cp, p.S, e0);
      end = cp[s + 1];
      int q, n;
      lens_of(p, s, q, n);
      had = pages_of(n - q, p.ps, lg);
    }
#pragma unroll
    for (int i = 0; i < kEntriesPerThread; ++i) {
      const int e = e0 + i;
      out[i] = -1;
      if (e < total_p && e < p.PTW) {
        if (e >= end) {
          do ++s; while (cp[s + 1] <= e);
          end = cp[s + 1];
          int q, n;
          lens_of(p, s, q, n);
          had = pages_of(n - q, p.ps, lg);
        }
        const int j = e - cp[s];
        int32_t* bt = p.block_table + (size_t)s * p.bt_stride + j;
        if (j < had) {
          out[i] = *bt;
        } else {
          out[i] = taken(s, j - had);
          *bt = out[i];
        }
      }
    }
    if (e0 + kEntriesPerThread <= p.PTW && p.vec_out) {
      *reinterpret_cast<int4*>(p.page_indices + e0) = make_int4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
      for (int i = 0; i < kEntriesPerThread; ++i)
        if (e0 + i < p.PTW) p.page_indices[e0 + i] = out[i];
    }
  }
  if (p.free_state && __syncthreads_or(last_cta)) {
    if (tid == 0) {
      __threadfence();
      p.free_state[kStateArrived] = 0;
      p.free_state[kStateUsed] = start;
      p.free_state[kStateTaken] = min(all.grow, p.F - start);
    }
    if (moved)
      for (int s = tid; s < p.S; s += kTbThreads) {
        p.free_state[kStateLens + s] = __ldg(p.q_lens + s);
        p.free_state[kStateLens + p.S + s] = __ldg(p.seq_lens + s);
      }
  }
}
}  // namespace

static size_t tables_smem(int S) { return 3 * ((size_t)S + 1) * sizeof(int); }

int run_page_tables(cudaStream_t stream, TablesParams p) {
  p.vec_out = (reinterpret_cast<uintptr_t>(p.page_indices) & 15u) == 0;
  const long long items = std::max<long long>(p.T, ((long long)p.PTW + kEntriesPerThread - 1) / kEntriesPerThread);
  const int grid = (int)std::max<long long>(1, std::min<long long>(2LL * sm_count(),
                                                                   (items + kTbThreads - 1) / kTbThreads));
  set_smem_attr_once(reinterpret_cast<const void*>(page_tables_kernel), (int)tables_smem(kTablesMaxRequests));
  DSA_LAUNCH_PDL(page_tables_kernel, dim3(grid), dim3(kTbThreads), tables_smem(p.S), stream, p);
  return DSA_OK;
}

}  // namespace dsa
