// Absorbed-MLA attention of requests that share a prefix, whose keys are read
// together for all of them. Per group of requests, and with rows (token, head):
//   S = Q K^T over 576 dims, online softmax, O += P V, V = the first 512 dims.
// The rows of a group are cut into tiles of 256, of any tokens and heads, since
// [T, H] rows lie one behind another. A tile's keys are a list of runs of up to
// 128: of the prefix, read through the page table of the group's first request,
// then of the own positions of each request that has rows in the tile, which the
// rows of others mask. Two runs, of one request or of two, make a key tile.
//
// Keys are fetched in boxes of min(page size, 64) rows. The shared part ends with the
// prefix's last whole box: the box of its end holds the first request's own rows as
// well, so every request reads that one from a page of its own.
//
// A cluster of four CTAs takes a row tile: CTA (c, r) = rank 2c + r has rows
// 128r .. of it, value columns 256c .. (128 rows of all 512 columns in fp32 would
// be the whole TMEM) and computes S for run c of a key tile, so that no
// product is computed twice; it gives its weights P to CTA (1 - c, r), which
// needs them for the other value columns, and the two agree on the rows' maxima.
// The MMAs are those of the pairs (c, 0), (c, 1): 256 rows, and either CTA
// fetches half of the keys' operands.
//
// Work: the key tiles of all row tiles in a row, dealt to the clusters in equal
// shares, wherever a share ends. A list that was divided leaves its parts in the
// workspace (at most two per cluster) and a second kernel merges them, in order,
// so outputs are the same on every run.
//
// A request's own values are added to its own rows alone (the MMA leaves the others
// of the tile as they are): their weights are zero, but 0 x NaN is not.
//
// Roles of a CTA: warp 0 issues the MMAs (r = 0), warp 1 copies queries and keys,
// warp 2 resolves the keys a few tiles ahead, warp 3 passes on that the other half's
// P has arrived, warps 4-11 run the softmax, a row and half of its columns of S per
// thread.
//
// Per key tile i: QK^T(i), then PV(i - 1). S is read into registers at once and P
// goes to shared memory, so that QK^T(i + 1) runs beside the softmax of tile i.
//
// What bounds it: the tensor pipe, 4352 clocks per key tile of 256 rows x 256 keys,
// with shared memory next to it (per CTA about 512 KB in and out, 4000 clocks). A key
// tile takes 2.84 us, and 36 clusters run at once: 1.81 PFLOP/s, 94 % of the card's
// measured rate. Another 20 us a call is not products: the plan 4-5, the first
// queries and keys 5, the last outputs 5, the merge 7. Measured on 32 requests x 16384
// shared keys, 128 heads (109 us in all, floor 77), step by step: pairs whose CTAs
// compute S twice 161, clusters that share it 131, PV in order of arrival of P 127, the
// plan's lengths in shared memory 121, keys resolved by a warp of their own 114,
// runs of 128 keys 112. Elsewhere: 64 requests x 32768 keys of 16 heads 81 us (39: the
// own keys of 16 requests in a row tile are each computed for all of its rows), 4 x
// 131072 keys of 128 heads 110 (77), ragged extends of 500 tokens 118 (78), two short
// requests 17 (latency).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "prefix.cuh"

namespace dsa {

namespace {
constexpr int kDk = 576, kDv = 512;
constexpr int kRows = 128, kTileRows = 2 * kRows;  // of a CTA, of a cluster
constexpr int kRun = 128;                          // keys of a run, of which a key tile has two
constexpr int kBlk = 64 * 128;                     // 64 keys x 64 dims
constexpr int kQBlk = kRows * 128;                 // 128 rows x 64 dims (queries) or keys (P)
// Stages of a key tile: five of two K blocks (64 keys of this CTA, dims 64j and
// 256 + 64j; the last has dims 512 alone), then four of V (64 keys, 128 dims of this
// CTA), first the keys whose P this CTA computes. Before a list that is not a
// cluster's first, four of queries for TMEM (128 rows x 64 dims).
constexpr int kStages = 5, kStage = 2 * kBlk;
constexpr int kKStages = 5, kVStages = 4, kQStages = 4;
constexpr int kDescs = 4;
constexpr int kSoftWarps = 8;
constexpr int kThreads = (4 + kSoftWarps) * 32;
// Registers a thread: the softmax holds 64 logits. All together are what the CTA is
// launched with; 104 and 200 took 1 % longer, 168 for all spills (2 %).
constexpr int kHelperRegs = 136, kSoftRegs = 184;
constexpr int kLaunchRegs = (kHelperRegs + kSoftWarps / 4 * kSoftRegs) / (1 + kSoftWarps / 4);
static_assert(kLaunchRegs * (1 + kSoftWarps / 4) == kHelperRegs + kSoftWarps / 4 * kSoftRegs, "registers");
constexpr float kRescaleThreshold = 8.f;  // log2 units: p stays <= 256
constexpr int kNoRow = -64;               // a box from here on lies outside the cache and lands as zeros

// the k lowest bits
__device__ __forceinline__ uint32_t below(int k) { return k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1u; }

// What the softmax, the copier and the MMA issuer know of a key tile's runs.
struct KeyRun {
  int row[4];  // cache rows of keys 0, 32, 64 and 96, or kNoRow
  int pos;     // of the first key
  int seg;     // -1: prefix; else the request whose own keys they are
  int valid;   // bit g: keys 32 g .. hold positions
  int rows;    // the tile's rows a .. b - 1 that may see them: a | b << 16
};
constexpr int kAllRows = kTileRows << 16;
struct KeyTile {
  KeyRun run[2];
};

constexpr int OFF_Q = 0;  // dims 256-575
// four blocks of 64 keys; before, the first list's queries for TMEM: dims 0-255
constexpr int OFF_P = OFF_Q + 5 * kQBlk;
constexpr int OFF_RING = OFF_P + 4 * kQBlk;
constexpr int OFF_LOCAL = OFF_RING + kStages * kStage;   // float [2][kRows]: maxima of the two halves of S's columns
constexpr int OFF_REMOTE = OFF_LOCAL + 2 * kRows * 4;    // float [2][kRows]: those of the other keys, two tiles
constexpr int OFF_DESC = OFF_REMOTE + 2 * kRows * 4;
constexpr int OFF_BAR = (OFF_DESC + kDescs * (int)sizeof(KeyTile) + 7) & ~7;
constexpr int kNumBars = 2 * kStages + 2 * kDescs + 9 + 4 + 8;
constexpr int OFF_MISC = OFF_BAR + kNumBars * 8;
constexpr int kSmem = OFF_MISC + 16;  // TMEM address, abort flag
static_assert(kSmem <= 227 * 1024, "shared memory");
static_assert(kQBlk <= kStage, "queries in a stage");
static_assert(OFF_P % 1024 == 0 && OFF_RING % 1024 == 0 && OFF_DESC % 16 == 0, "alignment");

constexpr uint32_t kIdescQK = make_idesc_bf16(kTileRows, 128, false, false);
constexpr uint32_t kIdescPV = make_idesc_bf16(kTileRows, 256, false, true);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColQ = 256, kColS = 384;

struct Bars {
  uint64_t* b;
  // the pair's first CTA's: both CTAs' copies
  __device__ __forceinline__ uint64_t* full(int s) const { return b + s; }
  // each CTA's: commits of its pair
  __device__ __forceinline__ uint64_t* empty(int s) const { return b + kStages + s; }
  // each CTA's: key tiles resolved, and read
  __device__ __forceinline__ uint64_t* dfull(int s) const { return b + 2 * kStages + s; }
  __device__ __forceinline__ uint64_t* dempty(int s) const { return b + 2 * kStages + kDescs + s; }
  __device__ __forceinline__ uint64_t* rest(int k) const { return b + 2 * kStages + 2 * kDescs + k; }
  __device__ __forceinline__ uint64_t* sfull() const { return rest(0); }   // each: commit of its pair
  __device__ __forceinline__ uint64_t* pvdone() const { return rest(1); }  // each: commits of both pairs
  __device__ __forceinline__ uint64_t* sempty() const { return rest(2); }  // pair's: softmax warps of both CTAs
  __device__ __forceinline__ uint64_t* pfull() const { return rest(3); }   // pair's: softmax warps of both CTAs
  __device__ __forceinline__ uint64_t* qready() const { return rest(4); }  // pair's: softmax warps of both CTAs
  __device__ __forceinline__ uint64_t* qbar() const { return rest(5); }    // each: the queries' copies
  __device__ __forceinline__ uint64_t* ppeer() const { return rest(6); }   // each: P from the other half
  __device__ __forceinline__ uint64_t* lbar() const { return rest(7); }    // each: sums of weights from the other half
  __device__ __forceinline__ uint64_t* pother() const { return rest(8); }  // pair's: P of the other half, both CTAs
  __device__ __forceinline__ uint64_t* local(int w) const { return rest(9 + w); }  // each: two warps of the same rows
  // each: those two and the maxima of the other half
  __device__ __forceinline__ uint64_t* remote(int w, int k) const { return rest(13 + 4 * k + w); }
};

// ------------------------------------------------------------- the work list
// Request s's own keys for rows of tokens up to `last`: from position `start` (the
// end of what is shared) to `end`.
struct Own {
  int start, end;
  __device__ __forceinline__ int runs() const { return end > start ? (end - start + kRun - 1) / kRun : 0; }
};
__device__ __forceinline__ Own own_keys(const PrefixParams& p, int q0, int q1, int seq_len, int last, int prefix) {
  Own w{0, 0};
  if (q1 <= q0 || last < q0) return w;
  const int kv = min(max(seq_len, 0), p.max_kv);
  const int end = min(kv, kv - (q1 - q0) + min(last, q1 - 1) - q0 + 1);
  if (end > prefix) w.start = prefix, w.end = end;
  return w;
}

constexpr int kPlanThreads = 512;
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  // inclusive, of one value per thread
  const int lane = lane_id(), w = warp_id();
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += y;
  }
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  int x = lane < kPlanThreads / 32 ? warp_sums[lane] : 0;
  total = __reduce_add_sync(0xffffffffu, x);
  v += __reduce_add_sync(0xffffffffu, lane < w ? x : 0);
  __syncthreads();
  return v;
}

// One CTA lays out the row tiles, counts their key tiles, a warp per row tile and
// a lane per request, and deals them out. What is read many times, or by other
// threads than wrote it, waits in shared memory, if it fits.
constexpr int kPlanRequests = 3000, kPlanGroups = 512, kPlanTiles = 1024, kPlanCopies = 128;
// A list that starts inside a share costs about as much as this many key tiles: the
// pipeline runs empty, the next queries are fetched, the outputs written.
// 3 / 2 / 1 take 109.2 / 108.9 / 111.1 us on the 32 x 16384 keys and 49.1 / 47.4 / 47.2
// on five groups of unlike size.
constexpr int kListCost = 2;
constexpr int kMaxShares = 128;
struct PlanGroup {
  int first_tile, a, b, prefix, page_base;  // requests [a, b), none if it is refused
};
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PrefixParams p) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ int warp_sums[kPlanThreads / 32];
  __shared__ int32_t s_cu_q[kPlanRequests + 1], s_seq[kPlanRequests];
  __shared__ PlanGroup s_group[kPlanGroups];
  __shared__ int s_cost[kListCost + 1], s_begin[kListCost + 1][kMaxShares + 1], s_tile[kListCost + 1][kMaxShares + 1];
  __shared__ int s_base[kPlanTiles + 1];  // unit_base
  __shared__ PrefixTile s_tile_copy[kPlanCopies];
  const int tid = threadIdx.x, lane = lane_id();
  const int32_t *cu_q = p.cu_q_lens, *seq = p.seq_lens;
  int bad = 0;
  // A group's requests [a, b) as they are given, its prefix and the page-table place
  // of its first request; whether its requests are in order.
  struct Given {
    int a, b, want, place;
    bool ok;
  };
  auto given = [&](int g) -> Given {
    Given x;
    x.want = __ldg(p.prefix_lens + g);
    x.a = p.group_offsets ? __ldg(p.group_offsets + g) : 0;
    x.b = p.group_offsets ? __ldg(p.group_offsets + g + 1) : p.S;
    x.ok = x.a >= 0 && x.b >= x.a && x.b <= p.S && (g > 0 || x.a == 0);
    x.place = x.ok && x.b > x.a ? __ldg(p.cu_kv_lens + x.a) : 0;
    return x;
  };
  auto group_of = [&](const Given& in, bool& ok) -> PlanGroup {
    PlanGroup x{0, 0, 0, 0, 0};
    ok = in.ok;
    if (ok && in.b > in.a) {
      x.page_base = in.place / p.ps;
      x.prefix = min(max(in.want, 0), min(max(seq[in.a], 0), p.max_kv));
      ok = cu_q[in.a] >= 0 && cu_q[in.b] >= cu_q[in.a] && cu_q[in.b] <= p.T;
      if (ok) x.a = in.a, x.b = in.b;
      if (in.want != x.prefix) bad = 1;
      x.prefix &= -min(p.ps, 64);  // whole boxes
    }
    return x;
  };
  // the first groups' loads beside the requests'
  Given early{};
  if (tid < 256 && tid < p.G) early = given(tid);
  bool down = false;
  if (p.S <= kPlanRequests) {
    for (int i = tid; i < p.S; i += kPlanThreads) {
      const int q0 = __ldg(p.cu_q_lens + i), q1 = __ldg(p.cu_q_lens + i + 1), n = __ldg(p.seq_lens + i);
      s_cu_q[i] = q0;
      if (i == p.S - 1) s_cu_q[p.S] = q1;
      s_seq[i] = n;
      down |= q1 < q0;
    }
    cu_q = s_cu_q;
    seq = s_seq;
  } else {
#pragma unroll 1
    for (int i = tid; i < p.S; i += kPlanThreads) down |= __ldg(p.cu_q_lens + i + 1) < __ldg(p.cu_q_lens + i);
  }
  if (tid <= kListCost) s_cost[tid] = 0;
  const bool descents = __syncthreads_or(down);
  int total;
  unsigned tiles = 0;
  // 256 groups at a time: whatever the metadata hold, their sum fits 32 bits
  for (int g0 = 0; g0 < p.G; g0 += 256) {
    const int g = g0 + tid;
    unsigned n = 0;
    PlanGroup x{};
    const bool mine = tid < 256 && g < p.G;
    if (mine) {
      bool ok;
      const Given in = g0 ? given(g) : early;
      x = group_of(in, ok);
#pragma unroll 1
      for (int s = x.a; descents && s < x.b; ++s)
        if (cu_q[s] > cu_q[s + 1]) ok = false, x.b = x.a;
      // requests behind the last group: no rows of theirs are written
      if (!ok || (g == p.G - 1 && in.b != p.S)) bad = 1;
      n = ((unsigned)(cu_q[x.b] - cu_q[x.a]) * p.H + kTileRows - 1) / kTileRows;
    }
    const unsigned end = block_scan(n, warp_sums, total);
    if (mine) {
      x.first_tile = (int)min(tiles + end - n, (unsigned)p.max_tiles);
      if (p.G <= kPlanGroups) s_group[g] = x;
      else p.tile_base[g] = x.first_tile;
    }
    tiles = min(tiles + (unsigned)total, (unsigned)p.max_tiles + 1u);
  }
  if (tiles > (unsigned)p.max_tiles) bad = 1;
  const int ntiles = (int)min(tiles, (unsigned)p.max_tiles);
  int* base = ntiles <= kPlanTiles ? s_base : p.unit_base;
  __syncthreads();
  for (int i = warp_id(); i < ntiles; i += kPlanThreads / 32) {
    int lo = 0, hi = p.G - 1;  // the group with first_tile <= i, the last such one: not empty
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((p.G <= kPlanGroups ? s_group[mid].first_tile : p.tile_base[mid]) <= i) lo = mid;
      else hi = mid - 1;
    }
    PlanGroup x;
    if (p.G <= kPlanGroups) {
      x = s_group[lo];
    } else {
      bool ok;
      x = group_of(given(lo), ok);  // in order, as it has tiles
      x.first_tile = p.tile_base[lo];
    }
    const int first = cu_q[x.a] * p.H + (i - x.first_tile) * kTileRows, rows = min(kTileRows, cu_q[x.b] * p.H - first);
    const int ta = first / p.H, tb = (first + rows - 1) / p.H;
    int s0 = x.a, top = x.b;  // the request of token ta: offsets of other groups may be in any order
    while (top - s0 > 1) {
      const int mid = (s0 + top) >> 1;
      if (cu_q[mid] <= ta) s0 = mid;
      else top = mid;
    }
    int n = 0;
    for (int b = s0; b < x.b; b += 32) {
      const int s = b + lane;
      const bool in = s < x.b && cu_q[s] <= tb;
      if (in) n += own_keys(p, cu_q[s], cu_q[s + 1], seq[s], tb, x.prefix).runs();
      if (!__all_sync(0xffffffffu, in)) break;
    }
    n = (__reduce_add_sync(0xffffffffu, n) + (x.prefix + kRun - 1) / kRun + 1) / 2;
    if (lane == 0) {
      // rows without any key still have an output; no more than ordered metadata give
      base[i] = n < 0 ? p.max_units : min(max(n, 1), p.max_units);
      PrefixTile r{};
      r.row0 = first;
      r.rows = rows;
      r.s0 = s0;
      r.s1 = x.b;
      r.last = tb;
      r.prefix = x.prefix;
      r.page_base = x.page_base;
      p.tiles[i] = r;
      if (i < kPlanCopies) s_tile_copy[i] = r;
    }
  }
  __syncthreads();
  int units = 0;
  for (int i0 = 0; i0 < ntiles; i0 += kPlanThreads) {
    const int i = i0 + tid;
    const int n = i < ntiles ? base[i] : 0, end = block_scan(n, warp_sums, total);
    if (i < ntiles) {
      base[i] = units + end - n;
      p.tiles[i].begin = units + end - n;
      p.tiles[i].end = units + end;
    }
    units += total;
  }
  if (tid == 0) base[ntiles] = units;
  __syncthreads();
  // The shares are equal runs of the lists with `gap` units of no work between
  // two of them, so that a share in which a list starts has less work; of the
  // gaps up to the cost of a start, the one with which the costliest share costs
  // least. A share is longer than the gap, so none is empty.
  const int n = min(p.shares, units), gaps = n ? min(kListCost, units / n - 1) + 1 : 0;
  for (int j = tid; j < gaps * (n + 1); j += kPlanThreads) {
    const int gap = j / (n + 1), k = j % (n + 1), all = units + gap * (ntiles - 1);
    const int v = all / n * k + all % n * k / n;  // all * k / n
    int lo = 0, hi = ntiles - 1;                  // the tile that holds v, from the gap before it on
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (base[mid] + gap * (mid - 1) <= v) lo = mid;
      else hi = mid - 1;
    }
    s_begin[gap][k] = k < n ? base[lo] + max(0, v - base[lo] - gap * lo) : units;
    s_tile[gap][k] = k < n ? lo : ntiles;
  }
  __syncthreads();
  for (int j = tid; j < gaps * n; j += kPlanThreads) {
    const int gap = j / n, k = j % n, e = s_begin[gap][k + 1], t = s_tile[gap][k + 1];
    const int starts = (e == base[t] ? t - 1 : t) - s_tile[gap][k];  // lists that start behind the share's begin
    atomicMax(s_cost + gap, e - s_begin[gap][k] + kListCost * starts);
  }
  __syncthreads();
  int gap = 0;
  for (int j = 1; j < gaps; ++j) gap = s_cost[j] < s_cost[gap] ? j : gap;
  for (int k = tid; k < p.shares; k += kPlanThreads) {
    PrefixShare r{};
    if (k < n) {
      auto copy_of = [&](int i) { return i < kPlanCopies ? s_tile_copy[i] : p.tiles[i]; };
      const int *sb = s_begin[gap], next = s_tile[gap][k + 1];
      r.begin = sb[k];
      r.end = sb[k + 1];
      r.tile = s_tile[gap][k];
      r.first = copy_of(r.tile);
      r.first.begin = base[r.tile];
      r.first.end = base[r.tile + 1];
      if (base[next] < r.end && r.begin <= base[next]) {
        const PrefixTile cut = copy_of(next);
        r.cut_row0 = cut.row0;
        r.cut_rows = cut.rows;
        r.first_slot = r.begin == base[next] ? 2 * k : 2 * k + 1;
        r.last = k + 1;  // the last share that begins inside the list
        while (r.last + 1 < n && sb[r.last + 1] < base[next + 1]) ++r.last;
      }
    }
    p.share[k] = r;
  }
  if (bad) set_status(p.dev_status, DSA_STATUS_BAD_METADATA);
}

// The runs of a list from run k on, resolved by one whole warp.
struct KeyCursor {
  const PrefixParams* p;
  int prefix, s1, seg;  // the group's end; the segment (-1: prefix)
  int s, own_start, own_end, own_base;  // 32 requests from s on, one per lane: their own keys and page-table entries
  uint32_t todo;                        // those with own keys still to visit
  int pos, end, left, page_base, lg;
  int win, page;  // first entry of the window of pages, this lane's page in it (-1: none)
  int row0, last, H;   // the tile's first row and last token; heads
  int rows, own_rows;  // rows that see the segment, and each lane's request

  __device__ __forceinline__ void open(int sg, int first, int stop, int runs, int base, int who) {
    seg = sg;
    pos = first;
    end = stop;
    left = runs;
    page_base = base;
    rows = who;
    win = -64;
  }
  __device__ void init(const PrefixParams& prm, const PrefixTile& tile, int k) {
    p = &prm;
    lg = 31 - __clz(prm.ps);
    prefix = tile.prefix;
    row0 = tile.row0;
    H = prm.H;
    last = tile.last;
    s1 = tile.s1;
    s = tile.s0 - 32;
    todo = 0;
    left = 0;
    const int np = (prefix + kRun - 1) / kRun;
    if (k < np) {
      open(-1, k * kRun, prefix, np - k, tile.page_base, kAllRows);
    } else {
      next_request(k - np);
    }
  }
  // the request that holds own run k of those still to visit
  __device__ void next_request(int k) {
    while (true) {
      if (todo) {
        const int n = todo >> lane_id() & 1 ? Own{own_start, own_end}.runs() : 0;
        int upto = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane_id() >= d) upto += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, upto > k);
        if (past) {
          const int l = __ffs(past) - 1;
          k -= __shfl_sync(0xffffffffu, upto - n, l);
          open(s + l, __shfl_sync(0xffffffffu, own_start, l) + k * kRun, __shfl_sync(0xffffffffu, own_end, l),
               __shfl_sync(0xffffffffu, n, l) - k, __shfl_sync(0xffffffffu, own_base, l),
               __shfl_sync(0xffffffffu, own_rows, l));
          todo &= 0xfffffffeu << l;
          return;
        }
        k -= __shfl_sync(0xffffffffu, upto, 31);
      }
      s += 32;
      const int me = s + lane_id();
      const int q0 = me < s1 ? __ldg(p->cu_q_lens + me) : last + 1;
      todo = 0;
      if (!__any_sync(0xffffffffu, q0 <= last)) break;
      Own w{0, 0};
      if (q0 <= last) {
        const int q1 = __ldg(p->cu_q_lens + me + 1);
        w = own_keys(*p, q0, q1, __ldg(p->seq_lens + me), last, prefix);
        // rows of [T * H] fit 31 bits, those of other tiles lie outside 0 .. 256
        own_rows = min(max(q0 * H - row0, 0), kTileRows) | min(max(q1 * H - row0, 0), kTileRows) << 16;
        own_base = __ldg(p->cu_kv_lens + me) >> lg;
      }
      own_start = w.start;
      own_end = w.end;
      todo = __ballot_sync(0xffffffffu, w.runs() > 0);
    }
    seg = p->S;  // no keys: behind the last run
    rows = kAllRows;
    pos = end = 0;
    left = 1;
    win = 0;
    page = -1;
  }
  // The next run, in every lane.
  __device__ KeyRun next() {
    if (!left) next_request(0);
    --left;
    KeyRun t;
    t.pos = pos;
    t.seg = seg;
    t.valid = 0;
    t.rows = rows;
    const int e0 = pos >> lg;
    if (pos < end && (e0 < win || ((pos + kRun - 1) >> lg) >= win + 32)) {
      win = e0;
      const int e = win + lane_id();
      page = -1;
      if ((long long)e << lg < end) {
        const long long ent = (long long)page_base + e;
        if (ent < 0 || ent >= p->PTW) {
          set_status(p->dev_status, DSA_STATUS_BAD_METADATA);
        } else {
          page = __ldg(p->page_indices + ent);
          if (page < 0 || page >= p->P) {
            set_status(p->dev_status, DSA_STATUS_BAD_METADATA);
            page = -1;
          }
        }
      }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int at = pos + 32 * g, pg = __shfl_sync(0xffffffffu, page, ((at >> lg) - win) & 31);
      const bool ok = at < end && pg >= 0;
      t.row[g] = ok ? (pg << lg) + (at & (p->ps - 1)) : kNoRow;
      t.valid |= ok ? 1 << g : 0;
    }
    pos += kRun;
    return t;
  }
};

// 64 keys x 64 dims as boxes of min(ps, 64) rows.
__device__ __forceinline__ void copy_block(uint32_t dst, const CUtensorMap* map, uint32_t bar, int dim, int r0, int r1,
                                           bool two) {
  tma_load_2d_pair(dst, map, bar, dim, r0);
  if (two) tma_load_2d_pair(dst + kBlk / 2, map, bar, dim, r1);
}

__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(kThreads, 1)
    prefix_mla_kernel(const __grid_constant__ PrefixParams prm, const __grid_constant__ CUtensorMap kvmap,
                      const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // in every CTA alike
    if (threadIdx.x == 0) set_status(prm.dev_status, DSA_STATUS_INTERNAL);
    return;
  }
  griddep_launch_dependents();
  const int warp = warp_id(), lane = lane_id(), tid = threadIdx.x;
  const int rank = (int)cluster_rank(), c = rank >> 1, r = rank & 1, share = blockIdx.x >> 2;
  const uint32_t smem0 = smem_u32(smem);
  const Bars br{reinterpret_cast<uint64_t*>(smem + OFF_BAR)};
  KeyTile* descs = reinterpret_cast<KeyTile*>(smem + OFF_DESC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(br.full(s), 1), mbar_init(br.empty(s), 1);
    for (int s = 0; s < kDescs; ++s) mbar_init(br.dfull(s), 1), mbar_init(br.dempty(s), kSoftWarps + 1 + (r == 0));
    mbar_init(br.sfull(), 1);
    mbar_init(br.pvdone(), 2);
    mbar_init(br.sempty(), 2 * kSoftWarps);
    mbar_init(br.pfull(), 2 * kSoftWarps);
    mbar_init(br.pother(), 2);
    mbar_init(br.qready(), 2 * kSoftWarps);
    mbar_init(br.qbar(), 1);
    mbar_init(br.ppeer(), 1);
    mbar_init(br.lbar(), kSoftWarps);
    for (int w = 0; w < 4; ++w) {
      mbar_init(br.local(w), 2);
      for (int k = 0; k < 2; ++k) mbar_init(br.remote(w, k), 2);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();
  tc_fence_after();
  griddep_wait();
  const uint32_t tmem = *tmem_slot;
  const PrefixShare work = prm.share[share];
  auto leader = [&](uint64_t* bar) { return cluster_addr(smem_u32(bar), rank & 2); };  // of the pair
  auto other = [&](uint32_t a) { return cluster_addr(a, rank ^ 2); };  // CTA (1 - c, r)
  // a role that gives up tells all CTAs
  auto give_up = [&]() {
    if (lane < 4) st_cluster_u32(cluster_addr(smem_u32(const_cast<int*>(abort_flag)), lane), 1);
    __syncwarp();
  };
  // every role counts what it has passed since the kernel began: a barrier's
  // phase is that number's parity
  uint32_t tc = 0, uc = 0, fc = 0;  // key tiles, lists, stages
  // a softmax thread's row of a tile: its request and visible positions
  auto row_of = [&](const PrefixTile& tile) -> int2 {
    const int row = (warp & 3) * 32 + lane;
    if (row >= tile.rows - r * kRows) return make_int2(-2, 0);
    const int t = (tile.row0 + r * kRows + row) / prm.H;
    int s = tile.s0, top = tile.s1;  // cu_q_lens[s] <= t < cu_q_lens[top]
    for (int step = 1; s + step < top; step *= 2) {
      if (__ldg(prm.cu_q_lens + s + step) > t) top = s + step;
      else s += step;
    }
    while (top - s > 1) {
      const int mid = (s + top) >> 1;
      if (__ldg(prm.cu_q_lens + mid) > t) top = mid;
      else s = mid;
    }
    const TokenGeom g = token_geom(prm.seq_lens, prm.cu_q_lens, prm.cu_kv_lens, prm.S, prm.ps, prm.max_kv, t,
                                   prm.dev_status, s);
    return make_int2(s, g.n_vis);
  };
  auto lists = [&](auto softmax) {
    constexpr bool kSoft = decltype(softmax)::value;
    int ti = work.tile;
    PrefixTile tile{};
    int2 mine{};  // my row of the tile
    if (work.begin < work.end) {
      tile = work.first;
      if constexpr (kSoft) mine = row_of(tile);
    }
    bool ok = true;
#pragma unroll 1
    for (int u = work.begin; ok && u < work.end; ++ti) {
      const int list0 = tile.begin, list1 = tile.end;  // the list's units
      const int k0 = u - list0, n = min(work.end, list1) - u;
      const bool whole = k0 == 0 && u + n == list1;
      const int slot_out = u == work.begin ? 2 * share : 2 * share + 1;
      const uint32_t from = fc;  // the first stage; from the second list on those of the queries for TMEM
      if (uc) fc += kQStages;
      const int row0 = tile.row0 + r * kRows;              // this CTA's first row of [T * H]
      const int rows = min(kRows, tile.rows - r * kRows);  // <= 0: none
      if constexpr (!kSoft) {
        if (warp == 0) {
          // -------------------------------------------------------- MMA issuer
          if (r == 0) {
            const uint32_t lead = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint64_t dq = make_sdesc(smem0 + OFF_Q, 16, 1024, kSwizzle128B);
            const uint64_t dp = make_sdesc(smem0 + OFF_P, 16, 1024, kSwizzle128B);
            const uint64_t dk = make_sdesc(smem0 + OFF_RING, 16, 1024, kSwizzle128B);
            const uint64_t dv = make_sdesc(smem0 + OFF_RING, kBlk, 1024, kSwizzle128B);  // MN-major
            const uint16_t pair = (uint16_t)(3 << rank);
            auto commit = [&](uint64_t* bar, uint16_t to) {
              if (lead) umma_commit_pair(bar, to);
              __syncwarp();
            };
            uint32_t slot = from % kStages, phase = (from / kStages) & 1;
            auto arrived = [&]() { return mbar_wait_warp(br.full(slot), phase, abort_flag); };
            auto pass = [&]() {
              commit(br.empty(slot), pair);
              if (++slot == kStages) slot = 0, phase ^= 1;
            };
            const int prefix_runs = (tile.prefix + kRun - 1) / kRun;
            ok = mbar_wait_warp_cluster(br.qready(), uc & 1, abort_flag);
            tc_fence_after();
            for (uint32_t j = from; j != fc; ++j) pass();  // the queries' stages have been read
#pragma unroll 1
            for (int i = 0; ok && i <= n; ++i) {
              // small loops: the roles share the instruction cache
              if (i < n) {
                // S is free once the tile before has been read into registers
                if (!(ok = mbar_wait_warp_cluster(br.sempty(), (tc & 1) ^ 1, abort_flag))) break;
                tc_fence_after();
                // queries in TMEM and in shared memory by turns: the latter's reads and
                // the copies into shared memory together are near its bandwidth
#pragma unroll 1
                for (int j = 0; j < kKStages; ++j) {
                  if (!(ok = arrived())) break;
                  const uint64_t kb = dk + (uint64_t)(slot * (kStage >> 4)), qb = dq + (uint64_t)(j * (kQBlk >> 4));
                  if (j < 4) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                      umma_pair_ts_lead(lead, tm + kColS, tm + kColQ + j * 32 + k * 8, kb + k * 2, kIdescQK,
                                        j || k ? 1u : 0u);
                      umma_pair_ss_lead(lead, tm + kColS, qb + k * 2, kb + (kBlk >> 4) + k * 2, kIdescQK, 1u);
                    }
                  } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                      umma_pair_ss_lead(lead, tm + kColS, qb + k * 2, kb + k * 2, kIdescQK, 1u);
                  }
                  pass();
                }
                if (!ok) break;
                commit(br.sfull(), pair);
                ++tc;
              }
              if (i > 0) {
                // the keys whose P was computed here, then those whose P comes from
                // the other half, which takes longer
                const uint32_t pv = tc - (i < n ? 2 : 1), parity = pv & 1;
                auto weighted = [&](auto half, auto product) {
#pragma unroll 1
                  for (int s = 0; s < kVStages; ++s) {
                    if (!(s & 1)) {
                      if (!(ok = mbar_wait_warp_cluster(s ? br.pother() : br.pfull(), parity, abort_flag))) break;
                      tc_fence_after();
                      half(s >> 1);
                    }
                    if (!(ok = arrived())) break;
                    const uint64_t vb = dv + (uint64_t)(slot * (kStage >> 4));
                    const uint64_t pb = dp + (uint64_t)(((rank + s) & 3) * (kQBlk >> 4));  // rank = 2c
#pragma unroll
                    for (int k = 0; k < 4; ++k) product(pb + k * 2, vb + k * 128);
                    pass();
                  }
                };
                if (2 * (k0 + i) <= prefix_runs) {
                  weighted([](int) {},
                           [&](uint64_t pb, uint64_t vb) {
                             umma_pair_ss_lead(lead, tm + kColO, pb, vb, kIdescPV, 1u);
                           });
                } else {
                  // Own keys: other requests' weights of them are zero, but zero times an
                  // infinity or a NaN among the values would reach those rows.
                  const KeyTile& keys = descs[pv % kDescs];
                  if (!(ok = mbar_wait_warp(br.dfull(pv % kDescs), (pv / kDescs) & 1, abort_flag))) break;
                  uint32_t off[2][8];
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    const int who = keys.run[c ^ x].rows, a = who & 0xffff, b = who >> 16;
#pragma unroll
                    for (int g = 0; g < 8; ++g)
                      off[x][g] = __ballot_sync(0xffffffffu, (unsigned)(32 * g + lane - a) >= (unsigned)(b - a));
                  }
                  uint32_t now[8];
                  weighted(
                      [&](int x) {
#pragma unroll
                        for (int g = 0; g < 8; ++g) now[g] = x ? off[1][g] : off[0][g];
                      },
                      [&](uint64_t pb, uint64_t vb) {
                        umma_pair_ss_rows_lead(lead, tm + kColO, pb, vb, kIdescPV, now);
                      });
                }
                if (!ok) break;
                if (lane == 0) mbar_arrive(br.dempty(pv % kDescs));
                __syncwarp();
                commit(br.pvdone(), 15);
              }
            }
            if (!ok) give_up();
          }
        } else if (warp == 1) {
          // ---------------------------------------------------- queries and keys
          // Query blocks: those for TMEM land in P's places, of later lists in stages
          // of the ring, the others where they stay, free once the last QK^T has run.
          uint32_t slot = from % kStages, phase = (from / kStages) & 1;
          if (uc) ok = mbar_wait_warp(br.sfull(), (tc - 1) & 1, abort_flag);
          if (ok && lane == 0) {
            mbar_arrive_expect_tx(br.qbar(), 9 * kQBlk);
#pragma unroll 1
            for (int b = uc ? kQStages : 0; b < 9; ++b)
              tma_load_2d(smem + (b < 4 ? OFF_P + b * kQBlk : OFF_Q + (b - 4) * kQBlk), &qmap, br.qbar(), b * 64,
                          row0);
          }
          __syncwarp();
#pragma unroll 1
          for (int b = 0; ok && uc && b < kQStages; ++b) {
            if (!(ok = mbar_wait_warp(br.empty(slot), phase ^ 1, abort_flag))) break;
            if (lane == 0) {
              if (r == 0) mbar_arrive(br.full(slot));  // keeps its phases; nobody waits for this one
              tma_load_2d(smem + OFF_RING + slot * kStage, &qmap, br.qbar(), b * 64, row0);
            }
            __syncwarp();
            if (++slot == kStages) slot = 0, phase ^= 1;
          }
          const bool two = prm.ps == 32;
          // a stage of two blocks of 64 keys, dims d0 .. and d1 .. (one: only the first)
          auto load = [&](int d0, int d1, int r0, int r1, bool one) -> bool {
            if (!mbar_wait_warp(br.empty(slot), phase ^ 1, abort_flag)) return false;
            if (lane == 0) {
              const uint32_t bar = leader(br.full(slot)), dst = smem0 + OFF_RING + slot * kStage;
              if (r == 0) mbar_arrive_expect_tx(br.full(slot), one ? kStage : 2 * kStage);
              copy_block(dst, &kvmap, bar, d0, r0, r1, two);
              if (!one) copy_block(dst + kBlk, &kvmap, bar, d1, r0, r1, two);
            }
            __syncwarp();
            if (++slot == kStages) slot = 0, phase ^= 1;
            return true;
          };
#pragma unroll 1
          for (int i = 0; ok && i <= n; ++i) {
            if (i < n) {
              const int ds = tc % kDescs;
              if (!(ok = mbar_wait_warp(br.dfull(ds), (tc / kDescs) & 1, abort_flag))) break;
              const KeyRun& mine = descs[ds].run[c];  // of which this CTA has 64 keys
              const int r0 = mine.row[2 * r], r1 = mine.row[2 * r + 1];
              ++tc;
#pragma unroll 1
              for (int j = 0; ok && j < kKStages; ++j)
                ok = j < 4 ? load(j * 64, 256 + j * 64, r0, r1, false) : load(512, 0, r0, r1, true);
              if (!ok) break;
            }
            if (i > 0) {  // V of the key tile before, first of run c
              const int ds = (tc - (i < n ? 2 : 1)) % kDescs;
#pragma unroll 1
              for (int s = 0; ok && s < kVStages; ++s) {
                const KeyRun& run = descs[ds].run[c ^ (s >> 1)];
                ok = load(c * 256 + r * 128, c * 256 + r * 128 + 64, run.row[2 * (s & 1)], run.row[2 * (s & 1) + 1],
                          false);
              }
              if (lane == 0) mbar_arrive(br.dempty(ds));
              __syncwarp();
            }
          }
          if (!ok) give_up();
        } else if (warp == 2) {
          // ----------------------------------------------------------- key tiles
          KeyCursor cur;
          cur.init(prm, tile, 2 * k0);
#pragma unroll 1
          for (int i = 0; i < n; ++i, ++tc) {
            const KeyRun run0 = cur.next(), run1 = cur.next();
            const int ds = tc % kDescs;
            if (!(ok = mbar_wait_warp(br.dempty(ds), ((tc / kDescs) & 1) ^ 1, abort_flag))) break;
            if (lane == 0) {
              descs[ds] = KeyTile{{run0, run1}};
              mbar_arrive(br.dfull(ds));
            }
            __syncwarp();
          }
          if (!ok) give_up();
        } else {
          // --------------------------- P of the other half, for the MMA issuer
          const uint32_t a_pother = leader(br.pother());
#pragma unroll 1
          for (int i = 0; i < n; ++i, ++tc) {
            if (lane == 0) mbar_arrive_expect_tx(br.ppeer(), 2 * kQBlk);
            if (!(ok = mbar_wait_warp(br.ppeer(), tc & 1, abort_flag))) break;
            if (lane == 0) mbar_arrive_cluster(a_pother);
            __syncwarp();
          }
          if (!ok) give_up();
        }
      } else {
        // ------------------------------------------------------------- softmax
        const int q = warp & 3, hh = (warp - 4) >> 2;  // 32 TMEM lanes (rows); half of S's columns
        const int row = q * 32 + lane;
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        const uint32_t a_sempty = leader(br.sempty()), a_pfull = leader(br.pfull());
        // this warp's part of P, 32 rows x 64 keys, here and at the other half
        const uint32_t p_blk = smem0 + OFF_P + (2 * c + hh) * kQBlk, p_run = p_blk + q * 32 * 128;
        const int my_s = mine.x, see = mine.y, prefix = tile.prefix;
        // The queries of list k for TMEM, from P's places or from the ring's stages from
        // `stage` on.
        auto take_queries = [&](uint32_t k, bool ring, uint32_t stage) {
          if (!(ok = mbar_wait_warp(br.qbar(), k & 1, abort_flag))) return;
#pragma unroll 1
          for (int b = 2 * hh; b < 2 * hh + 2; ++b) {
            const int at = ring ? OFF_RING + (int)((stage + b) % kStages) * kStage : OFF_P + b * kQBlk;
            const uint8_t* src = smem + at + row * 128;
            uint32_t v[32];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint4 x = *reinterpret_cast<const uint4*>(src + ((j ^ (row & 7)) << 4));
              v[4 * j] = x.x;
              v[4 * j + 1] = x.y;
              v[4 * j + 2] = x.z;
              v[4 * j + 3] = x.w;
            }
            tmem_st32(tmem + lane_base + kColQ + b * 32, v);
          }
          tmem_st_wait();
          tc_fence_before();
          // Bulk copies write here next: the other half's of P, of these 32 rows after it
          // has had this warp's maxima of the first tile, or keys.
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(leader(br.qready()));
          __syncwarp();
        };
        if (!uc) take_queries(0, false, 0);
        if (ok) {
          // PV adds to O from the first tile on, as a request's own keys do not reach all rows
          uint32_t zero[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) zero[j] = 0u;
#pragma unroll 1
          for (int k = 4 * hh; k < 4 * hh + 4; ++k) tmem_st32(tmem + lane_base + kColO + k * 32, zero);
          tmem_st_wait();
          tc_fence_before();
        }
        const float sl2 = prm.scale_log2;
        float m_run = -INFINITY, l_run = 0.f;  // l_run: of this thread's columns
        float* mx_local = reinterpret_cast<float*>(smem + OFF_LOCAL) + row;
#pragma unroll 1
        for (int i = 0; ok && i < n; ++i, ++tc) {
          const int ds = tc % kDescs;
          if (!(ok = mbar_wait_warp(br.dfull(ds), (tc / kDescs) & 1, abort_flag))) break;
          const KeyRun& run = descs[ds].run[c];
          const int p0 = run.pos + hh * 64, seg = run.seg, valid = run.valid >> (2 * hh);
          __syncwarp();
          if (lane == 0) mbar_arrive(br.dempty(ds));
          const int hi = (seg < 0 ? min(see, prefix) : seg == my_s ? see : 0) - p0;
          uint32_t mask[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) mask[g] = (valid >> g) & 1 ? below(hi - 32 * g) : 0u;
          const bool full = __all_sync(0xffffffffu, (mask[0] & mask[1]) == 0xffffffffu);
          if (!(ok = mbar_wait_warp(br.sfull(), tc & 1, abort_flag))) break;
          tc_fence_after();
          uint32_t s[2][32];
          tmem_ld32(tmem + lane_base + kColS + 64 * hh, s[0]);
          tmem_ld32(tmem + lane_base + kColS + 64 * hh + 32, s[1]);
          tmem_ld_wait_regs(s[0]);
          reg_fence(s[1]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(a_sempty);
          // scaled logits, those of masked keys -inf: they are left out of maximum
          // and weights, whatever they are
          const uint64_t sl22 = f32x2_pack(sl2, sl2);
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              float x0, x1;
              f32x2_unpack(fmul2(f32x2_pack(__uint_as_float(s[g][j]), __uint_as_float(s[g][j + 1])), sl22), x0, x1);
              s[g][j] = __float_as_uint(x0);
              s[g][j + 1] = __float_as_uint(x1);
            }
          if (!full) {
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
              for (int j = 0; j < 32; ++j) s[g][j] = (mask[g] >> j) & 1u ? s[g][j] : 0xff800000u;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int j = 0; j < 32; j += 2)
              mx[(j >> 1) & 3] = max3(mx[(j >> 1) & 3], __uint_as_float(s[g][j]), __uint_as_float(s[g][j + 1]));
          // The row's maximum over the tile: first with the warp of the other
          // columns, then one of the two tells the CTA of the other keys. The other
          // CTA sends tile i + 2's when PV(i) has run, so after this one has read
          // tile i's: two places are enough. One local place is: the second barrier
          // is passed when both warps have read. All waits have limits, which named
          // barriers' have not.
          mx_local[hh * kRows] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          __syncwarp();
          if (lane == 0) mbar_arrive(br.local(q));
          if (!(ok = mbar_wait_warp(br.local(q), tc & 1, abort_flag))) break;
          const float mine = fmaxf(mx_local[0], mx_local[kRows]);
          const uint32_t a_mx = smem0 + OFF_REMOTE + ((tc & 1) * kRows + row) * 4;
          uint64_t* rbar = br.remote(q, tc & 1);
          if (hh == 0) st_async_f32(other(a_mx), mine, other(smem_u32(rbar)));
          __syncwarp();
          if (lane == 0) {
            if (hh == 0) mbar_arrive_expect_tx(rbar, 32 * 4);
            else mbar_arrive(rbar);
          }
          if (!(ok = mbar_wait_warp(rbar, (tc >> 1) & 1, abort_flag))) break;
          const float m_new = max3(m_run, mine, *reinterpret_cast<volatile float*>(smem + (a_mx - smem0)));
          const bool need = m_new > m_run + kRescaleThreshold;  // also true when m_run == -inf
          const float m_use = need ? m_new : m_run;
          const float alpha = need ? exp2f(m_run - m_new) : 1.f;
          const float m_sub = m_use == -INFINITY ? 0.f : m_use;  // a row without keys so far: its weights are 2^-inf
          const uint64_t nm2 = f32x2_pack(-m_sub, -m_sub);
          uint64_t ps2[2] = {0ull, 0ull};
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float x0, x1;
              f32x2_unpack(fadd2(f32x2_pack(__uint_as_float(s[g][2 * k]), __uint_as_float(s[g][2 * k + 1])), nm2), x0,
                           x1);
              x0 = ex2_approx(x0);
              x1 = ex2_approx(x1);
              ps2[k & 1] = fadd2(ps2[k & 1], f32x2_pack(x0, x1));
              __nv_bfloat162 b2 = __floats2bfloat162_rn(x0, x1);  // P as a bf16 operand
              s[g][k] = *reinterpret_cast<uint32_t*>(&b2);
            }
          // P's places, here and at the other half, and O are free once both
          // pairs' PV of the tile before have run
          if (i > 0 && !(ok = mbar_wait_warp(br.pvdone(), (tc - 1) & 1, abort_flag))) break;
          if (i > 0 && __any_sync(0xffffffffu, need)) {
            tc_fence_after();
#pragma unroll 1
            for (int k = 4 * hh; k < 4 * hh + 4; ++k) {
              uint32_t ov[32];
              tmem_ld32(tmem + lane_base + kColO + k * 32, ov);
              tmem_ld_wait_regs(ov);
#pragma unroll
              for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
              tmem_st32(tmem + lane_base + kColO + k * 32, ov);
            }
            tmem_st_wait();
            tc_fence_before();
          }
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              st_shared_v4(p_blk + sw128_offset(row, g * 4 + k), s[g][4 * k], s[g][4 * k + 1], s[g][4 * k + 2],
                           s[g][4 * k + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            bulk_store_cluster(other(p_run), p_run, 32 * 128, other(smem_u32(br.ppeer())));
            mbar_arrive_cluster(a_pfull);
          }
          float pa, pb;
          f32x2_unpack(fadd2(ps2[0], ps2[1]), pa, pb);
          l_run = l_run * alpha + (pa + pb);
          m_run = m_use;
        }
        // ------------------------------------------------------------ epilogue
        if (ok && u + n < work.end) {  // while the last PV runs: the next list's row
          tile = prm.tiles[ti + 1];
          mine = row_of(tile);
        }
        ok = ok && mbar_wait_warp(br.pvdone(), (tc - 1) & 1, abort_flag);
        // P's places are idle now, on both sides. The sum of a row's weights comes in
        // four parts, to the start of this CTA's own; the other half's, of the rows
        // that the other CTA's warps of this number write, stage the outputs.
        if (ok) {
          const uint32_t a_l = OFF_P + 2 * c * kQBlk + ((2 * c + hh) * kRows + row) * 4;
          const uint32_t a_there = OFF_P + 2 * (1 - c) * kQBlk + ((2 * c + hh) * kRows + row) * 4;
          st_async_f32(other(smem0 + a_there), l_run, other(smem_u32(br.lbar())));
          *reinterpret_cast<float*>(smem + a_l) = l_run;
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(br.lbar(), 32 * 4);
          __syncwarp();
          ok = mbar_wait_warp(br.lbar(), uc & 1, abort_flag);
        }
        float l = 0.f;
        if (ok) {
          tc_fence_after();
          const volatile float* lp = reinterpret_cast<const volatile float*>(smem + OFF_P + 2 * c * kQBlk) + row;
          l = (lp[0] + lp[kRows]) + (lp[2 * kRows] + lp[3 * kRows]);
          // The next list's first QK^T runs while this one's outputs are written. The sums
          // have been read by then: its first P lands there.
          if (u + n < work.end) take_queries(uc + 1, true, fc + (kKStages + kVStages) * n);
        }
        if (ok) {
          const bool some = l != 0.f;  // a sum of weights is never negative; NaN counts
          const float inv_l = some ? 1.f / l : 0.f;
          const float lse2 = some ? m_run + log2f(l) : -INFINITY;
          // 128 bytes of 32 rows at a time, chunks of 16 bytes swizzled
          const int w0 = q * 32, nw = min(32, rows - w0);
          const uint32_t stg = smem0 + OFF_P + (2 * (1 - c) + hh) * kQBlk + w0 * 128;
          const uint32_t col = tmem + lane_base + kColO + 128 * hh;
          const size_t part_row = (size_t)slot_out * kTileRows + r * kRows + w0;  // or, undivided, the output's
          uint8_t* out = whole ? reinterpret_cast<uint8_t*>(prm.o + ((size_t)row0 + w0) * kDv + c * 256 + hh * 128)
                               : reinterpret_cast<uint8_t*>(prm.part_o + part_row * kDv + c * 256 + hh * 128);
          const size_t pitch = whole ? kDv * 2 : kDv * 4;
#pragma unroll 1
          for (int c0 = 0; c0 < 128; out += 128) {
            uint32_t o[32], v[32];
            tmem_ld32(col + c0, o);
            tmem_ld_wait_regs(o);
            if (whole) {
              auto pack = [&](int at) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[2 * j]) * inv_l,
                                                            __uint_as_float(o[2 * j + 1]) * inv_l);
                  v[at + j] = *reinterpret_cast<uint32_t*>(&b2);
                }
              };
              pack(0);
              tmem_ld32(col + c0 + 32, o);
              tmem_ld_wait_regs(o);
              pack(16);
              c0 += 64;
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(o[j]) * inv_l);
              c0 += 32;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
              st_shared_v4(stg + sw128_offset(lane, j), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int k = 4 * j + (lane >> 3);
              if (k < nw)
                *reinterpret_cast<uint4*>(out + k * pitch + (lane & 7) * 16) =
                    *reinterpret_cast<const uint4*>(smem + (stg - smem0) + sw128_offset(k, lane & 7));
            }
            __syncwarp();
          }
          if (c == 0 && hh == 0 && row < rows) {
            if (!whole) prm.part_lse[part_row + lane] = lse2;
            else if (prm.lse) prm.lse[(size_t)row0 + row] = lse2 * 0.69314718055994531f;
          }
          tc_fence_before();
          fence_proxy_async_smem();  // the other half's P is copied to its places next
          __syncwarp();
        } else {
          give_up();
        }
      }
      // No barrier here: the next list's queries and first keys are fetched while this
      // one's last PV runs, and its first QK^T runs while its outputs are written. Its
      // first PV waits for the softmax warps (pfull), so for their reads of O and the
      // zeros; its first P comes after an exchange of maxima with the warps whose
      // places it writes.
      fc += (kKStages + kVStages) * n;
      u += n;
      ++uc;
      if constexpr (!kSoft) {
        if (ok && u < work.end) tile = prm.tiles[ti + 1];
      }
    }
  };
  if (warp < 4) {
    regs_dec<kHelperRegs>();
    lists(std::false_type{});
  } else {
    regs_inc<kSoftRegs>();
    lists(std::true_type{});
  }
  __syncwarp();
  cluster_sync_all();
  if (*abort_flag) {
    // unwinding: copies and MMAs in flight land within microseconds; wait longer
    const long long t0 = clock64();
    while (clock64() - t0 < 4000000) __nanosleep(1000);
    if (tid == 0) set_status(prm.dev_status, DSA_STATUS_TIMEOUT);
  }
  __syncwarp();
  cluster_sync_all();
  if (warp == 0) tmem_dealloc_pair(tmem, kTmemCols);
}

// Merges the lists that were divided: block x takes the x-th of them, which the end of
// some share is the first to cut; a warp takes half a row or a quarter. About 8 us at
// 32 x 16384 keys: 2304 blocks, some of them idle, took 1 us more, whole rows or loops
// over rows as much.
constexpr int kMergeWarps = 8, kMergeCtas = 4;  // per SM
constexpr unsigned kFewLists = 8;
template <int kPieces>  // of 128 columns, 8 / kPieces parts of them in flight
__global__ void __launch_bounds__(kMergeWarps * 32, kMergeCtas) prefix_merge_kernel(const PrefixParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = lane_id();
  int x = blockIdx.x, k0 = -1;
#pragma unroll
  for (int j = 0; j < kMaxShares / 32; ++j) {
    const int k = 32 * j + lane;
    const uint32_t cuts = __ballot_sync(0xffffffffu, k < p.shares && p.share[k].cut_rows > 0);
    const uint32_t it = __ballot_sync(0xffffffffu, (cuts >> lane & 1) && __popc(cuts & below(lane)) == x);
    if (it) k0 = 32 * j + __ffs(it) - 1;
    x -= __popc(cuts);
  }
  if (k0 < 0) return;
  const PrefixShare share = p.share[k0];
  constexpr int kUnits = 4 / kPieces, kAhead = 8 / kPieces;  // units of a row
  const int w = blockIdx.y * kMergeWarps + warp_id(), r = w / kUnits, unit = w % kUnits, k1 = share.last;
  if (r >= share.cut_rows) return;
  auto row_of = [&](int k) { return (size_t)(k == k0 ? share.first_slot : 2 * k) * kTileRows + r; };
  // the first parts' rows are on their way while the weights are found
  float4 y[kAhead][kPieces];
  auto load = [&](int k) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (k + j > k1) break;
      const float4* src = reinterpret_cast<const float4*>(p.part_o + row_of(k + j) * kDv + unit * kPieces * 128);
#pragma unroll
      for (int h = 0; h < kPieces; ++h) y[j][h] = src[32 * h + lane];
    }
  };
  load(k0);
  float mx = -INFINITY, tot = 0.f;
  for (int k = k0 + lane; k <= k1; k += 32) mx = fmaxf(mx, p.part_lse[row_of(k)]);
  mx = warp_max_f32(mx);
  for (int k = k0 + lane; k <= k1; k += 32) {
    const float v = p.part_lse[row_of(k)];
    tot += v == -INFINITY ? 0.f : exp2f(v - mx);  // NaN stays NaN
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, d);
  const bool some = tot != 0.f;
  const float inv = some ? 1.f / tot : 0.f;
  float4 acc[kPieces];
#pragma unroll
  for (int h = 0; h < kPieces; ++h) acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int k = k0; k <= k1; k += kAhead) {
    if (k > k0) load(k);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (k + j > k1) break;
      const float v = p.part_lse[row_of(k + j)], wt = v == -INFINITY ? 0.f : exp2f(v - mx) * inv;
#pragma unroll
      for (int h = 0; h < kPieces; ++h) {
        acc[h].x = fmaf(wt, y[j][h].x, acc[h].x);
        acc[h].y = fmaf(wt, y[j][h].y, acc[h].y);
        acc[h].z = fmaf(wt, y[j][h].z, acc[h].z);
        acc[h].w = fmaf(wt, y[j][h].w, acc[h].w);
      }
    }
  }
  uint2* dst = reinterpret_cast<uint2*>(p.o + ((size_t)share.cut_row0 + r) * kDv + unit * kPieces * 128);
#pragma unroll
  for (int h = 0; h < kPieces; ++h) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(acc[h].x, acc[h].y), hi = __floats2bfloat162_rn(acc[h].z, acc[h].w);
    dst[32 * h + lane] = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  }
  if (unit == 0 && lane == 0 && p.lse)
    p.lse[(size_t)share.cut_row0 + r] = some ? (mx + log2f(tot)) * 0.69314718055994531f : -INFINITY;
}

int max_tiles_of(int T, int H, int G) { return (int)(((long long)T * H + kTileRows - 1) / kTileRows) + G; }
int max_shares() { return std::min(std::max(1, sm_count() / 4), kMaxShares); }
// Clusters that the current device runs at once (a cluster lies in one GPC, so
// there are fewer than SMs / 4), asked once per device.
int clusters_at_once() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return max_shares();
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(4 * max_shares());
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 4;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, prefix_mla_kernel, &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    return max_shares();
  }
  n = std::min(n, max_shares());
  cached[dev].store(n, std::memory_order_relaxed);
  return n;
}
// The kernel's launch has the registers that its warps share out later: a CTA that
// waits for more than there are would wait forever.
bool registers_fit() {
  static std::atomic<int> known{-1};
  int fit = known.load(std::memory_order_relaxed);
  if (fit >= 0) return fit;
  cudaFuncAttributes a;
  if (cudaFuncGetAttributes(&a, prefix_mla_kernel) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  fit = a.numRegs >= kLaunchRegs;
  known.store(fit, std::memory_order_relaxed);
  return fit;
}
struct Layout {
  size_t tile_base, tiles, unit_base, share, part_o, part_lse, bytes;
};
Layout layout_of(int T, int H, int G) {
  const size_t nt = (size_t)max_tiles_of(T, H, G), slots = 2 * (size_t)max_shares();
  Layout l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, 256);
    return here;
  };
  l.tile_base = take(((size_t)G + 1) * 4);
  l.tiles = take(nt * sizeof(PrefixTile));
  l.unit_base = take((nt + 1) * 4);
  l.share = take(slots / 2 * sizeof(PrefixShare));
  l.part_lse = take(slots * kTileRows * 4);
  l.part_o = take(slots * kTileRows * kDv * 4);
  l.bytes = at;
  return l;
}
}  // namespace

// Key tiles of a row tile, at most: it has rows of ceil(256 / H) + 1 requests or
// fewer, and the prefix.
static long long max_units_of(int H, int max_kv) {
  return (2LL + (kTileRows + H - 1) / H) * ((long long)max_kv / (2 * kRun) + 4);
}
bool prefix_units_fit(int T, int H, int G, int max_kv) {
  return max_tiles_of(T, H, G) * (max_units_of(H, max_kv) + kListCost) < (1LL << 31);
}

size_t prefix_workspace_bytes(int T, int H, int G) { return layout_of(T, H, G).bytes; }

int run_prefix_mla(cudaStream_t stream, PrefixParams prm, void* ws) {
  const Layout l = layout_of(prm.T, prm.H, prm.G);
  uint8_t* w = static_cast<uint8_t*>(ws);
  prm.tile_base = reinterpret_cast<int32_t*>(w + l.tile_base);
  prm.tiles = reinterpret_cast<PrefixTile*>(w + l.tiles);
  prm.unit_base = reinterpret_cast<int*>(w + l.unit_base);
  prm.share = reinterpret_cast<PrefixShare*>(w + l.share);
  prm.part_o = reinterpret_cast<float*>(w + l.part_o);
  prm.part_lse = reinterpret_cast<float*>(w + l.part_lse);
  prm.max_tiles = max_tiles_of(prm.T, prm.H, prm.G);
  prm.max_units = (int)max_units_of(prm.H, prm.max_kv);
  CUtensorMap kvmap, qmap;
  if (!encode_bf16_2d(&kvmap, prm.kv, (uint64_t)prm.P * prm.ps, (uint64_t)prm.row_stride, std::min(prm.ps, 64),
                      kDk) ||
      !encode_bf16_2d(&qmap, prm.q, (uint64_t)prm.T * prm.H, kDk, kRows, kDk) || !registers_fit())
    return DSA_ERR_CUDA;
  set_smem_attr_once(reinterpret_cast<const void*>(prefix_mla_kernel), kSmem);
  prm.shares = clusters_at_once();
  DSA_LAUNCH_PDL(prefix_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, prm);
  DSA_LAUNCH_PDL(prefix_mla_kernel, dim3(4 * prm.shares), dim3(kThreads), kSmem, stream, prm, kvmap, qmap);
  // Quarters of rows where few lists have many parts each: 4 row tiles 81.9 us, by halves
  // 83.0, 2 tiles 111.2 and 112.5; but 12 tiles 50.2 and 48.2, 16 tiles 113.2 and 109.8, and
  // 32 rows in all 17.5 and 17.2.
  const unsigned lists = (unsigned)std::min(prm.shares, prm.max_tiles);
  if (lists <= kFewLists && (long long)prm.T * prm.H > kTileRows)
    DSA_LAUNCH_PDL(prefix_merge_kernel<1>, dim3(lists, 4 * kTileRows / kMergeWarps), dim3(kMergeWarps * 32), 0, stream,
                   prm);
  else
    DSA_LAUNCH_PDL(prefix_merge_kernel<2>, dim3(lists, 2 * kTileRows / kMergeWarps), dim3(kMergeWarps * 32), 0, stream,
                   prm);
  return DSA_OK;
}

}  // namespace dsa
