// Absorbed-MLA attention over the 4-bit latent cache (token and page
// selections), and over the bf16 cache with a sliding window and sinks. The
// mathematics and the split of the work are attend.cu's:
//   S = Q K^T over 576 dims, online softmax, O += P V, V = the first 512 dims,
// one CTA per query token, 128 heads and half of the value columns, in tiles
// of 64 keys. With 64 heads or fewer half of those 128 rows would be empty:
//  - neighbouring tokens of a request share a CTA of the window form, 128 rows
//    of (token, head): they see nearly the same keys, and each row masks its own;
//  - a token by itself takes one CTA instead of two (kBoth): its queries stand
//    in rows 0-63 and again in rows 64-127, P is written twice, once with the
//    lower and once with the upper rows zero, and PV adds lower P times the
//    first 256 value columns and upper P times the others into the same TMEM
//    columns. QK^T, the keys' fetch and their unpacking happen once.
// 4-bit keys are 416-byte rows that sixteen copier warps turn into bf16 column
// blocks on their way to shared memory; bf16 keys are runs of 32 rows of a page,
// fetched by one thread as TMA boxes.
//
// Roles: warp 0 issues the MMAs, warp 1 resolves the keys (KeyList), warps
// 4-7 move the queries' first 256 dims into TMEM and run the softmax, others
// copy. Key lists are split over a cluster of up to eight CTAs, whose
// partial outputs are merged through distributed shared memory: no workspace,
// no counters, and every CTA of the cluster merges a share of the head rows.
//
// The loops are rolled. Five roles share the SM's instruction cache; with
// attend.cu's unrolled loops it hit 60% of the time here and warps waited for
// instructions more than for anything else, rolled it hits 95%.
#include <atomic>
#include <type_traits>

#include "attend.cuh"
#include "common.cuh"
#include "q4.cuh"
#include "steps.cuh"

namespace dsa {

namespace {
// what an instantiation reads
enum : int { kCacheBf16 = 0, kCache4Bit = 1 };

constexpr int kDk = 576, kDv = 512;
constexpr int kSubKeys = 32;  // keys resolved per step
constexpr int kTile = 64, kSteps = kTile / kSubKeys;
constexpr int kRing = 8;       // tiles resolved ahead (their rows are pulled into L2 meanwhile)
constexpr int kMaxSplits = 8;  // CTAs of a portable cluster
constexpr int kNoKeys = 0x7fffff00;  // the position of a run that holds no keys
constexpr float kRescaleThreshold = 8.f;  // log2 units: p stays <= 256
constexpr int kHeads = 128;  // rows of a CTA: heads, or heads of neighbouring tokens

// shared memory: 128-byte-swizzled blocks of 64 columns. The queries' dims
// 0-255 live in TMEM. A tile is nine blocks of keys: the four of this CTA's
// value half (the V part) stay until PV has read them, the other four and the
// rotary block (the K part) until QK^T has.
constexpr int kBlk = kTile * 128, kQBlk = kHeads * 128;
constexpr int kKStage = 5 * kBlk, kVStage = 4 * kBlk;
constexpr int OFF_Q = 0;  // dims 256-575
constexpr int OFF_K = OFF_Q + 5 * kQBlk;
constexpr int OFF_V = OFF_K + 2 * kKStage;
constexpr int OFF_RING = OFF_V + 2 * kVStage;           // int32 [kRing][kTile] rows
constexpr int OFF_MASK = OFF_RING + kRing * kTile * 4;  // uint32 [kRing][kSteps]; bf16: a run's first position
constexpr int OFF_END = OFF_MASK + kRing * kSteps * 4;  // uint32 [kRing]
constexpr int OFF_BAR = OFF_END + kRing * 4;
constexpr int kNumBars = 2 * kRing + 15;
constexpr int OFF_MISC = OFF_BAR + kNumBars * 8;  // TMEM address, abort flag
constexpr int kSmem = OFF_MISC + 32;  // and the CTA's tokens
static_assert(kSmem <= 227 * 1024, "shared memory budget");
static_assert(OFF_K % 1024 == 0 && OFF_V % 1024 == 0 && OFF_BAR % 8 == 0, "alignment");
static_assert(4 * kQBlk <= 2 * kKStage, "the queries for TMEM land in the key stages");
// after the last MMA: fp32 partial rows of 256 value columns, padded against
// bank conflicts, their log-sums, and the weights of the splits
constexpr int kStageLd = 256 + 4;
constexpr int kOutLd = 512 + 16;  // bytes of a staged bf16 row
static_assert(kHeads * kOutLd <= 2 * kKStage, "bf16 rows are staged in the key stages");
constexpr int OFF_LSE = kHeads * kStageLd * 4;
constexpr int OFF_WTS = OFF_LSE + kHeads * 4;
static_assert(OFF_WTS + kMaxSplits * kHeads * 4 <= OFF_RING, "split stage");

constexpr uint32_t kIdescQK = make_idesc_bf16(kHeads, kTile, false, false);
constexpr uint32_t kIdescPV = make_idesc_bf16(kHeads, 256, false, true);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColQ = 0;    // 128 columns of packed bf16 pairs
constexpr uint32_t kColS = 128;  // two S buffers of 64 columns; P (bf16 pairs) overwrites S
constexpr uint32_t kColO = 256;

// 4-bit rows: sixteen warps of four keys each (eight warps of eight keys
// waited for their loads a quarter of the time)
template <int kCache>
constexpr int kCopyWarps = kCache == kCache4Bit ? 16 : 1;
// the 4-bit copiers are warps 8-23; the TMA issuer is warp 2, away from the MMA
// issuer's quarter of the SM (as warp 8 it costs 4%: 924 against 885 us for 2049
// tokens; for the 4-bit copiers it made no difference where they were)
template <int kCache>
constexpr int kThreads = (kCache == kCache4Bit ? 8 + kCopyWarps<kCache> : 8) * 32;
template <int kCache>
__device__ __forceinline__ int copier_of(int warp) {  // its number, or -1
  return kCache == kCache4Bit ? max(warp - 8, -1) : warp == 2 ? 0 : -1;
}

// The keys a CTA visits, 32 at a time, resolved by one whole warp. 4-bit cache:
// windows of 32 selected tokens, or runs of 32 rows of selected pages; bf16
// cache: runs of 32 rows of the pages that hold sinks, then of those that hold
// the window. The CTAs of a cluster take equal shares of the list.
template <int kCache>
struct KeyList {
  static constexpr int kBatch = 8;  // token windows resolved at a time
  const AttendParams* p;
  int t, n_vis, page_base, lg;  // lg: the page size is 2^lg
  int key_lo, n_sink, p_skip;   // window: its first position, pages of sinks before its pages, pages skipped between
  int e, e1;                    // next entry of the list, end of this CTA's share
  // tokens: the batch's rows, one key per lane, and its windows with keys
  int row_of[kBatch];
  uint32_t mask_of[kBatch], left;
  // pages: a window of 32 entries, one per lane, and those still to visit
  uint32_t pend;
  int phys, first_key;          // this lane's page (-1: none) and its first position
  int cur_phys, cur_key, sub;   // the page being walked and its next run

  // the list of tokens tok .. tok + ntok - 1 of one request (ntok > 1: bf16)
  __device__ void init(const AttendParams& prm, int tok, int ntok, int split) {
    p = &prm;
    t = tok;
    lg = 31 - __clz(prm.ps);
    const int s = seq_of_token_warp(prm.cu_q_lens, prm.S, tok);
    const TokenGeom g = token_geom(prm.seq_lens, prm.cu_q_lens, prm.cu_kv_lens, prm.S, prm.ps, 0x3fffffff, tok,
                                   prm.dev_status, s);
    n_vis = max(0, min(g.kv_len, g.pos + ntok));  // of the last token
    page_base = g.page_base;
    left = pend = 0;
    sub = prm.ps / kSubKeys;
    int n = prm.K, share;
    if constexpr (kCache == kCacheBf16) {
      key_lo = max(0, g.pos - prm.window + 1);
      const int p_lo = key_lo >> lg;
      n_sink = (int)min((long long)p_lo, ((long long)prm.sinks + prm.ps - 1) >> lg);
      p_skip = p_lo - n_sink;
      n = ((n_vis + prm.ps - 1) >> lg) - p_skip;
    }
    share = (max(n, 0) + prm.nsplit - 1) / prm.nsplit;
    if (kCache == kCache4Bit && prm.mode == kModeToken) share = (share + 31) & ~31;
    e = min(max(n, 0), split * share);
    e1 = min(max(n, 0), e + share);
  }

  // physical page of packed page-table entry `ent`, or -1
  __device__ __forceinline__ int page_of(int ent) const {
    if (ent < 0 || ent >= p->PTW) {
      set_status(p->dev_status, DSA_STATUS_BAD_INDEX);
      return -1;
    }
    const int pg = __ldg(p->page_indices + ent);
    if (pg < 0 || pg >= p->P) {
      set_status(p->dev_status, DSA_STATUS_BAD_METADATA);
      return -1;
    }
    return pg;
  }

  // The next 32 keys: this lane's row (-1: masked) and the mask of the rows
  // (bf16: of those that any token sees); base: the first row of a run and
  // pos0: its position. False: the share is exhausted.
  __device__ bool next(int& row, uint32_t& mask, int& base, int& pos0) {
    if (kCache == kCache4Bit && p->mode == kModeToken) return next_tokens(row, mask);
    while (true) {
      if (sub < (p->ps >> 5)) {
        const int k0 = sub * kSubKeys + lane_id(), key = cur_key + k0;
        bool v = key < n_vis;
        if constexpr (kCache == kCacheBf16) v = v && (key >= key_lo || key < p->sinks);
        base = (cur_phys << lg) + sub * kSubKeys;
        pos0 = cur_key + sub * kSubKeys;
        ++sub;
        row = v ? (cur_phys << lg) + k0 : -1;
        mask = __ballot_sync(0xffffffffu, v);
        if (mask) return true;
        continue;
      }
      if (!pend) {
        if (e >= e1) return false;
        int pg = e + lane_id();
        bool v = pg < e1;
        if constexpr (kCache == kCacheBf16) {
          pg += pg < n_sink ? 0 : p_skip;
        } else {
          pg = v ? __ldg(p->sel + (size_t)t * p->K + pg) : -1;
          v = pg >= 0 && ((long long)pg << lg) < n_vis;
        }
        phys = v ? page_of(page_base + pg) : -1;
        first_key = v ? pg << lg : 0;
        pend = __ballot_sync(0xffffffffu, phys >= 0);
        e += 32;
        continue;
      }
      const int bit = __ffs(pend) - 1;
      pend &= pend - 1u;
      cur_phys = __shfl_sync(0xffffffffu, phys, bit);
      cur_key = __shfl_sync(0xffffffffu, first_key, bit);
      sub = 0;
    }
  }

  __device__ __forceinline__ bool next_tokens(int& row, uint32_t& mask) {
    while (!left) {
      if (e >= e1) return false;
      // two dependent rounds of loads (entries, pages) for a whole batch;
      // array indexes are constants, so the batch stays in registers
      int j[kBatch], pg[kBatch];
#pragma unroll
      for (int g = 0; g < kBatch; ++g) {
        const int ee = e + 32 * g + lane_id();
        j[g] = ee < e1 ? __ldg(p->sel + (size_t)t * p->K + ee) : -1;
      }
#pragma unroll
      for (int g = 0; g < kBatch; ++g) pg[g] = j[g] >= 0 && j[g] < n_vis ? page_of(page_base + (j[g] >> lg)) : -1;
#pragma unroll
      for (int g = 0; g < kBatch; ++g) {
        row_of[g] = pg[g] >= 0 ? (pg[g] << lg) + (j[g] & (p->ps - 1)) : -1;
        mask_of[g] = __ballot_sync(0xffffffffu, pg[g] >= 0);
        left |= (mask_of[g] ? 1u : 0u) << g;
      }
      e += 32 * kBatch;
    }
    const int w = __ffs(left) - 1;
    left &= left - 1u;
#pragma unroll
    for (int g = 0; g < kBatch; ++g)
      if (g == w) row = row_of[g], mask = mask_of[g];
    return true;
  }
};

struct Bars {
  uint64_t* b;
  __device__ __forceinline__ uint64_t* rfull(int s) const { return b + s; }                  // generator
  __device__ __forceinline__ uint64_t* rempty(int s) const { return b + kRing + s; }         // readers of a ring slot
  __device__ __forceinline__ uint64_t* full(int part, int s) const { return b + 2 * kRing + 2 * part + s; }  // copier warps
  __device__ __forceinline__ uint64_t* empty(int part, int s) const { return b + 2 * kRing + 4 + 2 * part + s; }  // commit
  __device__ __forceinline__ uint64_t* sfull(int s) const { return b + 2 * kRing + 8 + s; }  // commit
  __device__ __forceinline__ uint64_t* pfull(int s) const { return b + 2 * kRing + 10 + s; } // softmax warps
  __device__ __forceinline__ uint64_t* pvdone() const { return b + 2 * kRing + 12; }         // commit
  __device__ __forceinline__ uint64_t* qbar() const { return b + 2 * kRing + 13; }           // the queries' copies
  __device__ __forceinline__ uint64_t* fin() const { return b + 2 * kRing + 14; }            // commit while unwinding
};

// The MMA issuer (one converged warp). Per tile i: QK^T(i) over the K part,
// then over the V part, then PV(i - 1), so that the softmax of a tile runs
// beside the next tile's QK^T. With kBoth PV reads the K part as well, which
// then stays as long as the V part.
template <bool kBoth>
__device__ __forceinline__ void issue_mmas(int half, uint32_t tmem, uint32_t smem0, const Bars& br,
                                           volatile const uint32_t* ring_end, volatile int* abort_flag) {
  const uint32_t lead = elect_one();
  const uint64_t dq = make_sdesc(smem0 + OFF_Q, 16, 1024, kSwizzle128B);
  const uint64_t dk = make_sdesc(smem0 + OFF_K, 16, 1024, kSwizzle128B);
  const uint64_t dv = make_sdesc(smem0 + OFF_V, 16, 1024, kSwizzle128B);
  // MN-major, as operands of PV: blocks kBlk apart
  const uint64_t dkn = make_sdesc(smem0 + OFF_K, kBlk, 1024, kSwizzle128B);
  const uint64_t dvn = make_sdesc(smem0 + OFF_V, kBlk, 1024, kSwizzle128B);
  // N column blocks of keys from b against the query blocks in TMEM (0-3), or
  // in shared memory from a
  auto blocks_ts = [&](uint32_t tS, uint64_t b, uint32_t acc) {
#pragma unroll
    for (int k = 0; k < 16; ++k, acc = 1u)
      umma_bf16_ts_lead(lead, tS, tmem + kColQ + k * 8, b + (k >> 2) * (kBlk >> 4) + (k & 3) * 2, kIdescQK, acc);
  };
  auto blocks_ss = [&](uint32_t tS, uint64_t a, uint64_t b, uint32_t acc, auto N) {
#pragma unroll
    for (int k = 0; k < 4 * decltype(N)::value; ++k, acc = 1u)
      umma_bf16_ss_lead(lead, tS, a + (k >> 2) * (kQBlk >> 4) + (k & 3) * 2, b + (k >> 2) * (kBlk >> 4) + (k & 3) * 2,
                        kIdescQK, acc);
  };
  using One = std::integral_constant<int, 1>;
  using Four = std::integral_constant<int, 4>;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return mbar_wait_warp(bar, parity, abort_flag); };
  auto commit = [&](uint64_t* bar) {
    if (lead) umma_commit(bar);
    __syncwarp();
  };
  bool ok = wait(br.qbar(), 0), issued = false;
#pragma unroll 1
  for (int i = 0; ok; ++i) {
    const int slot = i % kRing, st = i & 1, ph = (i >> 1) & 1;
    if (!(ok = wait(br.rfull(slot), (i / kRing) & 1))) break;
    const bool end = __any_sync(0xffffffffu, ring_end[slot] != 0);
    if (lead) mbar_arrive(br.rempty(slot));
    __syncwarp();
    if (!end) {
      const uint32_t tS = tmem + kColS + (uint32_t)st * kTile;
      const uint64_t kb = dk + (uint64_t)(st * (kKStage >> 4)), vb = dv + (uint64_t)(st * (kVStage >> 4));
      if (!(ok = wait(br.full(0, st), ph))) break;
      fence_proxy_async_smem();
      tc_fence_after();
      // value half 0: dims 256-575 are the K part, dims 0-255 the V part;
      // half 1 and kBoth: dims 0-255 and the rotary block, then dims 256-511
      if (half) blocks_ts(tS, kb, 0u);
      else blocks_ss(tS, dq, kb, 0u, Four{});
      blocks_ss(tS, dq + 4 * (kQBlk >> 4), kb + 4 * (kBlk >> 4), 1u, One{});
      if (!kBoth) commit(br.empty(0, st));
      issued = true;
      if (!(ok = wait(br.full(1, st), ph))) break;
      fence_proxy_async_smem();
      tc_fence_after();
      if (half) blocks_ss(tS, dq, vb, 1u, Four{});
      else blocks_ts(tS, vb, 1u);
      commit(br.sfull(st));
    }
    if (i > 0) {
      const int j = i - 1, sj = j & 1;
      if (!(ok = wait(br.pfull(sj), (j >> 1) & 1))) break;
      tc_fence_after();
      const uint32_t tP = tmem + kColS + (uint32_t)sj * kTile;
      auto pv = [&](uint32_t a, uint64_t b, uint32_t acc) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k, acc = 1u)
          umma_bf16_ts_lead(lead, tmem + kColO, a + k * 8, b + (uint64_t)(k * 128), kIdescPV, acc);
      };
      if (kBoth) {  // the K part holds the first 256 value columns
        pv(tP, dkn + (uint64_t)(sj * (kKStage >> 4)), j > 0 ? 1u : 0u);
        commit(br.empty(0, sj));
      }
      pv(tP + (kBoth ? 32 : 0), dvn + (uint64_t)(sj * (kVStage >> 4)), kBoth || j > 0 ? 1u : 0u);
      commit(br.empty(1, sj));
      commit(br.pvdone());
    }
    if (end) break;
  }
  if (!ok && issued) {  // unwinding: no MMA may be left reading shared memory
    commit(br.fin());
    mbar_wait_drain(br.fin(), 0);
  }
}

// A copier warp: four keys of every tile, a K part and a V part each. Sixteen
// lanes share a key: a lane holds one group of 16 dims (two words, one scale),
// so a load is two keys' runs of 128 bytes. The loads of the next part are in
// flight while this one is unpacked.
//
// A word's bits are shifted into place as bf16 bit patterns worth 2^-126 of
// the codes' values, and one packed multiply by the scale times 2^119 finishes
// them: the product with 2^126 would overflow at scales above 2 (the largest
// is 448 < 2^9), so a tile holds the keys times 2^-7. The rotary dims are
// multiplied to match, the softmax scales the logits back and the epilogue
// the output; powers of two, so all exact.
//
// The two words of a lane are two neighbouring 16-byte chunks of a block's
// row; every other quarter of a key stores them in the other order, so that
// eight lanes always hit eight different bank groups.
__device__ __forceinline__ void copy_keys(const uint8_t* __restrict__ cache, int half, int cw, uint8_t* smem,
                                          const int* ring_rows, volatile const uint32_t* ring_end, const Bars& br,
                                          volatile int* abort_flag) {
  constexpr int kKeysPerWarp = kTile / kCopyWarps<kCache4Bit>, N = kKeysPerWarp / 2;  // pairs of keys
  static_assert(kKeysPerWarp == 4, "eight lanes per key cover the rotary dims of a warp's keys");
  const int lane = lane_id();
  const int kl = lane >> 4, g = lane & 15;  // key of the pair, group of the part
  const int key0 = cw * kKeysPerWarp;
  const bool swap = lane & 4;
  const uint32_t smem0 = smem_u32(smem);
  struct Part {
    uint2 w[N];
    uint32_t b[N];
    uint4 rp;  // 16 bytes of the rotary dims of key key0 + lane / 8
  };
  auto load = [&](Part& x, int i, int part) {
    const int* rows = ring_rows + i % kRing * kTile + key0;
    const int code = (part ? half : half ^ 1) * 128 + g * 8;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int r = rows[2 * k + kl];
      const uint8_t* p = cache + (size_t)max(r, 0) * kRow4Bytes;
      // a masked key (r < 0) has zero codes and a zero scale
      x.w[k] = r >= 0 ? __ldg(reinterpret_cast<const uint2*>(p + code)) : make_uint2(0u, 0u);
      x.b[k] = r >= 0 ? __ldg(p + kRow4Codes + code / 8) : 0u;
    }
    if (!part) {
      const int r = rows[lane >> 3];
      const uint8_t* p = cache + (size_t)max(r, 0) * kRow4Bytes + kRow4Codes + kRow4Scales;
      x.rp = r >= 0 ? __ldg(reinterpret_cast<const uint4*>(p) + (lane & 7)) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  // whether there is a tile i (the list may end, or a wait give up)
  auto tile = [&](int i) -> bool {
    return mbar_wait_warp(br.rfull(i % kRing), (i / kRing) & 1, abort_flag) && !ring_end[i % kRing];
  };
  Part cur, nxt;
  bool have = tile(0);
  if (have) load(cur, 0, 0);
#pragma unroll 1
  for (int u = 0; have; ++u) {  // part u & 1 of tile u / 2
    const int i = u >> 1, part = u & 1, st = i & 1;
    const bool more = !part || tile(i + 1);
    if (more) load(nxt, i + part, part ^ 1);
    if (!mbar_wait_warp(br.empty(part, st), ((i >> 1) & 1) ^ 1, abort_flag)) break;
    const uint32_t base = smem0 + (part ? OFF_V + st * kVStage : OFF_K + st * kKStage);
    const uint32_t d = base + (g >> 2) * kBlk;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t s2 = bf16x2_of(e4m3_value(cur.b[k]) * 0x1p119f), key = key0 + 2 * k + kl, c = 2 * (g & 3);
      const uint4 a = q4_scaled8(swap ? cur.w[k].y : cur.w[k].x, s2), b = q4_scaled8(swap ? cur.w[k].x : cur.w[k].y, s2);
      st_shared_v4(d + sw128_offset(key, c + (swap ? 1 : 0)), a.x, a.y, a.z, a.w);
      st_shared_v4(d + sw128_offset(key, c + (swap ? 0 : 1)), b.x, b.y, b.z, b.w);
    }
    if (!part) {
      constexpr uint32_t k2m7 = 0x3c003c00u;  // 2^-7 in both halves
      st_shared_v4(base + 4 * kBlk + sw128_offset(key0 + (lane >> 3), lane & 7), mul_bf16x2(cur.rp.x, k2m7),
                   mul_bf16x2(cur.rp.y, k2m7), mul_bf16x2(cur.rp.z, k2m7), mul_bf16x2(cur.rp.w, k2m7));
    }
    fence_proxy_async_smem();  // this lane's stores, for the MMAs
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(br.full(part, st));
      if (part) mbar_arrive(br.rempty(i % kRing));
    }
    cur = nxt;
    have = more;
  }
}

// The copier of the bf16 cache, one thread: every step of a tile is 32
// consecutive rows of one page, boxes of 32 rows x 64 columns. An empty step's
// first row is -32: its boxes lie wholly outside the cache and land as zeros.
__device__ __forceinline__ void copy_boxes(const CUtensorMap* kvmap, int half, uint8_t* smem, const int* ring_rows,
                                           volatile const uint32_t* ring_end, const Bars& br,
                                           volatile int* abort_flag) {
  constexpr uint32_t kBox = kSubKeys * 128;
  bool ok = true;
  int i = 0, part = 0;
#pragma unroll 1
  for (;; part ^= 1, i += !part) {
    const int st = i & 1, n = part ? 4 : 5;
    if (!part && (!(ok = mbar_wait(br.rfull(i % kRing), (i / kRing) & 1, abort_flag)) || ring_end[i % kRing])) break;
    if (!(ok = mbar_wait(br.empty(part, st), ((i >> 1) & 1) ^ 1, abort_flag))) break;
    const int* base = ring_rows + i % kRing * kTile;
    uint8_t* d = smem + (part ? OFF_V + st * kVStage : OFF_K + st * kKStage);
    mbar_arrive_expect_tx(br.full(part, st), n * kSteps * kBox);
#pragma unroll 1
    for (int c = 0; c < n; ++c) {
      const int dims = (c == 4 ? 8 : 4 * (part ? half : half ^ 1) + c) * 64;
      for (int s = 0; s < kSteps; ++s)
        tma_load_2d(d + c * kBlk + s * kBox, kvmap, br.full(part, st), dims, base[s]);
    }
    if (part) mbar_arrive(br.rempty(i % kRing));
  }
  if (!ok) {  // unwinding: no copy may land after the CTA has gone
#pragma unroll 1
    for (int u = max(0, 2 * i + part - 4); u < 2 * i + part; ++u)
      mbar_wait_drain(br.full(u & 1, (u >> 1) & 1), (u >> 2) & 1);
  }
}

// The g-th run of up to G neighbouring tokens of one request, request by
// request: its first token and length (0: there are fewer runs). One warp.
__device__ __forceinline__ int2 token_run(const AttendParams& p, int g, int G) {
  const int lane = lane_id();
  long long before = 0;  // runs of the requests before
  for (int s0 = 0; s0 < p.S; s0 += 32) {
    const int s = s0 + lane;
    const int q0 = s < p.S ? __ldg(p.cu_q_lens + s) : 0, q1 = s < p.S ? __ldg(p.cu_q_lens + s + 1) : 0;
    const int n = q1 > q0 && q0 >= 0 ? (int)(((long long)q1 - q0 + G - 1) / G) : 0;
    long long x = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    const long long k = g - (before + x - n);  // the run's number within this lane's request
    const uint32_t has = __ballot_sync(0xffffffffu, k >= 0 && k < n);
    if (has) {
      const int src = __ffs(has) - 1;
      const long long first = q0 + k * G;
      const int t0 = (int)__shfl_sync(0xffffffffu, first, src);
      const int len = (int)__shfl_sync(0xffffffffu, min((long long)G, min((long long)q1, (long long)p.T) - first), src);
      return make_int2(t0, max(len, 0));
    }
    before += __shfl_sync(0xffffffffu, x, 31);
  }
  return make_int2(0, 0);
}

// kBoth: H <= 64, a CTA has both value halves
template <int kCache, bool kBoth>
__global__ void __launch_bounds__(kThreads<kCache>, 1)
    cache_mla_kernel(const AttendParams prm, const __grid_constant__ CUtensorMap kvmap,
                     const __grid_constant__ CUtensorMap qmap) {
  constexpr bool k4 = kCache == kCache4Bit;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // in every CTA alike
    if (threadIdx.x == 0) set_status(prm.dev_status, DSA_STATUS_INTERNAL);
    return;
  }
  griddep_launch_dependents();
  const int warp = warp_id(), lane = lane_id(), tid = threadIdx.x;
  constexpr int kRows = kBoth ? kHeads / 2 : kHeads;  // output rows of the CTA
  // kBoth loads and multiplies as value half 1 does
  const int half = kBoth ? 1 : blockIdx.x & 1, h0 = kBoth ? 0 : (blockIdx.x >> 1) * kHeads;
  const int split = blockIdx.z;  // the rank in the cluster
  int* ring_rows = reinterpret_cast<int*>(smem + OFF_RING);
  volatile uint32_t* ring_mask = reinterpret_cast<volatile uint32_t*>(smem + OFF_MASK);
  volatile uint32_t* ring_end = reinterpret_cast<volatile uint32_t*>(smem + OFF_END);
  const Bars br{reinterpret_cast<uint64_t*>(smem + OFF_BAR)};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  if (tid == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(br.rfull(s), 1);
      mbar_init(br.rempty(s), 4 + kCopyWarps<kCache> + 1);  // softmax and copier warps, the MMA issuer
    }
    for (int s = 0; s < 2; ++s) {
      for (int part = 0; part < 2; ++part) {
        mbar_init(br.full(part, s), kCopyWarps<kCache>);
        mbar_init(br.empty(part, s), 1);
      }
      mbar_init(br.sfull(s), 1);
      mbar_init(br.pfull(s), 4);
    }
    mbar_init(br.pvdone(), 1);
    mbar_init(br.qbar(), 1);
    mbar_init(br.fin(), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  const uint32_t tmem = *tmem_slot;
  // this CTA's tokens t .. t + ntok - 1
  int t = (int)blockIdx.y, ntok = t < __ldg(prm.cu_q_lens + prm.S) ? 1 : 0;
  if constexpr (!k4) {
    if (prm.pack > 1) {
      volatile int* tokens = reinterpret_cast<volatile int*>(smem + OFF_MISC + 16);
      if (warp == 0) {
        const int2 run = token_run(prm, t, prm.pack);
        if (lane == 0) tokens[0] = run.x, tokens[1] = run.y;
      }
      __syncthreads();
      t = tokens[0];
      ntok = tokens[1];
    }
  }
  if (ntok == 0) {  // a padding row behind the last request: left as it is
    if (warp == 0) tmem_dealloc(tmem, kTmemCols);
    return;
  }
  // rows r of the CTA are rows first_row + r of [T * H], below `rows`
  const int first_row = t * prm.H + h0, rows = min(kRows, ntok * prm.H - h0);
  auto value_half = [&](int r) { return kBoth ? r / kRows : half; };  // of TMEM lane r
  const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;  // this warp's TMEM lanes
  const int r = (warp & 3) * 32 + lane;                          // and this thread's: a row
  if (tid == 0) {
    // the query rows, with kBoth twice (those past `rows` belong to other tokens
    // or lie past the tensor; their outputs are never stored): dims 0-255 wait
    // in the unused key stages until they are moved into TMEM
    mbar_arrive_expect_tx(br.qbar(), 9 * kQBlk);
#pragma unroll 1
    for (int c = 0; c < 9; ++c)
      for (int k = 0; k < kHeads / kRows; ++k)
        tma_load_2d(smem + (c < 4 ? OFF_K + c * kQBlk : OFF_Q + (c - 4) * kQBlk) + k * (kQBlk / 2), &qmap, br.qbar(),
                    c * 64, first_row);
  }
  // the generator resolves its first keys while the queries arrive
  KeyList<kCache> gen;
  if (warp == 1) gen.init(prm, t, ntok, split);
  if (warp >= 4 && warp < 8) {
    if (mbar_wait_warp(br.qbar(), 0, abort_flag)) {
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        const uint8_t* row = smem + OFF_K + c * kQBlk + r * 128;
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 x = *reinterpret_cast<const uint4*>(row + ((j ^ (r & 7)) << 4));
          v[4 * j] = x.x;
          v[4 * j + 1] = x.y;
          v[4 * j + 2] = x.z;
          v[4 * j + 3] = x.w;
        }
        tmem_st32(tmem + lane_base + kColQ + c * 32, v);
      }
    }
    tmem_st_wait();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp == 0) {
    issue_mmas<kBoth>(half, __shfl_sync(0xffffffffu, tmem, 0), smem_u32(smem), br, ring_end, abort_flag);
  } else if (warp == 1) {
    // ---------------------------------------------------------- key generator
    bool more = true;
#pragma unroll 1
    for (int i = 0;; ++i) {
      const int slot = i % kRing;
      int ok = 1;
      if (lane == 0) ok = mbar_wait(br.rempty(slot), ((i / kRing) & 1) ^ 1, abort_flag) ? 1 : 0;
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      bool any = false;
#pragma unroll 1
      for (int s = 0; s < kSteps; ++s) {
        int row = -1, base = -kSubKeys, pos0 = kNoKeys;
        uint32_t mask = 0;
        if (more && !(more = gen.next(row, mask, base, pos0))) row = -1, mask = 0, base = -kSubKeys, pos0 = kNoKeys;
        any |= mask != 0;
        if constexpr (k4) {
          ring_rows[slot * kTile + s * kSubKeys + lane] = row;
          if (row >= 0) {
            // rows come from all over HBM: start pulling them into L2 now
            const uint8_t* rp = prm.kv4 + (size_t)row * kRow4Bytes;
#pragma unroll
            for (int l = 0; l < kRow4Bytes; l += 128) prefetch_l2(rp + l);
            prefetch_l2(rp + kRow4Bytes - 1);  // a row may end in a fifth line
          }
        } else if (lane == 0) {
          ring_rows[slot * kTile + s] = base;  // the step's first row
        }
        if (lane == 0) ring_mask[slot * kSteps + s] = k4 ? mask : (uint32_t)pos0;
      }
      if (lane == 0) ring_end[slot] = any ? 0u : 1u;
      __syncwarp();
      if (lane == 0) mbar_arrive(br.rfull(slot));
      if (!any) break;
    }
  } else if (warp < 4 || warp >= 8) {
    // ---------------------------------------------------------------- copier
    const int cw = copier_of<kCache>(warp);
    if constexpr (k4) {
      if (cw >= 0) copy_keys(prm.kv4, half, cw, smem, ring_rows, ring_end, br, abort_flag);
    } else if (cw >= 0 && lane == 0)
      copy_boxes(&kvmap, half, smem, ring_rows, ring_end, br, abort_flag);
  } else if (warp >= 4) {
    // --------------------------------------------------------------- softmax
    // one row per thread (kBoth: two threads, one per value half); tiles of
    // 4-bit keys hold them times 2^-7 (copy_keys)
    const bool capped = !k4 && prm.soft_cap_on;
    const float sl2 = k4 ? prm.scale_log2 * 128.f : capped ? 1.f : prm.scale_log2;
    auto load_s = [&](uint32_t ts, uint32_t (&s)[32]) {
      tmem_ld32(ts, s);
      tmem_ld_wait_regs(s);
      if (capped) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          s[j] = __float_as_uint(prm.cap_log2 * tanh_approx(__uint_as_float(s[j]) * prm.inv_cap_scale));
      }
    };
    // bf16: this row's visible prefix and window
    int see = 0, from = 0;
    if constexpr (!k4) {
      const TokenGeom g = token_geom(prm.seq_lens, prm.cu_q_lens, prm.cu_kv_lens, prm.S, prm.ps, 0x3fffffff, t,
                                     nullptr, seq_of_token_warp(prm.cu_q_lens, prm.S, t));
      const int pos = g.pos + (ntok > 1 ? r / prm.H : 0);
      see = r % kRows < rows ? max(0, min(g.kv_len, pos + 1)) : 0;
      from = max(0, pos - prm.window + 1);
    }
    auto mask_of = [&](uint32_t x) -> uint32_t {
      if constexpr (k4) return x;
      auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
      const int p0 = (int)x;
      return below(see - p0) & (~below(from - p0) | below(prm.sinks - p0));
    };
    // whether a run is unmasked in every row of the warp
    auto full = [&](uint32_t mk) -> bool { return k4 ? mk == 0xffffffffu : __all_sync(0xffffffffu, mk == 0xffffffffu); };
    float m_run = -INFINITY, l_run = 0.f;
    int n = 0;
    bool ok = true;
#pragma unroll 1
    for (int i = 0;; ++i) {
      const int slot = i % kRing;
      if (!(ok = mbar_wait_warp(br.rfull(slot), (i / kRing) & 1, abort_flag))) break;
      if (ring_end[slot]) break;
      const uint32_t mlo = mask_of(ring_mask[slot * kSteps]), mhi = mask_of(ring_mask[slot * kSteps + 1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(br.rempty(slot));
      if (!(ok = mbar_wait_warp(br.sfull(i & 1), (i >> 1) & 1, abort_flag))) break;
      tc_fence_after();
      const uint32_t tS = tmem + lane_base + kColS + (uint32_t)(i & 1) * 64;
      // Two passes over S in TMEM, 32 keys at a time: the largest logit, then
      // the weights. A masked key is left out of both, whatever its logit is.
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t s[32];
        load_s(tS + 32 * h, s);
        const uint32_t mk = h ? mhi : mlo;
        if (full(mk)) {
#pragma unroll
          for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(s[j]) * sl2);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            mx[j & 3] = ((mk >> j) & 1u) ? fmaxf(mx[j & 3], __uint_as_float(s[j]) * sl2) : mx[j & 3];
        }
      }
      const float m_new = fmaxf(m_run, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
      const bool need = m_new > m_run + kRescaleThreshold;  // also true when m_run == -inf
      const float m_use = need ? m_new : m_run;
      const float alpha = need ? exp2f(m_run - m_new) : 1.f;
      if (i > 0 && __any_sync(0xffffffffu, need)) {
        // rescaling O waits until PV(i - 1) has added into it
        if (!(ok = mbar_wait_warp(br.pvdone(), (i - 1) & 1, abort_flag))) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t ov[32];
          tmem_ld32(tmem + lane_base + kColO + c * 32, ov);
          tmem_ld_wait_regs(ov);
#pragma unroll
          for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
          tmem_st32(tmem + lane_base + kColO + c * 32, ov);
        }
        tmem_st_wait();
      }
      const uint64_t sl2x2 = f32x2_pack(sl2, sl2), nm2 = f32x2_pack(-m_use, -m_use);
      uint64_t ps2[2] = {0ull, 0ull};  // packed (0.f, 0.f)
      // P goes over the halves of S that both passes have read: columns 0-31,
      // or for the upper value half columns 32-63, starting with S's upper half
      const int upper = kBoth ? r >> 6 : 0;
#pragma unroll 1
      for (int hh = 0; hh < 2; ++hh) {
        const int h = hh ^ upper;
        uint32_t s[32], pw[16];
        load_s(tS + 32 * h, s);
        const uint32_t mk = h ? mhi : mlo;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          float x0, x1;
          f32x2_unpack(ffma2(f32x2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sl2x2, nm2), x0, x1);
          s[2 * c] = __float_as_uint(ex2_approx(x0));
          s[2 * c + 1] = __float_as_uint(ex2_approx(x1));
        }
        if (!full(mk)) {
#pragma unroll
          for (int j = 0; j < 32; ++j) s[j] = ((mk >> j) & 1u) ? s[j] : 0u;
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float p0 = __uint_as_float(s[2 * c]), p1 = __uint_as_float(s[2 * c + 1]);
          ps2[c & 1] = fadd2(ps2[c & 1], f32x2_pack(p0, p1));
          __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);  // P as a bf16 operand
          pw[c] = *reinterpret_cast<uint32_t*>(&b2);
        }
        tmem_st16(tS + 32 * upper + 16 * h, pw);
      }
      if (kBoth) {  // the other half's P has zeros in this row
        const uint32_t zero[16] = {};
        tmem_st16(tS + 32 * (upper ^ 1), zero);
        tmem_st16(tS + 32 * (upper ^ 1) + 16, zero);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(br.pfull(i & 1));
      float pa, pb;
      f32x2_unpack(fadd2(ps2[0], ps2[1]), pa, pb);
      l_run = l_run * alpha + (pa + pb);
      m_run = m_use;
      n = i + 1;
    }
    // -------------------------------------------------------------- epilogue
    if (ok && n > 0) ok = mbar_wait_warp(br.pvdone(), (n - 1) & 1, abort_flag);
    tc_fence_after();
    const bool have_o = n > 0 && ok;
    const bool some = l_run != 0.f;  // a sum of weights is never negative; NaN counts
    const float inv_l = some ? (k4 ? 128.f : 1.f) / l_run : 0.f;
    const float lse_v = some ? (m_run + log2f(l_run)) * 0.69314718055994531f : -INFINITY;
    auto load_o = [&](int c0, uint32_t (&o)[32]) {
      if (have_o) {
        tmem_ld32(tmem + lane_base + kColO + c0, o);
        tmem_ld_wait_regs(o);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = 0u;
      }
    };
    if (prm.nsplit == 1) {
      // the warp stages its 32 rows as bf16 in the idle key stages and writes
      // them one contiguous 512-byte row at a time
      uint8_t* stg = smem + OFF_K + (warp & 3) * (32 * kOutLd);
#pragma unroll 1
      for (int c0 = 0; c0 < 256; c0 += 32) {
        uint32_t o[32];
        load_o(c0, o);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[8 * j + 2 * e]) * inv_l,
                                                      __uint_as_float(o[8 * j + 2 * e + 1]) * inv_l);
            pk[e] = *reinterpret_cast<uint32_t*>(&b2);
          }
          *reinterpret_cast<uint4*>(stg + lane * kOutLd + c0 * 2 + j * 16) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      }
      __syncwarp();
      const int w0 = (warp & 3) * 32 % kRows, nw = min(32, rows - w0);
      uint16_t* orow = prm.o + ((size_t)first_row + w0) * kDv + value_half((warp & 3) * 32) * 256;
#pragma unroll 4
      for (int i = 0; i < nw; ++i)
        reinterpret_cast<uint4*>(orow + (size_t)i * kDv)[lane] =
            *reinterpret_cast<const uint4*>(stg + i * kOutLd + lane * 16);
      if (value_half(r) == 0 && r < rows && prm.lse) prm.lse[(size_t)first_row + r] = lse_v;
    } else {
      // split keys: normalised partial rows and their log-sums in shared
      // memory (the queries' and keys' places, idle after the last PV)
      float4* row = reinterpret_cast<float4*>(smem + r * (kStageLd * 4));
#pragma unroll 1
      for (int c0 = 0; c0 < 256; c0 += 32) {
        uint32_t o[32];
        load_o(c0, o);
#pragma unroll
        for (int v = 0; v < 8; ++v)
          row[c0 / 4 + v] =
              make_float4(__uint_as_float(o[4 * v]) * inv_l, __uint_as_float(o[4 * v + 1]) * inv_l,
                          __uint_as_float(o[4 * v + 2]) * inv_l, __uint_as_float(o[4 * v + 3]) * inv_l);
      }
      reinterpret_cast<float*>(smem + OFF_LSE)[r] = lse_v;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    if (*abort_flag && lane == 0) {
      set_status(prm.dev_status, DSA_STATUS_TIMEOUT);
      mbar_wait_drain(br.qbar(), 0);  // the query copy must not land after the CTA has gone
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (prm.nsplit > 1) {
    // Every CTA of the cluster merges its share of the head rows out of all
    // CTAs' shared memory, the splits in the order 0, 1, ..., whichever CTA
    // merges. A warp takes whole rows, 32 lanes over consecutive 16 bytes.
    __syncwarp();
    cluster_sync_all();
    const int Z = prm.nsplit, share = kHeads / Z, row0 = split * share;
    // lanes row0 .. row0 + share - 1; with kBoth they are rows of one value half
    const int out0 = row0 % kRows, nrows = max(0, min(share, rows - out0)), vh = value_half(row0);
    const uint32_t smem0 = smem_u32(smem);
    float* wts = reinterpret_cast<float*>(smem + OFF_WTS);
    if (tid < nrows) {
      float lz[kMaxSplits], mx = -INFINITY, tot = 0.f;  // all loads in flight at once
#pragma unroll
      for (int z = 0; z < kMaxSplits; ++z)
        lz[z] = z < Z ? ld_cluster_f32(cluster_addr(smem0 + OFF_LSE + (row0 + tid) * 4, z)) : -INFINITY;
#pragma unroll
      for (int z = 0; z < kMaxSplits; ++z) mx = fmaxf(mx, lz[z]);
#pragma unroll
      for (int z = 0; z < kMaxSplits; ++z) {
        // a split without keys weighs nothing; NaN stays NaN
        lz[z] = lz[z] == -INFINITY ? 0.f : exp2f((lz[z] - mx) * 1.4426950408889634f);
        tot += lz[z];
      }
      const bool some = tot != 0.f;
      const float inv = some ? 1.f / tot : 0.f;
#pragma unroll
      for (int z = 0; z < kMaxSplits; ++z) wts[z * kHeads + tid] = lz[z] * inv;
      if (vh == 0 && prm.lse)
        prm.lse[(size_t)first_row + out0 + tid] = some ? mx + logf(tot) : -INFINITY;
    }
    __syncthreads();
    uint16_t* orow = prm.o + ((size_t)first_row + out0) * kDv + vh * 256;
#pragma unroll 1
    for (int i = warp; i < nrows; i += kThreads<kCache> / 32) {
      float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
      const uint32_t src = smem0 + (row0 + i) * (kStageLd * 4) + lane * 16;
#pragma unroll 4
      for (int z = 0; z < Z; ++z) {
        const uint32_t a = cluster_addr(src, z);
        const float w = wts[z * kHeads + i];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 v = ld_cluster_v4(a + 512 * k);
          acc[k].x = fmaf(w, v.x, acc[k].x);
          acc[k].y = fmaf(w, v.y, acc[k].y);
          acc[k].z = fmaf(w, v.z, acc[k].z);
          acc[k].w = fmaf(w, v.w, acc[k].w);
        }
      }
      uint2* dst = reinterpret_cast<uint2*>(orow + (size_t)i * kDv);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        __nv_bfloat162 lo = __floats2bfloat162_rn(acc[k].x, acc[k].y), hi = __floats2bfloat162_rn(acc[k].z, acc[k].w);
        dst[32 * k + lane] = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while another reads its rows
  }
}

using Kernel = void (*)(AttendParams, CUtensorMap, CUtensorMap);

// How many clusters of 2^lz CTAs the current device runs at once (a cluster
// lies in one GPC, so this is less than SMs / 2^lz); asked once per device.
int clusters_at_once(Kernel kern, bool k4, bool both, int lz) {
  static std::atomic<int> cached[64][4][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::atomic<int>& slot = cached[dev][2 * both + k4][lz];
  int n = slot.load(std::memory_order_relaxed);
  if (n) return n - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1 << lz);
  cfg.blockDim = dim3(k4 ? kThreads<kCache4Bit> : kThreads<kCacheBf16>);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1 << lz;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  slot.store(n + 1, std::memory_order_relaxed);
  return n;
}

// Splits of a list of n entries (tokens, or pages of ps keys): a power of two
// up to eight, as long as all clusters run at once, 64 keys are left for each
// split on average (128 among eight) and the longest share gets shorter: pages
// are dealt out whole, so one page is not split. Measured, 4-bit cache, z = 1 /
// 2 / 4 / 8, 128 heads: one request of 128 keys 12.5 / 13.4 / 14.3 / 16.6 us,
// 256 keys 17.1 / 15.7 / 14.6 / 16.8, 1024 keys 40.9 / 28.0 / 20.9 / 19.1, 8
// requests of 2048 keys 72.4 / 44.2 / 29.4 / 46.2 (16 clusters of eight are more
// than fit); 16 heads, one request of 128 keys 11.7 / 11.6 / 11.5 / 13.0, 256
// keys 16.1 / 13.8 / 11.9 / 12.9. One page of 128 keys, 8 requests: 13.7 us in
// two splits and 10.8 in one with 128 heads, 12.1 and 10.1 with 16.
int log2_splits(Kernel kern, bool k4, bool both, long long clusters, long long n, int unit) {
  const auto longest = [&](int lz) { return (n + (1 << lz) - 1) >> lz; };
  int lz = 0;
  while (lz < 3 && ((n * unit) >> (lz + 1)) >= (lz == 2 ? 128 : 64) && longest(lz + 1) < longest(lz) &&
         clusters <= clusters_at_once(kern, k4, both, lz + 1))
    ++lz;
  return lz;
}
}  // namespace

int run_attend_cache(cudaStream_t stream, AttendParams prm) {
  if (prm.T == 0 || prm.H == 0) return DSA_OK;
  if (prm.ps < kSubKeys || (prm.ps & (prm.ps - 1))) return DSA_ERR_UNSUPPORTED;  // pages: 2^n rows, n >= 5
  const bool k4 = prm.kv4 != nullptr;
  CUtensorMap kvmap{}, qmap;  // kvmap: the bf16 cache; 4-bit rows are read without one
  if (!k4 && !encode_bf16_2d(&kvmap, prm.kv, (uint64_t)prm.P * prm.ps, (uint64_t)prm.row_stride, kSubKeys, kDk))
    return DSA_ERR_CUDA;
  // Neighbouring tokens share a CTA where they fit and a request has two on
  // average: 2049 tokens, window 1024: 134 us with eight tokens a CTA against
  // 597 with one for 16 heads, 461 against 611 for 64, 20 against 590 for one.
  // A CTA finds its run by a scan over the requests, 32 at a time, which 1024 of
  // them bound.
  prm.pack = !k4 && prm.H <= kHeads / 2 && prm.S <= 1024 && prm.T >= 2 * prm.S ? kHeads / prm.H : 1;
  const long long runs = std::min<long long>(prm.T, (prm.T + (long long)prm.S * (prm.pack - 1)) / prm.pack);
  // One CTA per token of up to 64 heads (kBoth) does twice the PV work and
  // takes 1.1 to 1.2 times as long, so it is taken where two CTAs per token in
  // as many splits would not all run at once. Measured with two / one, 4-bit
  // cache, 2048 keys each, 64 heads: 1 request 20.6 / 24.4 us, 16 requests 29.0
  // / 32.8, 48 requests 73.3 / 51.9; 16 heads: 1 request 19.5 / 20.7, 8 requests
  // 27.0 / 21.7, 32 requests 43.5 / 31.1; window 4096 and 64 sinks, 32 requests
  // of 16 heads 67.4 / 57.8.
  const auto choose = [&](bool one) -> Kernel {
    if (k4) return one ? cache_mla_kernel<kCache4Bit, true> : cache_mla_kernel<kCache4Bit, false>;
    return one ? cache_mla_kernel<kCacheBf16, true> : cache_mla_kernel<kCacheBf16, false>;
  };
  const int unit = prm.mode == kModeToken ? 1 : prm.ps;
  bool both = prm.H <= kHeads / 2 && prm.pack == 1;
  int lz = 0;
  if (both) {
    for (const bool one : {false, true}) set_smem_attr_once(reinterpret_cast<const void*>(choose(one)), kSmem);
    lz = log2_splits(choose(true), k4, true, runs, prm.K, unit);
    both = 2 * runs > clusters_at_once(choose(false), k4, false, lz);
  }
  const Kernel kern = choose(both);
  set_smem_attr_once(reinterpret_cast<const void*>(kern), kSmem);
  const int cols = both ? 1 : 2 * ((prm.H + kHeads - 1) / kHeads);
  if (!both) lz = log2_splits(kern, k4, false, cols * runs, prm.K, unit);
  prm.nsplit = 1 << lz;
  if (!encode_bf16_2d(&qmap, prm.q, (uint64_t)prm.T * prm.H, kDk, both ? kHeads / 2 : kHeads, kDk)) return DSA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cols, (unsigned)runs, prm.nsplit);
  cfg.blockDim = dim3(k4 ? kThreads<kCache4Bit> : kThreads<kCacheBf16>);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = prm.nsplit;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, prm, kvmap, qmap) != cudaSuccess) {
    (void)cudaGetLastError();
    return DSA_ERR_CUDA;
  }
  note_launch();
  return DSA_OK;
}

}  // namespace dsa
