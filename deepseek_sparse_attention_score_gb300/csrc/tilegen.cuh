// The key lists of the attention kernels: which cache rows a CTA visits.
#pragma once
#include "attend.cuh"
#include "common.cuh"

namespace dsa {

constexpr int kSubKeys = 32;  // keys resolved per generator step

// What a kernel instantiation reads: the bf16 cache (every mode), the same
// with a window and sinks (dense mode), or the 4-bit cache (token and page
// modes).
enum : int { kCacheBf16 = 0, kCacheBf16Window = 1, kCache4Bit = 2 };

// Warp-wide generator of 32-key tiles. Every lane gets the flat physical row
// of "its" key (or -1) and the ballot of valid keys; returns false when the
// CTA's key list is exhausted. Runs on one full warp. Loads are batched so a
// whole window of selections (8 x 32 token entries, or 32 pages / union
// slots) resolves to physical rows in two or three dependent global loads.
template <int kCache>
struct TileGen {
  static constexpr int GB = 8;  // token windows resolved per refill
  const AttendParams* p;
  int mode, t, seq, pos, kv_len, n_vis, page_base;
  int e, e1;          // token / page modes: next entry, end of this CTA's range
  int win;            // page / qblock: start of the next 32-window
  // token mode: buffered tiles
  int buf_row[GB];
  uint32_t buf_mask[GB];
  uint32_t buf_pend;  // windows of the buffer with keys, not returned yet
  // page / qblock modes: current window
  uint32_t pend;      // units of the window still to visit
  int w_key0;         // this lane's unit: first key position (page) or kp base (qblock)
  int w_phys;         // this lane's unit: physical page, -1 if none
  int cur_key0, cur_phys, sub, cur_valid;
  int b, qq, cnt;     // qblock
  int ps_log2;        // the page size is a power of two
  int key_lo;         // dense: first key position inside the window
  int n_sink, p_skip; // with sinks: pages listed before the window's, pages skipped after them

  __device__ void init(const AttendParams& prm, int tok, int split) {
    p = &prm;
    mode = prm.mode;
    ps_log2 = 31 - __clz(prm.ps);
    t = tok;
    const int sq = seq_of_token_warp(prm.cu_q_lens, prm.S, tok);
    TokenGeom g = token_geom(prm.seq_lens, prm.cu_q_lens, prm.cu_kv_lens, prm.S, prm.ps, 0x3fffffff, tok,
                             prm.dev_status, sq);
    seq = g.seq;
    pos = g.pos;
    kv_len = g.kv_len;
    n_vis = g.n_vis;
    page_base = g.page_base;
    buf_pend = 0;
    pend = 0;
    sub = 0;
    cur_valid = 0;
    key_lo = 0;
    if (mode == kModeDense) {
      // every page that holds a visible position inside the window, split
      // evenly across the CTAs of this token
      key_lo = prm.window > 0 ? max(0, pos - prm.window + 1) : 0;
      int p_lo = key_lo / prm.ps, p_hi = (n_vis + prm.ps - 1) / prm.ps;
      if constexpr (kCache == kCacheBf16Window) {
        // the list is the sinks' pages below the window, then the window's
        n_sink = (int)min((long long)p_lo, ((long long)prm.sinks + prm.ps - 1) / prm.ps);
        p_skip = p_lo - n_sink;
        p_lo = 0;
        p_hi -= p_skip;
      }
      const int per = (max(0, p_hi - p_lo) + prm.nsplit - 1) / prm.nsplit;
      e = min(p_hi, p_lo + split * per);
      e1 = min(p_hi, e + per);
      win = e;
    } else if (mode == kModeQblock) {
      b = tok / prm.QB;
      qq = tok % prm.QB;
      cnt = min(__ldg(prm.counts + b), prm.u_max);
      win = 0;
    } else {
      int per = ((prm.K + prm.nsplit - 1) / prm.nsplit + 31) & ~31;
      // pages are 32 keys at least: a share need not be a whole window of 32
      if constexpr (kCache == kCache4Bit)
        if (mode == kModePage) per = (prm.K + prm.nsplit - 1) / prm.nsplit;
      e = split * per;
      e1 = min(prm.K, e + per);
      win = e;
    }
  }

  // physical page of packed page-table entry `ent` (checked), or -1
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

  // base: first physical row of the tile when its 32 keys are 32 consecutive
  // rows of one page (page and qblock modes), else -1
  __device__ bool next(long long& row, uint32_t& mask, long long& base) {
    const int lane = lane_id();
    const int ps = p->ps;
    base = -1;
    if (kCache != kCacheBf16Window && mode == kModeToken) {
      while (!buf_pend) {
        if (e >= e1) return false;
        int j[GB];
#pragma unroll
        for (int g = 0; g < GB; ++g) {
          const int ee = e + 32 * g + lane;
          j[g] = ee < e1 ? __ldg(p->sel + (size_t)t * p->K + ee) : -1;
        }
        int pg[GB];
#pragma unroll
        for (int g = 0; g < GB; ++g) pg[g] = (j[g] >= 0 && j[g] < n_vis) ? page_of(page_base + (j[g] >> ps_log2)) : -1;
        // every array index below is a compile-time constant, so the buffer
        // stays in registers
#pragma unroll
        for (int g = 0; g < GB; ++g) {
          const bool v = pg[g] >= 0;
          const uint32_t m = __ballot_sync(0xffffffffu, v);
          buf_row[g] = v ? pg[g] * ps + (j[g] & (ps - 1)) : -1;
          buf_mask[g] = m;
          buf_pend |= (m ? 1u : 0u) << g;
        }
        e += 32 * GB;
      }
      const int gsel = __ffs(buf_pend) - 1;
      buf_pend &= buf_pend - 1u;
      int r = -1;
      uint32_t m = 0;
#pragma unroll
      for (int g = 0; g < GB; ++g)
        if (g == gsel) {
          r = buf_row[g];
          m = buf_mask[g];
        }
      row = r;
      mask = m;
      return true;
    }
    const int tiles_per_unit = ps / kSubKeys;
    while (true) {
      if (cur_valid && sub < tiles_per_unit) {
        const int k0 = sub * kSubKeys + lane;
        bool v;
        if (kCache == kCache4Bit || (kCache == kCacheBf16 && mode == kModePage)) {
          v = cur_key0 + k0 < n_vis;
        } else if (kCache == kCacheBf16Window) {
          v = cur_key0 + k0 < n_vis && (cur_key0 + k0 >= key_lo || cur_key0 + k0 < p->sinks);
        } else if (mode == kModeDense) {
          v = cur_key0 + k0 < n_vis && cur_key0 + k0 >= key_lo;
        } else {
          const int kp = cur_key0 + k0;  // kp = g*ps + r - base_tok
          v = kp <= pos && kp < kv_len;
        }
        base = (long long)cur_phys * ps + sub * kSubKeys;
        ++sub;
        row = v ? (long long)cur_phys * ps + k0 : -1;
        mask = __ballot_sync(0xffffffffu, v);
        if (mask) return true;
        continue;
      }
      cur_valid = 0;
      sub = 0;
      if (!pend) {
        // resolve a window of 32 candidate units to physical pages
        if (kCache == kCacheBf16Window || (kCache == kCacheBf16 && mode == kModeDense)) {
          if (win >= e1) return false;
          int pgl = win + lane;
          const bool in = pgl < e1;
          if constexpr (kCache == kCacheBf16Window) pgl += pgl < n_sink ? 0 : p_skip;
          w_phys = in ? page_of(page_base + pgl) : -1;
          w_key0 = pgl * ps;
        } else if (kCache == kCache4Bit || mode == kModePage) {
          if (win >= e1) return false;
          const int ee = win + lane;
          const int pgl = ee < e1 ? __ldg(p->sel + (size_t)t * p->K + ee) : -1;
          const bool v = pgl >= 0 && (long long)pgl * ps < n_vis;
          w_phys = v ? page_of(page_base + pgl) : -1;
          w_key0 = pgl * ps;
        } else {
          if (win >= cnt) return false;
          const int u = win + lane;
          bool has = false;
          int g = -1;
          if (u < cnt) {
            const uint32_t wd = __ldg(p->member + ((size_t)b * p->u_max + u) * (p->QB / 32) + (qq >> 5));
            g = __ldg(p->units + (size_t)b * p->u_max + u);
            has = (wd >> (qq & 31)) & 1u;
          }
          w_phys = has ? page_of(g) : -1;
          w_key0 = (g - page_base) * ps;
        }
        pend = __ballot_sync(0xffffffffu, w_phys >= 0);
        win += 32;
        continue;
      }
      const int bit = __ffs(pend) - 1;
      pend &= pend - 1u;
      cur_phys = __shfl_sync(0xffffffffu, w_phys, bit);
      cur_key0 = __shfl_sync(0xffffffffu, w_key0, bit);
      cur_valid = 1;
    }
  }
};

}  // namespace dsa
