/*
 * dsa.h - C ABI of the GB300 (sm_103a) DeepSeek-Sparse-Attention hot path.
 *
 * The operations follow the sglang-jax DSA pages:
 *   "ref.py" (jnp reference implementations): build_index_share_map,
 *       streamindex_topk_ref, streamindex_page_topk_ref, sparse_mla_ref;
 *   "sparse_mla_prefill_qblock.py" (blocked sparse-MLA prefill):
 *       build_block_unit_tables, _qblock_kernel, sparse_mla_attention_qblock;
 *   "dsa_sparse_backend.py" (DSA sparse attention backend): IndexShare and the
 *       page budgets.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Memory.   Every tensor pointer is a DEVICE pointer owned by the caller,
 *           except where an argument is marked "host". The library allocates
 *           no memory: scratch space is a caller-provided workspace whose size
 *           the matching *_workspace_size() call reports.
 * Streams.  Every device entry point only enqueues kernels on `stream` (a
 *           cudaStream_t; NULL is the legacy default stream) and never
 *           synchronises, so calls may be captured in a CUDA graph.
 * dtypes.   bf16 tensors are passed as uint16_t (the raw bit pattern);
 *           metadata is int32.
 * Ragged batch metadata (identical for all calls, "D4" of the pages):
 *   seq_lens     [S]    kv length of request s, INCLUDING its new tokens;
 *   cu_q_lens    [S+1]  query-token offsets (cu_q_lens[S] == T);
 *   cu_kv_lens   [S+1]  cumulative page-aligned kv lengths; request s owns the
 *                       packed page-table entries starting at cu_kv_lens[s]/ps;
 *   page_indices [PTW]  physical page of every packed page-table entry, < P.
 *   Query token t of request s sits at absolute position
 *   pos(t) = seq_lens[s] - q_len(s) + (t - cu_q_lens[s]); it sees the key
 *   positions j with j < seq_lens[s] and j <= pos(t) (causal + kv_len mask).
 * Padding.  Unused index slots are -1. Selected sets are written in
 *           ascending index order.
 * Status.   Host-detected errors return a negative DSA_ERR_* code and enqueue
 *           nothing. Conditions detected on the device are OR-ed into the
 *           optional `dev_status` word (device int32, may be NULL): the
 *           offending access is skipped, never trapped.
 */
#ifndef DSA_H_
#define DSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define DSA_API __attribute__((visibility("default")))
#else
#define DSA_API
#endif

typedef void* dsa_stream_t; /* a cudaStream_t */

enum dsa_error {
  DSA_OK = 0,
  DSA_ERR_INVALID_ARGUMENT = -1, /* null pointer, negative size, T != ... */
  DSA_ERR_UNSUPPORTED = -2,      /* a shape this build does not implement */
  DSA_ERR_WORKSPACE = -3,        /* workspace missing or too small */
  DSA_ERR_CUDA = -4,             /* a CUDA call or kernel launch failed */
  DSA_ERR_SHARED_BEFORE_FULL = -5,
  DSA_ERR_BAD_INDEXER_TYPE = -6,
  DSA_ERR_ALIGNMENT = -7,    /* a pointer is not 16-byte aligned */
  DSA_ERR_SCRATCH_LIMIT = -8 /* needs more than the built-in scratch of
                                dsa_sparse_mla_decode_noalloc (24 MiB) */
};

/* Bits OR-ed into *dev_status by the kernels. */
#define DSA_STATUS_UNION_TRUNCATED 0x1 /* a block's union exceeded u_max */
#define DSA_STATUS_BAD_METADATA 0x2    /* ragged metadata out of range */
#define DSA_STATUS_BAD_INDEX 0x4       /* a selected unit or page id out of range */
#define DSA_STATUS_TIMEOUT 0x8         /* a pipeline wait gave up (about 2 s) */
#define DSA_STATUS_INTERNAL 0x10       /* a launch-time invariant failed on the device */
#define DSA_STATUS_NO_PAGES 0x20       /* the free list holds fewer pages than a step takes */

/* ------------------------------------------------------------------------
 * IndexShare layer -> slot map (host only).
 * ref.py, build_index_share_map: a full layer (type 0) opens a new indexer
 * slot; a shared layer (type 1) consumes the slot of the nearest preceding
 * full layer and runs no indexer. types == NULL means every layer is full.
 * skip_offset is accepted and ignored, as on the page.
 *   types      host int32 [num_layers] (0 = full, 1 = shared) or NULL
 *   full_slot  host int32 [num_layers] out: slot of a full layer, -1 otherwise
 *   src_slot   host int32 [num_layers] out: slot whose top-k the layer uses
 *   num_full   host int32 out: number of full layers (= indexer key caches)
 * Errors: DSA_ERR_SHARED_BEFORE_FULL, DSA_ERR_BAD_INDEXER_TYPE.
 * ------------------------------------------------------------------------ */
DSA_API int dsa_index_build_share_map(const int32_t* types, int num_layers, int skip_offset, int32_t* full_slot,
                              int32_t* src_slot, int32_t* num_full);

/* ------------------------------------------------------------------------
 * Lightning indexer + exact token top-k.
 * ref.py, streamindex_topk_ref: s[t,j] = sum_h relu(q[t,h,:] . k[j,:]) * w[t,h]
 * accumulated in fp32 over the visible prefix j < min(seq_lens[s], pos(t)+1);
 * then the k highest-scoring visible positions, ties to the lower index
 * (exact: the pages' approximate top-k is not used).
 *   q        bf16 [T, Hi, Di]       indexer queries
 *   w        fp32 [T, Hi]           head weights (any scale folded in)
 *   kcache   bf16 [P, ps, Di]       paged indexer keys
 *   max_kv   upper bound of seq_lens (sizes the score workspace); a larger
 *            seq_len is clamped and flagged DSA_STATUS_BAD_METADATA
 *   topk     int32 [T, k] out       ascending positions, -1 padded
 *   topk_scores fp32 [T, k] out or NULL: the scores of `topk` (-inf on pads)
 *   ws/ws_bytes  workspace of dsa_indexer_workspace_size(T, S, max_kv, ps) bytes
 * Supported: Hi == 32, Di == 128, ps in {32, 64, 128}, 1 <= k.
 * ------------------------------------------------------------------------ */
DSA_API size_t dsa_indexer_workspace_size(int T, int S, int max_kv, int ps);
DSA_API int dsa_indexer_topk(dsa_stream_t stream, const uint16_t* q, const float* w, const uint16_t* kcache,
                     const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                     const int32_t* page_indices, int T, int S, int P, int PTW, int ps, int Hi, int Di, int max_kv,
                     int k, int32_t* topk, float* topk_scores, void* ws, size_t ws_bytes, int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Lightning indexer + page top-k (and, optionally, the token top-k from the
 * same score pass).
 * ref.py, streamindex_page_topk_ref: the token scores are max-pooled per page
 * of ps positions (masked positions excluded), then the k_pages best pages
 * are kept (ties to the lower page); pages with no visible position are never
 * selected. Page ids are sequence-local; unused slots are -1.
 * The prefill budget of dsa_sparse_backend.py is k_pages = ceil(k / ps); the
 * decode page budget is min(budget, pages_per_seq).
 *   topk_pages  int32 [T, k_pages] out
 *   k, topk, topk_scores  as dsa_indexer_topk; topk == NULL skips the token
 *               top-k (k is then ignored).
 * ------------------------------------------------------------------------ */
DSA_API int dsa_indexer_page_topk(dsa_stream_t stream, const uint16_t* q, const float* w, const uint16_t* kcache,
                          const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                          const int32_t* page_indices, int T, int S, int P, int PTW, int ps, int Hi, int Di,
                          int max_kv, int k_pages, int32_t* topk_pages, int k, int32_t* topk, float* topk_scores,
                          void* ws, size_t ws_bytes, int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Per-query-block union of selected units and the membership bitmap.
 * sparse_mla_prefill_qblock.py, build_block_unit_tables (plus the lift of
 * sparse_mla_attention_qblock's ragged mode): token t's sequence-local page
 * ids p >= 0 become global page-table keys g = cu_kv_lens[seq(t)]/ps + p
 * (cu_q_lens == NULL: ids are already global). T is padded to a multiple of
 * QB with empty rows. For block b:
 *   units   int32 [nQB, u_max]        ascending unique ids, -1 padded; a union
 *                                      larger than u_max keeps its u_max
 *                                      smallest ids and sets
 *                                      DSA_STATUS_UNION_TRUNCATED
 *   member  uint32 [nQB, u_max, QB/32] bit (q % 32) of word q/32 of slot u is
 *                                      1 iff query q of the block selected
 *                                      units[b, u] (slot-major, bit-packed)
 *   counts  int32 [nQB]               true (uncapped) union size
 * with nQB = ceil(T / QB). u_max <= 0 selects the lossless bound
 * min(QB * K, PTW); the outputs must then be sized with that value.
 *   topk_units int32 [T, K]  selected units per query, -1 padded
 * Supported: QB % 32 == 0, QB <= 1024. Needs no workspace.
 * ------------------------------------------------------------------------ */
DSA_API int dsa_build_block_union(dsa_stream_t stream, const int32_t* topk_units, int T, int K, int QB, int u_max,
                          const int32_t* cu_q_lens, const int32_t* cu_kv_lens, int S, int ps, int PTW,
                          int32_t* units, uint32_t* member, int32_t* counts, int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Sparse absorbed-MLA attention over per-query selections (decode form).
 * ref.py, sparse_mla_ref: for query t and head h,
 *   o[t,h,:] = sum_j softmax_j(sm_scale * q[t,h,:Dk] . kv[j,:Dk]) kv[j,:Dv]
 * over the selected positions j that are visible (j < seq_len, j <= pos(t));
 * the value is the first Dv columns of the same latent row. A query with no
 * visible selected key outputs 0 (lse = -inf). Logits and softmax in fp32,
 * output rounded to bf16.
 *   q      bf16 [T, H, Dk]               [q_nope | q_rope]
 *   kv     bf16 [P, ps, row_stride]      [c_kv(Dv) | k_rope | pad]
 *   sel    int32 [T, K]  unit == 1: token positions; unit == ps: sequence-
 *                        local page ids (each expands to ps positions);
 *                        -1 entries are ignored, order does not matter
 *   o      bf16 [T, H, Dv] out
 *   lse    fp32 [T, H] out or NULL: natural-log sum of exp of the logits
 *   ws     workspace of dsa_sparse_mla_decode_workspace_size(T, H, Dv) bytes
 *          (split-key partials; 0 bytes needed when T*H is large)
 * Supported: Dk == 576, Dv == 512, row_stride in {576, 640}, ps in
 * {32, 64, 128}, H >= 1 (heads are processed 128 at a time), T <= 65535 (this
 * and every attention entry below).
 * Cache contents: with page units (and in the query-block and dense forms)
 * whole runs of 32 rows of each selected page are read and the rows past
 * the visible length are masked with a probability of exactly 0, so those
 * rows (the unwritten tail of a request's last page) must hold finite values
 * (0 x NaN is NaN), as in the pages' kernels; token units read only the
 * selected rows.
 * Reproducibility: every output is the same on every run: when a row's
 * keys are split across CTAs (few queries, long selections) the merging CTA
 * adds the splits in a fixed order, whichever CTA of the row finishes last.
 * ------------------------------------------------------------------------ */
DSA_API size_t dsa_sparse_mla_decode_workspace_size(int T, int H, int Dv);
DSA_API int dsa_sparse_mla_decode(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv, int row_stride,
                          const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                          const int32_t* page_indices, const int32_t* sel, int K, int unit, int T, int S, int P,
                          int PTW, int ps, int H, int Dk, int Dv, float sm_scale, uint16_t* o, float* lse,
                          void* ws, size_t ws_bytes, int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Sparse MLA decode without any allocation or caller workspace.
 * The source pages have no counterpart of this entry point. It is for
 * callers that cannot allocate device memory on this path: for example a
 * plugin that an inference engine hands only its input and output buffers,
 * or code that must not allocate once it is running. It computes the same
 * result as dsa_sparse_mla_decode (same arguments minus the workspace);
 * when the key list is split across CTAs, the split partials live in a
 * 24 MiB device array built into the library instead of a workspace.
 *  - Memory: nothing is allocated. The array is part of the library image,
 *    so every GPU that loads the library holds it until the process exits.
 *  - Set-up: the first call on a device looks up the array's address on that
 *    device; make that first call before any stream capture.
 *  - Sharing: all calls use the same array and leave their last contents in
 *    it (the merge counters are cleared on every call). Calls that overlap on
 *    the GPU (other streams, other host threads) race on the array, so
 *    serialise them.
 *  - Limit: a problem whose split scratch would exceed 24 MiB returns
 *    DSA_ERR_SCRATCH_LIMIT and enqueues nothing; use dsa_sparse_mla_decode
 *    with a workspace for it. Only devices 0..63 are served: on a device
 *    with a higher ordinal a call that needs the array returns DSA_ERR_CUDA.
 * ------------------------------------------------------------------------ */
DSA_API int dsa_sparse_mla_decode_noalloc(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv,
                                          int row_stride, const int32_t* seq_lens, const int32_t* cu_q_lens,
                                          const int32_t* cu_kv_lens, const int32_t* page_indices, const int32_t* sel,
                                          int K, int unit, int T, int S, int P, int PTW, int ps, int H, int Dk, int Dv,
                                          float sm_scale, uint16_t* o, float* lse, int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Query-block sparse-MLA prefill over the block unions.
 * sparse_mla_prefill_qblock.py, _qblock_kernel / sparse_mla_attention_qblock:
 * query t of block b = t / QB walks the slots u < min(counts[b], u_max) of its
 * block; unit g = units[b,u] is physical page page_indices[g] whose row r is
 * key position kp = g*ps + r - (cu_kv_lens[seq(t)]/ps)*ps, visible iff the
 * membership bit of (u, t % QB) is set and kp <= pos(t) and kp < seq_len.
 * Same masked-softmax math and output as dsa_sparse_mla_decode with page
 * units (the pages' parity claim between the blocked and per-query kernels).
 *   units/member/counts  as written by dsa_build_block_union (same QB, u_max)
 *   o      bf16 [T, H, Dv] out; lse fp32 [T, H] out or NULL
 * Supported: as dsa_sparse_mla_decode. Needs no workspace.
 * ------------------------------------------------------------------------ */
DSA_API int dsa_sparse_mla_prefill_qblock(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv, int row_stride,
                                  const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                                  const int32_t* page_indices, const int32_t* units, const uint32_t* member,
                                  const int32_t* counts, int QB, int u_max, int T, int S, int P, int PTW, int ps,
                                  int H, int Dk, int Dv, float sm_scale, uint16_t* o, float* lse,
                                  int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Query-block sparse-MLA prefill for a contiguous range of query tokens.
 * The pages have no counterpart of this entry point: it computes the rows
 * t_begin <= t < t_end of dsa_sparse_mla_prefill_qblock's output, with the
 * same arithmetic (bit for bit), and writes no other row. A caller that runs
 * one layer's attention in a few token ranges can start copying the finished
 * rows off the GPU while the later ranges compute.
 *   t_begin, t_end  0 <= t_begin <= t_end <= T (t_begin == t_end: nothing)
 *   every other argument as dsa_sparse_mla_prefill_qblock (q, o and lse keep
 *   their full [T, ...] extent; token t stays row t)
 * Errors: as dsa_sparse_mla_prefill_qblock; DSA_ERR_INVALID_ARGUMENT for a
 * range outside [0, T].
 * ------------------------------------------------------------------------ */
DSA_API int dsa_sparse_mla_prefill_qblock_range(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv,
                                                int row_stride, const int32_t* seq_lens, const int32_t* cu_q_lens,
                                                const int32_t* cu_kv_lens, const int32_t* page_indices,
                                                const int32_t* units, const uint32_t* member, const int32_t* counts,
                                                int QB, int u_max, int T, int S, int P, int PTW, int ps, int H,
                                                int Dk, int Dv, float sm_scale, int t_begin, int t_end, uint16_t* o,
                                                float* lse, int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Approximate token top-k (the trade the pages make with approx_max_k on
 * their fast path; ref.py, streamindex_topk_ref is the exact definition).
 * Scores as dsa_indexer_topk. A row of n visible scores is folded into
 * B = min(n, over*k) bins (bin b holds positions b, b+B, b+2B, ...); each
 * bin keeps its largest score (lowest position on ties); the selection is
 * the exact top-k of the B bin maxima (ties to the lower bin), written as
 * ascending positions, -1 padded. count = min(k, n); over*k >= n makes it
 * the exact top-k up to ties; a larger `over` raises the recall.
 *   ws  workspace of dsa_indexer_topk_approx_workspace_size(T, S, max_kv,
 *       ps, k, over) bytes
 * Supported: as dsa_indexer_topk, k <= 16384, over >= 1.
 * ------------------------------------------------------------------------ */
DSA_API size_t dsa_indexer_topk_approx_workspace_size(int T, int S, int max_kv, int ps, int k, int over);
DSA_API int dsa_indexer_topk_approx(dsa_stream_t stream, const uint16_t* q, const float* w, const uint16_t* kcache,
                                    const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                                    const int32_t* page_indices, int T, int S, int P, int PTW, int ps, int Hi,
                                    int Di, int max_kv, int k, int over, int32_t* topk, void* ws, size_t ws_bytes,
                                    int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Dense causal absorbed-MLA attention: the route the backend takes for
 * layers without an indexer (dsa_sparse_backend.py, _run_dense, which calls
 * the dense ragged paged MLA kernel with the layer's sliding window and
 * logit soft cap; that kernel's module is not shown on the pages). For query
 * t every position j with j < seq_len, j <= pos(t) and, when
 * sliding_window > 0, j > pos(t) - sliding_window; with soft_cap > 0 each
 * logit l = sm_scale * q.k becomes soft_cap * tanh(l / soft_cap) before the
 * softmax. Output and lse as dsa_sparse_mla_decode.
 *   max_kv  an upper bound on seq_lens (host-known), sizes the key splits
 *   ws      workspace of dsa_sparse_mla_decode_workspace_size(T, H, Dv) bytes
 * Supported: as dsa_sparse_mla_decode; sliding_window >= 0, soft_cap >= 0.
 * With a sliding window dsa_window_mla (num_sinks = 0) computes the same and
 * is the faster call, most of all with 64 heads or fewer, where it takes
 * neighbouring tokens together.
 * ------------------------------------------------------------------------ */
DSA_API int dsa_dense_mla(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv, int row_stride,
                          const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                          const int32_t* page_indices, int max_kv, int T, int S, int P, int PTW, int ps, int H,
                          int Dk, int Dv, float sm_scale, int sliding_window, float soft_cap, uint16_t* o,
                          float* lse, void* ws, size_t ws_bytes, int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Paged write-back of the new tokens' rows into a paged cache: the step
 * directly before the indexer and the attention, which read these rows.
 * dsa_sparse_backend.py, _scatter_paged (and the Pallas paged_write_back of
 * sparse_mla_prefill_qblock.py): query token t of request s sits at position
 * pos(t) = seq_lens[s] - q_len(s) + (t - cu_q_lens[s]) and its row is copied
 * to row pos(t) % ps of physical page page_indices[cu_kv_lens[s]/ps +
 * pos(t)/ps]. Every other cache row is left untouched.
 *   rows   bf16 [T, src_stride]  the first D columns of row t are written
 *   cache  bf16 [P, ps, cache_stride]  updated in place; the first D columns
 *          of the destination rows are overwritten
 * Use it once per cache: D = 576 for the latent [c_kv | k_rope] cache
 * (cache_stride 576 or 640), D = 128 for the indexer key cache.
 * There are no padding rows in this ABI (T == cu_q_lens[S]), so no row is
 * sent to a sentinel page: a token whose destination falls outside the page
 * table or the pool sets DSA_STATUS_BAD_METADATA and is skipped.
 * Supported: D, src_stride, cache_stride multiples of 8 (16-byte rows),
 * D <= src_stride, D <= cache_stride, rows and cache 16-byte aligned.
 * Needs no workspace. Tokens write distinct rows whenever the metadata is
 * valid (positions of one request are distinct, requests own disjoint
 * page-table entries that map to distinct pages).
 * ------------------------------------------------------------------------ */
DSA_API int dsa_paged_write_back(dsa_stream_t stream, const uint16_t* rows, int src_stride, int D, uint16_t* cache,
                                 int cache_stride, const int32_t* seq_lens, const int32_t* cu_q_lens,
                                 const int32_t* cu_kv_lens, const int32_t* page_indices, int T, int S, int P,
                                 int PTW, int ps, int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Paged write-back into two caches that share one page table, in one launch
 * (no counterpart on the pages, which write each cache separately): a
 * layer's latent rows and, on a full layer, its indexer keys. Each token's
 * slot is found once; (rows0, src_stride0, D0, cache0, cache_stride0) and
 * (rows1, ...) follow the rules of dsa_paged_write_back, and both caches
 * hold P pages of ps rows. rows1 == cache1 == NULL with D1 == 0 writes the
 * first cache alone (dsa_paged_write_back is that call). Errors as
 * dsa_paged_write_back, for either target.
 * ------------------------------------------------------------------------ */
DSA_API int dsa_paged_write_back_pair(dsa_stream_t stream, const uint16_t* rows0, int src_stride0, int D0,
                                      uint16_t* cache0, int cache_stride0, const uint16_t* rows1, int src_stride1,
                                      int D1, uint16_t* cache1, int cache_stride1, const int32_t* seq_lens,
                                      const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                                      const int32_t* page_indices, int T, int S, int P, int PTW, int ps,
                                      int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Token top-k -> page list, for the page-level decode shape of the pages.
 * dsa_sparse_backend.py, compute_topk_pages (k_pages_max = 512 there): per
 * query row, the ascending unique pages (position / ps) of the selected
 * tokens; the first `cap` of them are written, the rest of the row is -1.
 *   topk   int32 [T, K]  token positions, any order, -1 entries ignored
 *   pages  int32 [T, cap] out
 *   counts int32 [T] out or NULL: number of unique pages (not capped), so
 *          counts[t] > cap means row t was truncated
 * A position at or beyond max_pages * ps sets DSA_STATUS_BAD_INDEX and is
 * ignored. Supported: 1 <= max_pages <= 2^20, cap >= 1. Needs no workspace.
 * ------------------------------------------------------------------------ */
DSA_API int dsa_topk_pages_from_tokens(dsa_stream_t stream, const int32_t* topk, int T, int K, int ps,
                                       int max_pages, int cap, int32_t* pages, int32_t* counts,
                                       int32_t* dev_status);

/* ------------------------------------------------------------------------
 * A step's page tables from its requests' lengths (the ragged metadata that
 * every other call reads, which the pages' backend assembles on the host;
 * dsa_sparse_backend.py, _scatter_paged and _fixed_stride_pages).
 * Request s has q_lens[s] new tokens and seq_lens[s] positions with them. It
 * holds its pages in a row of `block_table`; the pages that its new tokens
 * are the first to need are taken from `free_pages` in order, request by
 * request, and written into the row. With had = ceil((seq - q) / ps) and
 * need = ceil(seq / ps):
 *   q_lens, seq_lens  int32 [S]
 *   block_table  int32 [S, bt_stride] in/out: entries [0, had) are read,
 *                [had, need) written, no others touched; the first `width`
 *                entries of a row may be used
 *   free_pages   int32 [F], NULL with F == 0 (a step that takes no page)
 *   cu_q_lens    int32 [S+1] out   cu_kv_lens  int32 [S+1] out
 *   page_indices int32 [PTW] out   packed rows, -1 behind the last
 *   token_seq, positions, slots  int32 [T] out: request, absolute position
 *                and cache slot (page * ps + row) of every token, -1 behind
 *                the last token, so T and PTW may be upper bounds
 *   n_taken      int32 [1] out     pages this step takes from the list
 * cu_q_lens, cu_kv_lens and page_indices are the metadata of the other calls
 * when T is the number of tokens. The call reads no state of its own: run
 * again on the same inputs it writes the same values. It always takes from the
 * list's first entry on: before the next step that takes pages the caller
 * passes the rest of the list, or uses dsa_build_page_tables_next.
 * Device conditions: a request with q < 0, seq < q or seq > width * ps counts
 * as empty and sets DSA_STATUS_BAD_METADATA, as do more tokens than T or more
 * pages than PTW (those past the end, and block-table entries behind them,
 * are not written); a list that runs out sets DSA_STATUS_NO_PAGES, its
 * missing pages and their slots are -1 and n_taken says how many it takes.
 * Supported: ps in {32, 64, 128}, S <= 16384, width * ps < 2^31, T and PTW
 * up to 2^30. Outputs overlap no input. Needs no workspace.
 * ------------------------------------------------------------------------ */
DSA_API int dsa_build_page_tables(dsa_stream_t stream, const int32_t* q_lens, const int32_t* seq_lens,
                                  int32_t* block_table, int64_t bt_stride, int width, const int32_t* free_pages,
                                  int F, int S, int T, int PTW, int ps, int32_t* cu_q_lens, int32_t* cu_kv_lens,
                                  int32_t* page_indices, int32_t* token_seq, int32_t* positions, int32_t* slots,
                                  int32_t* n_taken, int32_t* dev_status);
/* The same for a sequence of steps over one free list. A step's pages stay in
 * the block table and must not be handed out again, so the list goes on where
 * the last step stopped:
 *   free_state  int32 [3 + 2 S] in/out, zeros before the first step on a list
 *               (and again whenever the list is filled anew), or NULL: the
 *               call above, every step from the list's first entry
 *                 [0]  for the call's own use
 *                 [1]  entries that the steps before the last one used
 *                 [2]  entries that the last one used
 *                 [3, 3 + S) and [3 + S, 3 + 2 S)  its q_lens and seq_lens
 * A step with exactly the lengths of the last one is that step again (a retry,
 * a replay of a captured graph) and takes the same pages; any other starts
 * behind them. Where equal lengths do mean a new step (every request was
 * replaced by another of its lengths, and the old ones keep their pages), fill
 * the remembered lengths with -1. Pages of a step that is taken back stay
 * used. DSA_STATUS_NO_PAGES is set when fewer than the step takes are left.
 * Steps on one state run one after another. */
DSA_API int dsa_build_page_tables_next(dsa_stream_t stream, const int32_t* q_lens, const int32_t* seq_lens,
                                       int32_t* block_table, int64_t bt_stride, int width,
                                       const int32_t* free_pages, int F, int32_t* free_state, int S, int T, int PTW,
                                       int ps, int32_t* cu_q_lens, int32_t* cu_kv_lens, int32_t* page_indices,
                                       int32_t* token_seq, int32_t* positions, int32_t* slots, int32_t* n_taken,
                                       int32_t* dev_status);


/* ------------------------------------------------------------------------
 * Rotary positions (no counterpart on the pages, whose queries and rows
 * arrive rotated). Pair i of a row at position p turns by p * freqs[i]:
 *   (a, b) -> scale * (a cos - b sin, b cos + a sin)
 * with (a, b) the elements (2i, 2i+1) (DSA_ROPE_INTERLEAVED) or
 * (i, i + rot_dim/2) (DSA_ROPE_HALF) of columns [rot_off, rot_off + rot_dim).
 * `inverse` != 0 turns by the negative angle: that call maps an output's
 * gradient to the input's. The targets of a call are rotated in one launch (a
 * layer's queries, latent rows, indexer queries and indexer keys), in two if
 * only some of them lie on 16 bytes.
 *   x, y       [T, H, D] of `dtype` with element strides (*_stride_t,
 *              *_stride_h, 1). y == x (same strides) works in place and
 *              touches the rotated columns only; otherwise y receives the
 *              other columns too and must not overlap x. Rows of y must not
 *              overlap each other
 *   positions  int32 [T]; a row with a negative position is left as it is
 *   freqs      fp64 [rot_dim / 2], radians per position (dsa_rope_freqs)
 * Angles are reduced in fp64; products are fp32, rounded once to `dtype`.
 * Supported: 1 to 8 targets, even rot_dim <= 512, H <= 65536, D <= 4096. Any strides and alignment
 * of whole elements; a target moves 16 bytes at a time if its addresses,
 * strides, D, rot_off and rot_dim / 2 are multiples of 16 bytes, else element by
 * element.
 * ------------------------------------------------------------------------ */
enum dsa_dtype { DSA_DTYPE_BF16 = 0, DSA_DTYPE_F32 = 1 };
enum dsa_rope_layout { DSA_ROPE_INTERLEAVED = 0, DSA_ROPE_HALF = 1 };
typedef struct dsa_rope_target {
  const void* x;
  void* y;
  int64_t x_stride_t, x_stride_h, y_stride_t, y_stride_h;
  int32_t H, D, rot_off;
  int32_t layout; /* dsa_rope_layout */
  int32_t dtype;  /* dsa_dtype */
  float scale;
} dsa_rope_target;
DSA_API int dsa_rope(dsa_stream_t stream, const dsa_rope_target* targets /* host */, int n_targets, int T,
                     int rot_dim, const int32_t* positions, const double* freqs, int inverse);

/* Frequencies of the rotary pairs (host only): base^(-2i / rot_dim) radians
 * per position, scaled for contexts beyond the trained `orig_max_pos`:
 *   DSA_ROPE_SCALE_NONE    as they are (factor is ignored)
 *   DSA_ROPE_SCALE_LINEAR  divided by factor (positions interpolated)
 *   DSA_ROPE_SCALE_YARN    by parts: pairs that turn more than beta_fast
 *       times within orig_max_pos keep their frequency, those below beta_slow
 *       turns are divided by factor, a linear ramp over the pair index between
 *   freqs   host fp64 [rot_dim / 2] out
 *   mscale  host out or NULL: YaRN's factor m = 0.1 ln(factor) + 1, else 1.
 *           Its square is a temperature of the whole logit. As the scale of
 *           the rotated columns of queries and keys it is that only where all
 *           columns rotate; a head of which a part rotates (here 64 of 576
 *           columns) takes dsa_rope_attention_scales */
enum dsa_rope_scaling { DSA_ROPE_SCALE_NONE = 0, DSA_ROPE_SCALE_LINEAR = 1, DSA_ROPE_SCALE_YARN = 2 };
DSA_API int dsa_rope_freqs(int rot_dim, double base, int scaling, double factor, int orig_max_pos, double beta_fast,
                           double beta_slow, double* freqs, double* mscale);
/* YaRN's factors for a head of which only a part rotates (host only). With
 * m(c) = 0.1 c ln(factor) + 1 and a model's two coefficients (mscale and
 * mscale_all_dim of its configuration):
 *   rotated  host out: m(mscale) / m(mscale_all_dim), the scale of the rotated
 *            columns of queries and keys (dsa_rope_target.scale); 1 when the
 *            coefficients are equal
 *   logits   host out: m(mscale_all_dim)^2, the factor of sm_scale
 * factor >= 1 (1: both are 1); m(mscale_all_dim) > 0. */
DSA_API int dsa_rope_attention_scales(double factor, double mscale, double mscale_all_dim, double* rotated,
                                      double* logits);

/* ------------------------------------------------------------------------
 * 4-bit latent cache: the rows [c_kv(512) | k_rope(64)] in 416 bytes instead
 * of 1152 (no counterpart on the pages). A row:
 *   bytes   0..255  512 codes e2m1. 32-bit word w holds dims 8w .. 8w+7: the
 *                   even dims in nibbles 0..3, the odd ones in nibbles 4..7
 *   bytes 256..287  32 scales e4m3, one per 16 dims
 *   bytes 288..415  the 64 rotary dims as bf16, as they came
 * Writing: scale = max|x| / 6 rounded to e4m3, code = x / scale rounded to
 * e2m1 (both to the nearest, ties to even, saturating); the value is code *
 * scale, exact in bf16. A group with an infinity or a NaN gets the scale NaN
 * and zero codes and reads back as NaN,
 * one with max|x| <= 6 * 2^-10 as zeros. Scales below 2^-6 are subnormal and
 * coarser: 4 significant bits for max|x| >= 0.094, then 3, 2 and 1 below 0.094,
 * 0.047 and 0.024. There is no second scale: a layer whose latent rows are that
 * small is written times a power of two, with the queries' first 512 dims and
 * the output times its inverse, which changes nothing else.
 *
 * dsa_q4_write_back is dsa_paged_write_back into such a cache: token t's row
 * goes to the slot of its position, every other row is left untouched, and a
 * token without a slot sets DSA_STATUS_BAD_METADATA and is skipped. T may be
 * an upper bound: rows from cu_q_lens[S] on are padding and are ignored.
 * Tokens write distinct rows whenever the metadata is valid.
 *   rows   bf16 [T, src_stride], the first 576 columns
 *   cache  [P, ps, 416] bytes
 * dsa_q4_read_rows writes the values of N slots (page * ps + row, as
 * dsa_build_page_tables numbers them) as bf16 rows of 576 columns; a
 * negative slot gives zeros, one past the cache too and sets
 * DSA_STATUS_BAD_INDEX.
 * Supported: strides that are multiples of 8 and at least 576, 16-byte
 * aligned rows and cache, P * ps < 2^31. Need no workspace.
 * ------------------------------------------------------------------------ */
#define DSA_Q4_ROW_BYTES 416
DSA_API int dsa_q4_write_back(dsa_stream_t stream, const uint16_t* rows, int src_stride, uint8_t* cache,
                              const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                              const int32_t* page_indices, int T, int S, int P, int PTW, int ps,
                              int32_t* dev_status);
DSA_API int dsa_q4_read_rows(dsa_stream_t stream, const uint8_t* cache, int P, int ps, const int32_t* slots, int N,
                             uint16_t* rows, int dst_stride, int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Appending rows to the paged caches with the rotary positions applied on the
 * way (no counterpart on the pages, whose rows arrive rotated): dsa_rope of a
 * step's new rows and their write-back in one pass, and with it, in the same
 * launch, dsa_rope of other targets, such as the layer's queries. Row t of an append
 * target goes to cache row slots[t] (page * ps + row, as dsa_build_page_tables
 * numbers them); every other row of the cache, and the columns of a row from D
 * on, are left untouched.
 *   append     host [n_append], 1 to 4 targets; all caches have P pages of ps
 *              rows
 *     x, x_stride          bf16 [T, D]; with x_rot, [T, D - rot_dim]: the
 *                          columns that do not rotate, without a gap
 *     x_rot, x_rot_stride  bf16 [T, rot_dim]: the rotated columns when they are
 *                          a tensor of their own, else NULL
 *     cache, cache_stride  DSA_CACHE_BF16: bf16 [P, ps, cache_stride], written
 *                          in place; DSA_CACHE_Q4: bytes [P, ps, 416], the row
 *                          quantised as dsa_q4_write_back does (the stride is
 *                          not read; D 576, rot_off 512, rot_dim 64)
 *     D, rot_off           columns [rot_off, rot_off + rot_dim) rotate
 *     layout, scale        as in dsa_rope_target
 *   rotate     host [n_rotate], 0 to 8 targets of dsa_rope (NULL with 0)
 *   positions  int32 [T], slots int32 [T]: a row where either is negative
 *              (padding) is appended nowhere; the targets of `rotate` follow
 *              the position alone
 *   freqs      fp64 [rot_dim / 2], finite
 * A slot >= P * ps sets DSA_STATUS_BAD_INDEX and its row is skipped. Slots of
 * a call are distinct: of rows with one slot any may win, 16 bytes at a time.
 * No source may overlap a cache or an output of `rotate`, no cache another or
 * what `rotate` reads or writes: such a call is refused (rows that lie between
 * another tensor's, as in a fused projection, are not an overlap). Products and rounding are those of
 * dsa_rope; angles are formed another way, to fp32's relative precision too (and
 * 2^-65 of a turn per position), so that a result may lie one rounding step apart.
 * Supported: rot_dim a multiple of 16 up to 512, D <= 4096, D, rot_off and the
 * strides multiples of 8, 16-byte aligned rows and caches, P * ps < 2^31.
 * Targets of `rotate` that do not lie on 16 bytes take a launch of their own.
 * Needs no workspace.
 * ------------------------------------------------------------------------ */
enum dsa_cache_format { DSA_CACHE_BF16 = 0, DSA_CACHE_Q4 = 1 };
typedef struct dsa_append_target {
  const void* x;
  const void* x_rot;
  void* cache;
  int64_t x_stride, x_rot_stride, cache_stride;
  int32_t D, rot_off;
  int32_t layout; /* dsa_rope_layout */
  int32_t format; /* dsa_cache_format */
  float scale;
} dsa_append_target;
DSA_API int dsa_rope_append(dsa_stream_t stream, const dsa_append_target* append /* host */, int n_append,
                            const dsa_rope_target* rotate /* host */, int n_rotate, int T, int rot_dim,
                            const int32_t* positions, const int32_t* slots, const double* freqs, int P, int ps,
                            int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Sparse absorbed-MLA attention over the 4-bit latent cache: as
 * dsa_sparse_mla_decode (token or page units, lse, empty rows,
 * reproducibility) with `cache` [P, ps, 416] bytes in the place of kv and
 * row_stride. Split key lists are merged inside clusters: ws may be NULL (it
 * is taken for symmetry with dsa_sparse_mla_decode and not used). Only rows of visible selected positions are read, in page units
 * too, so unwritten rows may hold anything. Prefill tokens go through it with
 * page units, one selection per token.
 * An entry listed twice counts twice. T may be an upper bound: rows of o and
 * lse from cu_q_lens[S] on are left as they are.
 * Supported: as dsa_sparse_mla_decode, K <= 2^30, T * H < 2^31, |sm_scale| *
 * 185 finite in fp32.
 * ------------------------------------------------------------------------ */
DSA_API int dsa_sparse_mla_decode_q4(dsa_stream_t stream, const uint16_t* q, const uint8_t* cache,
                                     const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                                     const int32_t* page_indices, const int32_t* sel, int K, int unit, int T, int S,
                                     int P, int PTW, int ps, int H, int Dk, int Dv, float sm_scale, uint16_t* o,
                                     float* lse, void* ws, size_t ws_bytes, int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Absorbed-MLA attention with a sliding window and sinks: dsa_dense_mla where
 * token t sees, of the positions j < seq_len with j <= pos(t), those with
 * j > pos(t) - sliding_window and the first num_sinks, j < num_sinks (a
 * position that is both counts once). With sliding_window == 0 every position
 * is visible. T may be an upper bound: rows of o and lse from cu_q_lens[S] on
 * are left as they are.
 * Only pages that hold a visible position are read, in runs of 32 rows: a
 * cache may drop the pages between the sinks and the window. The finite-rows
 * rule of dsa_sparse_mla_decode holds for these runs and, with H <= 64, for
 * those of the up to 128 / H neighbouring tokens of the same request, which
 * are computed together.
 *   max_kv  as dsa_dense_mla
 *   ws      taken as there and not used (may be NULL): split key lists are
 *           merged inside clusters
 * Supported: as dsa_dense_mla; num_sinks >= 0, T * H < 2^31, any soft_cap
 * (from 2^60 on the logits stay as they are), |sm_scale| * 1.5 finite in fp32.
 * ------------------------------------------------------------------------ */
DSA_API int dsa_window_mla(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv, int row_stride,
                           const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                           const int32_t* page_indices, int max_kv, int T, int S, int P, int PTW, int ps, int H,
                           int Dk, int Dv, float sm_scale, int sliding_window, int num_sinks, float soft_cap,
                           uint16_t* o, float* lse, void* ws, size_t ws_bytes, int32_t* dev_status);

/* ------------------------------------------------------------------------
 * Absorbed-MLA attention of requests that share a prefix (no counterpart on
 * the pages): dsa_dense_mla without window and cap, where the keys that a group
 * of requests has in common are read once for every 256 of its rows (token and
 * head), of any of its requests.
 * Groups are runs of requests: group g has the requests group_offsets[g] ..
 * group_offsets[g + 1] - 1, whose first prefix_lens[g] positions hold the same
 * rows: the same pages, or copies of them. The prefix's whole runs of min(ps, 64)
 * positions are read through the page table of the group's first request, the
 * positions behind them, the rest of the prefix among them, through each
 * request's own. Visible are, as ever, j <= pos(t), j < seq_len: a
 * request may be shorter than the prefix or have new tokens inside it. Measured
 * on decode steps of 8 to 64 requests, 1 to 128 heads and 32 to 16384 own
 * positions each, it pays from about 4000 shared positions on, with 128 heads or
 * 64 requests from 2000 on; below, dsa_window_mla without a window, each request
 * by itself, is as fast or faster.
 *   prefix_lens    int32 [G], 0 (nothing shared) .. the first request's length
 *   group_offsets  int32 [G + 1], 0 .. S in order; NULL with G == 1: one group
 *   max_kv         upper bound of seq_lens (a longer one is clamped and flagged)
 *   ws             workspace of dsa_prefix_mla_workspace_size(T, H, G) bytes,
 *                  16-byte aligned: calls that may run at once, captured graphs
 *                  among them, need one each
 *   T may be an upper bound: rows of o and lse from cu_q_lens[S] on are left as
 *   they are.
 * Device conditions: a prefix below 0 or longer than its group's first request
 * is clamped to that (each request reads the rest through its own pages) and
 * sets DSA_STATUS_BAD_METADATA, as does a group whose requests or tokens are
 * out of order or out of range, whose rows are not written.
 * Cache contents: of pages that hold a visible position runs of min(ps, 64) rows
 * are read; rows of a run past the visible length must hold finite values (see
 * dsa_sparse_mla_decode), and so must a group's prefix for each of its requests,
 * though it end or have tokens inside it. What a request holds from the prefix
 * on, the group's first one too, reaches its own outputs alone, whatever it is.
 * Outputs are the same on every run.
 * Supported: as dsa_dense_mla, T <= 65535 among it; 1 <= G <= 2^20, T * H <
 * 2^31 - 2^16, |sm_scale| * 1.5 finite in fp32, max_kv <= 2^30 and with
 * (T * H / 256 + 1 + G) * (2 + ceil(256 / H)) * (max_kv / 256 + 6) below 2^31
 * (65535 tokens of 128 heads: four million keys).
 * ------------------------------------------------------------------------ */
DSA_API size_t dsa_prefix_mla_workspace_size(int T, int H, int G);
DSA_API int dsa_prefix_mla(dsa_stream_t stream, const uint16_t* q, const uint16_t* kv, int row_stride,
                           const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* cu_kv_lens,
                           const int32_t* page_indices, const int32_t* prefix_lens, const int32_t* group_offsets, int G,
                           int max_kv, int T, int S, int P, int PTW, int ps, int H, int Dk, int Dv, float sm_scale,
                           uint16_t* o, float* lse, void* ws, size_t ws_bytes, int32_t* dev_status);

/* Self-test of failure detection; the source pages have no counterpart.
 * Every pipeline wait in these kernels is bounded: when it runs out, the CTA
 * sets DSA_STATUS_TIMEOUT in the status word, unwinds and returns instead of
 * hanging or trapping. This entry runs one such wait on a barrier that
 * nothing arrives on, bounded by limit_clocks SM clocks (1 .. 1e10), so a
 * test can check that the status is set and the context stays usable; and one
 * of a whole warp that runs out in half of its lanes, which sets
 * DSA_STATUS_INTERNAL too if any lane takes it for met.
 *   dev_status  device int32, required */
DSA_API int dsa_selftest_wait_timeout(dsa_stream_t stream, long long limit_clocks, int32_t* dev_status);

/* Number of streaming multiprocessors the kernels size their grids for
 * (device of the current context); a query helper, no device work. */
DSA_API int dsa_device_sm_count(void);

/* Number of kernels this process has enqueued through the library so far
 * (a host-side counter; a diagnostic, no device work). */
DSA_API long long dsa_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* DSA_H_ */
