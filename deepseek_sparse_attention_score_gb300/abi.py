"""Thin Python binding of the C ABI in ``include/dsa.h``.

Every function here has the name of the C entry point it wraps and does
argument marshalling only: shape/dtype/device checks, optional allocation of
output and workspace tensors with PyTorch, the ctypes call on the current CUDA
stream, and turning a negative return code into an exception. All arithmetic
runs in the CUDA kernels of ``libdsa_gb300.so``; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa_gb300.so")

ERRORS = {
    -1: "DSA_ERR_INVALID_ARGUMENT",
    -2: "DSA_ERR_UNSUPPORTED",
    -3: "DSA_ERR_WORKSPACE",
    -4: "DSA_ERR_CUDA",
    -5: "DSA_ERR_SHARED_BEFORE_FULL",
    -6: "DSA_ERR_BAD_INDEXER_TYPE",
    -7: "DSA_ERR_ALIGNMENT",
    -8: "DSA_ERR_SCRATCH_LIMIT",
}
STATUS_UNION_TRUNCATED = 0x1
STATUS_BAD_METADATA = 0x2
STATUS_BAD_INDEX = 0x4
STATUS_TIMEOUT = 0x8
STATUS_INTERNAL = 0x10
STATUS_NO_PAGES = 0x20

EXPORTS = (
    "dsa_index_build_share_map",
    "dsa_indexer_workspace_size",
    "dsa_indexer_topk",
    "dsa_indexer_page_topk",
    "dsa_build_block_union",
    "dsa_sparse_mla_decode_workspace_size",
    "dsa_sparse_mla_decode",
    "dsa_sparse_mla_prefill_qblock",
    "dsa_sparse_mla_prefill_qblock_range",
    "dsa_paged_write_back",
    "dsa_paged_write_back_pair",
    "dsa_dense_mla",
    "dsa_selftest_wait_timeout",
    "dsa_indexer_topk_approx_workspace_size",
    "dsa_indexer_topk_approx",
    "dsa_topk_pages_from_tokens",
    "dsa_device_sm_count",
    "dsa_launch_count",
    "dsa_sparse_mla_decode_noalloc",
    "dsa_build_page_tables",
    "dsa_build_page_tables_next",
    "dsa_rope",
    "dsa_rope_freqs",
    "dsa_rope_attention_scales",
    "dsa_q4_write_back",
    "dsa_q4_read_rows",
    "dsa_sparse_mla_decode_q4",
    "dsa_window_mla",
)
Q4_ROW_BYTES = 416  # one row of the 4-bit latent cache


class DSAError(RuntimeError):
    def __init__(self, fn, rc):
        super().__init__(f"{fn} returned {rc} ({ERRORS.get(rc, 'unknown')})")
        self.rc = rc


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_Z = ctypes.c_size_t
_F = ctypes.c_float
_D = ctypes.c_double
_L = ctypes.c_int64

# dsa_rope_target: x, y, x_stride_t, x_stride_h, y_stride_t, y_stride_h, H, D,
# rot_off, layout, dtype, scale (72 bytes without padding). Packed bytes: a
# ctypes.Structure takes four times as long to fill.
_rope_target = struct.Struct("=QQqqqqiiiiif").pack


def lib() -> ctypes.CDLL:
    """Load the in-tree library (built by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
            "(there is no non-CUDA implementation of this package)")
    L = ctypes.CDLL(LIB_PATH)
    L.dsa_index_build_share_map.argtypes = [_P, _I, _I, _P, _P, _P]
    L.dsa_indexer_workspace_size.argtypes = [_I, _I, _I, _I]
    L.dsa_indexer_workspace_size.restype = _Z
    L.dsa_indexer_topk.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P,
                                   _Z, _P]
    L.dsa_indexer_page_topk.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _I,
                                        _P, _P, _P, _Z, _P]
    L.dsa_build_block_union.argtypes = [_P, _P, _I, _I, _I, _I, _P, _P, _I, _I, _I, _P, _P, _P, _P]
    L.dsa_sparse_mla_decode_workspace_size.argtypes = [_I, _I, _I]
    L.dsa_sparse_mla_decode_workspace_size.restype = _Z
    L.dsa_sparse_mla_decode.argtypes = [_P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                                        _F, _P, _P, _P, _Z, _P]
    L.dsa_sparse_mla_prefill_qblock.argtypes = [_P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                                                _I, _I, _I, _I, _F, _P, _P, _P]
    L.dsa_sparse_mla_prefill_qblock_range.argtypes = [_P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                                                      _I, _I, _I, _I, _I, _F, _I, _I, _P, _P, _P]
    L.dsa_sparse_mla_decode_noalloc.argtypes = [_P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I,
                                                _I, _I, _F, _P, _P, _P]
    L.dsa_paged_write_back.argtypes = [_P, _P, _I, _I, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]
    L.dsa_paged_write_back_pair.argtypes = [_P, _P, _I, _I, _P, _I, _P, _I, _I, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I,
                                            _I, _P]
    L.dsa_topk_pages_from_tokens.argtypes = [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P]
    L.dsa_dense_mla.argtypes = [_P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _F,
                                _P, _P, _P, _Z, _P]
    L.dsa_indexer_topk_approx_workspace_size.argtypes = [_I, _I, _I, _I, _I, _I]
    L.dsa_indexer_topk_approx_workspace_size.restype = _Z
    L.dsa_indexer_topk_approx.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                                          _P, _P, _Z, _P]
    L.dsa_selftest_wait_timeout.argtypes = [_P, ctypes.c_longlong, _P]
    L.dsa_build_page_tables.argtypes = [_P, _P, _P, _P, _L, _I, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P]
    L.dsa_build_page_tables_next.argtypes = [_P, _P, _P, _P, _L, _I, _P, _I, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P,
                                             _P, _P]
    L.dsa_rope.argtypes = [_P, _P, _I, _I, _I, _P, _P, _I]
    L.dsa_rope_freqs.argtypes = [_I, _D, _I, _D, _I, _D, _D, _P, _P]
    L.dsa_rope_attention_scales.argtypes = [_D, _D, _D, _P, _P]
    L.dsa_q4_write_back.argtypes = [_P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]
    L.dsa_q4_read_rows.argtypes = [_P, _P, _I, _I, _P, _I, _P, _I, _P]
    L.dsa_sparse_mla_decode_q4.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F,
                                           _P, _P, _P, _Z, _P]
    L.dsa_window_mla.argtypes = [_P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I, _F,
                                 _P, _P, _P, _Z, _P]
    L.dsa_device_sm_count.argtypes = []
    L.dsa_launch_count.argtypes = []
    L.dsa_launch_count.restype = ctypes.c_longlong
    for name in EXPORTS:
        if name not in ("dsa_indexer_workspace_size", "dsa_sparse_mla_decode_workspace_size",
                        "dsa_launch_count", "dsa_indexer_topk_approx_workspace_size"):
            getattr(L, name).restype = _I
    _lib = L
    return L


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(fn, rc):
    if rc != 0:
        raise DSAError(fn, rc)


def _need(t, name, dtype, device, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")


def _meta(device, seq_lens, cu_q_lens, cu_kv_lens, page_indices):
    for n, t in (("seq_lens", seq_lens), ("cu_q_lens", cu_q_lens), ("cu_kv_lens", cu_kv_lens),
                 ("page_indices", page_indices)):
        _need(t, n, torch.int32, device, 1)
    return seq_lens.numel(), page_indices.numel()


# --------------------------------------------------------------------- host
def dsa_index_build_share_map(indexer_types, num_layers, skip_offset=0):
    """IndexShare layer -> slot map. ``indexer_types``: sequence of 0 (full) /
    1 (shared), or None for all full. Returns (full_slot, src_slot, num_full)
    as Python lists / int (full_slot is -1 on shared layers)."""
    L = lib()
    types = None
    if indexer_types is not None:
        types = (ctypes.c_int32 * num_layers)(*[int(x) for x in indexer_types])
    full = (ctypes.c_int32 * max(1, num_layers))()
    src = (ctypes.c_int32 * max(1, num_layers))()
    nf = ctypes.c_int32(0)
    rc = L.dsa_index_build_share_map(types, num_layers, skip_offset, full, src, ctypes.byref(nf))
    _check("dsa_index_build_share_map", rc)
    return list(full)[:num_layers], list(src)[:num_layers], nf.value


def dsa_indexer_workspace_size(T, S, max_kv, ps):
    return int(lib().dsa_indexer_workspace_size(T, S, max_kv, ps))


def dsa_sparse_mla_decode_workspace_size(T, H, Dv=512):
    return int(lib().dsa_sparse_mla_decode_workspace_size(T, H, Dv))


def dsa_device_sm_count():
    return int(lib().dsa_device_sm_count())


def dsa_launch_count():
    return int(lib().dsa_launch_count())


# ------------------------------------------------------------------ indexer
def dsa_indexer_topk(q, w, kcache, seq_lens, cu_q_lens, cu_kv_lens, page_indices, *, k, max_kv, topk=None,
                     topk_scores=None, want_scores=False, ws=None, dev_status=None):
    """Indexer score + exact token top-k. Returns ``topk`` (and the scores of
    the selected positions when ``want_scores`` or ``topk_scores`` is given)."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    _need(w, "w", torch.float32, dev, 2)
    _need(kcache, "kcache", torch.bfloat16, dev, 3)
    S, PTW = _meta(dev, seq_lens, cu_q_lens, cu_kv_lens, page_indices)
    T, Hi, Di = q.shape
    P, ps, _ = kcache.shape
    if topk is None:
        topk = torch.empty((T, k), dtype=torch.int32, device=dev)
    if want_scores and topk_scores is None:
        topk_scores = torch.empty((T, k), dtype=torch.float32, device=dev)
    if ws is None:
        ws = torch.empty(max(1, dsa_indexer_workspace_size(T, S, max_kv, ps)), dtype=torch.uint8, device=dev)
    rc = lib().dsa_indexer_topk(_stream(dev), _ptr(q), _ptr(w), _ptr(kcache), _ptr(seq_lens), _ptr(cu_q_lens),
                                _ptr(cu_kv_lens), _ptr(page_indices), T, S, P, PTW, ps, Hi, Di, max_kv, k,
                                _ptr(topk), _ptr(topk_scores), _ptr(ws), ws.numel(), _ptr(dev_status))
    _check("dsa_indexer_topk", rc)
    return (topk, topk_scores) if topk_scores is not None else topk


def dsa_indexer_page_topk(q, w, kcache, seq_lens, cu_q_lens, cu_kv_lens, page_indices, *, k_pages, max_kv,
                          topk_pages=None, k=0, topk=None, with_tokens=False, topk_scores=None, ws=None,
                          dev_status=None):
    """Indexer score + page top-k (max-pooled per page); with ``with_tokens``
    (or a ``topk`` tensor) also the token top-k from the same score pass.
    Returns ``topk_pages`` or ``(topk_pages, topk)``."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    _need(w, "w", torch.float32, dev, 2)
    _need(kcache, "kcache", torch.bfloat16, dev, 3)
    S, PTW = _meta(dev, seq_lens, cu_q_lens, cu_kv_lens, page_indices)
    T, Hi, Di = q.shape
    P, ps, _ = kcache.shape
    if topk_pages is None:
        topk_pages = torch.empty((T, k_pages), dtype=torch.int32, device=dev)
    if with_tokens and topk is None:
        topk = torch.empty((T, k), dtype=torch.int32, device=dev)
    if ws is None:
        ws = torch.empty(max(1, dsa_indexer_workspace_size(T, S, max_kv, ps)), dtype=torch.uint8, device=dev)
    rc = lib().dsa_indexer_page_topk(_stream(dev), _ptr(q), _ptr(w), _ptr(kcache), _ptr(seq_lens),
                                     _ptr(cu_q_lens), _ptr(cu_kv_lens), _ptr(page_indices), T, S, P, PTW, ps, Hi,
                                     Di, max_kv, k_pages, _ptr(topk_pages), k, _ptr(topk), _ptr(topk_scores),
                                     _ptr(ws), ws.numel(), _ptr(dev_status))
    _check("dsa_indexer_page_topk", rc)
    return (topk_pages, topk) if topk is not None else topk_pages


# -------------------------------------------------------------------- union
def dsa_build_block_union(topk_units, *, QB, u_max=0, cu_q_lens=None, cu_kv_lens=None, ps=64, PTW,
                          units=None, member=None, counts=None, dev_status=None):
    """Per-block sorted union, bit-packed slot-major membership and true
    counts. Returns (units [nQB,u_max], member [nQB,u_max,QB/32] int32 view of
    the uint32 words, counts [nQB])."""
    dev = topk_units.device
    _need(topk_units, "topk_units", torch.int32, dev, 2)
    T, K = topk_units.shape
    S = 0
    if cu_q_lens is not None:
        _need(cu_q_lens, "cu_q_lens", torch.int32, dev, 1)
        _need(cu_kv_lens, "cu_kv_lens", torch.int32, dev, 1)
        S = cu_q_lens.numel() - 1
    if u_max <= 0:
        u_max = min(QB * K, PTW)
    nqb = (T + QB - 1) // QB
    if units is None:
        units = torch.empty((nqb, u_max), dtype=torch.int32, device=dev)
    if member is None:
        member = torch.empty((nqb, u_max, QB // 32), dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty((nqb,), dtype=torch.int32, device=dev)
    rc = lib().dsa_build_block_union(_stream(dev), _ptr(topk_units), T, K, QB, u_max, _ptr(cu_q_lens),
                                     _ptr(cu_kv_lens), S, ps, PTW, _ptr(units), _ptr(member), _ptr(counts),
                                     _ptr(dev_status))
    _check("dsa_build_block_union", rc)
    return units, member, counts


# ------------------------------------------------------------------- attend
def dsa_sparse_mla_decode(q, kv, seq_lens, cu_q_lens, cu_kv_lens, page_indices, sel, *, unit, sm_scale, o=None,
                          lse=None, want_lse=False, ws=None, dev_status=None, Dv=512):
    """Sparse absorbed-MLA attention over per-query selections (token ids when
    ``unit == 1``, sequence-local pages when ``unit == page_size``)."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    _need(kv, "kv", torch.bfloat16, dev, 3)
    _need(sel, "sel", torch.int32, dev, 2)
    S, PTW = _meta(dev, seq_lens, cu_q_lens, cu_kv_lens, page_indices)
    T, H, Dk = q.shape
    P, ps, row_stride = kv.shape
    K = sel.shape[1]
    if o is None:
        o = torch.empty((T, H, Dv), dtype=torch.bfloat16, device=dev)
    if want_lse and lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    if ws is None:
        nb = dsa_sparse_mla_decode_workspace_size(T, H, Dv)
        ws = torch.empty(max(1, nb), dtype=torch.uint8, device=dev)
    rc = lib().dsa_sparse_mla_decode(_stream(dev), _ptr(q), _ptr(kv), row_stride, _ptr(seq_lens), _ptr(cu_q_lens),
                                     _ptr(cu_kv_lens), _ptr(page_indices), _ptr(sel), K, unit, T, S, P, PTW, ps, H,
                                     Dk, Dv, float(sm_scale), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
                                     _ptr(dev_status))
    _check("dsa_sparse_mla_decode", rc)
    return (o, lse) if lse is not None else o


def dsa_sparse_mla_prefill_qblock(q, kv, seq_lens, cu_q_lens, cu_kv_lens, page_indices, units, member, counts, *,
                                  QB, sm_scale, o=None, lse=None, want_lse=False, dev_status=None, Dv=512,
                                  t_range=None):
    """Query-block sparse-MLA prefill over the union tables of
    ``dsa_build_block_union`` (same QB and u_max). ``t_range=(b, e)``
    computes only the output rows of tokens b .. e-1
    (``dsa_sparse_mla_prefill_qblock_range``)."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    _need(kv, "kv", torch.bfloat16, dev, 3)
    _need(units, "units", torch.int32, dev, 2)
    _need(member, "member", torch.int32, dev, 3)
    _need(counts, "counts", torch.int32, dev, 1)
    S, PTW = _meta(dev, seq_lens, cu_q_lens, cu_kv_lens, page_indices)
    T, H, Dk = q.shape
    P, ps, row_stride = kv.shape
    u_max = units.shape[1]
    if o is None:
        o = torch.empty((T, H, Dv), dtype=torch.bfloat16, device=dev)
    if want_lse and lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    if t_range is None:
        rc = lib().dsa_sparse_mla_prefill_qblock(_stream(dev), _ptr(q), _ptr(kv), row_stride, _ptr(seq_lens),
                                                 _ptr(cu_q_lens), _ptr(cu_kv_lens), _ptr(page_indices), _ptr(units),
                                                 _ptr(member), _ptr(counts), QB, u_max, T, S, P, PTW, ps, H, Dk, Dv,
                                                 float(sm_scale), _ptr(o), _ptr(lse), _ptr(dev_status))
        _check("dsa_sparse_mla_prefill_qblock", rc)
    else:
        rc = lib().dsa_sparse_mla_prefill_qblock_range(
            _stream(dev), _ptr(q), _ptr(kv), row_stride, _ptr(seq_lens), _ptr(cu_q_lens), _ptr(cu_kv_lens),
            _ptr(page_indices), _ptr(units), _ptr(member), _ptr(counts), QB, u_max, T, S, P, PTW, ps, H, Dk, Dv,
            float(sm_scale), int(t_range[0]), int(t_range[1]), _ptr(o), _ptr(lse), _ptr(dev_status))
        _check("dsa_sparse_mla_prefill_qblock_range", rc)
    return (o, lse) if lse is not None else o


def dsa_sparse_mla_decode_noalloc(q, kv, seq_lens, cu_q_lens, cu_kv_lens, page_indices, sel, *, unit, sm_scale,
                                  o=None, lse=None, want_lse=False, dev_status=None, Dv=512):
    """Same result as :func:`dsa_sparse_mla_decode`, without a workspace.

    For callers that cannot allocate device memory on this path, for example a
    plugin that is handed only its input and output buffers. The library keeps
    its split scratch in a built-in 24 MiB device array. The first call on a
    device looks up that array's address (make it before any stream capture),
    calls that overlap on the GPU race on the array, and a problem needing more
    scratch raises DSA_ERR_SCRATCH_LIMIT. ``o``/``lse`` may be preallocated by
    the caller; when omitted they are allocated here with PyTorch (the library
    call itself allocates nothing)."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    _need(kv, "kv", torch.bfloat16, dev, 3)
    _need(sel, "sel", torch.int32, dev, 2)
    S, PTW = _meta(dev, seq_lens, cu_q_lens, cu_kv_lens, page_indices)
    T, H, Dk = q.shape
    P, ps, row_stride = kv.shape
    K = sel.shape[1]
    if o is None:
        o = torch.empty((T, H, Dv), dtype=torch.bfloat16, device=dev)
    if want_lse and lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    rc = lib().dsa_sparse_mla_decode_noalloc(_stream(dev), _ptr(q), _ptr(kv), row_stride, _ptr(seq_lens),
                                             _ptr(cu_q_lens), _ptr(cu_kv_lens), _ptr(page_indices), _ptr(sel), K,
                                             unit, T, S, P, PTW, ps, H, Dk, Dv, float(sm_scale), _ptr(o), _ptr(lse),
                                             _ptr(dev_status))
    _check("dsa_sparse_mla_decode_noalloc", rc)
    return (o, lse) if lse is not None else o


# ------------------------------------------------------------ write-back
def dsa_paged_write_back(rows, cache, seq_lens, cu_q_lens, cu_kv_lens, page_indices, *, D=None, dev_status=None):
    """Write each query token's row (``rows`` [T, W], its first ``D`` columns)
    into its slot of the paged ``cache`` [P, ps, W'] in place."""
    dev = cache.device
    _need(rows, "rows", torch.bfloat16, dev, 2)
    _need(cache, "cache", torch.bfloat16, dev, 3)
    S, PTW = _meta(dev, seq_lens, cu_q_lens, cu_kv_lens, page_indices)
    T, src_stride = rows.shape
    P, ps, cache_stride = cache.shape
    if D is None:
        D = min(src_stride, cache_stride)
    rc = lib().dsa_paged_write_back(_stream(dev), _ptr(rows), src_stride, D, _ptr(cache), cache_stride,
                                    _ptr(seq_lens), _ptr(cu_q_lens), _ptr(cu_kv_lens), _ptr(page_indices), T, S, P,
                                    PTW, ps, _ptr(dev_status))
    _check("dsa_paged_write_back", rc)
    return cache


def dsa_paged_write_back_pair(rows0, cache0, rows1, cache1, seq_lens, cu_q_lens, cu_kv_lens, page_indices, *,
                              D0=None, D1=None, dev_status=None):
    """Both caches (sharing one page table) in one launch: the first ``D0``
    columns of ``rows0`` into ``cache0`` and the first ``D1`` of ``rows1``
    into ``cache1``, in place."""
    dev = cache0.device
    _need(rows0, "rows0", torch.bfloat16, dev, 2)
    _need(cache0, "cache0", torch.bfloat16, dev, 3)
    _need(rows1, "rows1", torch.bfloat16, dev, 2)
    _need(cache1, "cache1", torch.bfloat16, dev, 3)
    S, PTW = _meta(dev, seq_lens, cu_q_lens, cu_kv_lens, page_indices)
    T, s0 = rows0.shape
    T1, s1 = rows1.shape
    P, ps, c0 = cache0.shape
    P1, ps1, c1 = cache1.shape
    if T1 != T or P1 != P or ps1 != ps:
        raise ValueError("dsa_paged_write_back_pair: both targets need the same tokens, pages and page size")
    D0 = min(s0, c0) if D0 is None else D0
    D1 = min(s1, c1) if D1 is None else D1
    rc = lib().dsa_paged_write_back_pair(_stream(dev), _ptr(rows0), s0, D0, _ptr(cache0), c0, _ptr(rows1), s1, D1,
                                         _ptr(cache1), c1, _ptr(seq_lens), _ptr(cu_q_lens), _ptr(cu_kv_lens),
                                         _ptr(page_indices), T, S, P, PTW, ps, _ptr(dev_status))
    _check("dsa_paged_write_back_pair", rc)
    return cache0, cache1


def dsa_topk_pages_from_tokens(topk, *, ps, max_pages, cap=512, pages=None, counts=None, dev_status=None):
    """Ascending unique pages of each query's selected tokens, the first
    ``cap`` of them, -1 padded; returns ``(pages [T, cap], counts [T])`` with
    the uncapped number of unique pages per row."""
    dev = topk.device
    _need(topk, "topk", torch.int32, dev, 2)
    T, K = topk.shape
    if pages is None:
        pages = torch.empty((T, cap), dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty((T,), dtype=torch.int32, device=dev)
    rc = lib().dsa_topk_pages_from_tokens(_stream(dev), _ptr(topk), T, K, ps, max_pages, cap, _ptr(pages),
                                          _ptr(counts), _ptr(dev_status))
    _check("dsa_topk_pages_from_tokens", rc)
    return pages, counts


def dsa_dense_mla(q, kv, seq_lens, cu_q_lens, cu_kv_lens, page_indices, *, max_kv, sm_scale, sliding_window=0,
                  soft_cap=0.0, o=None, lse=None, want_lse=False, ws=None, dev_status=None, Dv=512):
    """Dense causal absorbed-MLA over every visible position (optionally the
    ``sliding_window`` most recent ones, with a tanh logit cap)."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    _need(kv, "kv", torch.bfloat16, dev, 3)
    S, PTW = _meta(dev, seq_lens, cu_q_lens, cu_kv_lens, page_indices)
    T, H, Dk = q.shape
    P, ps, row_stride = kv.shape
    if o is None:
        o = torch.empty((T, H, Dv), dtype=torch.bfloat16, device=dev)
    if want_lse and lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    if ws is None:
        nb = dsa_sparse_mla_decode_workspace_size(T, H, Dv)
        ws = torch.empty(max(1, nb), dtype=torch.uint8, device=dev)
    rc = lib().dsa_dense_mla(_stream(dev), _ptr(q), _ptr(kv), row_stride, _ptr(seq_lens), _ptr(cu_q_lens),
                             _ptr(cu_kv_lens), _ptr(page_indices), int(max_kv), T, S, P, PTW, ps, H, Dk, Dv,
                             float(sm_scale), int(sliding_window), float(soft_cap), _ptr(o), _ptr(lse), _ptr(ws),
                             ws.numel(), _ptr(dev_status))
    _check("dsa_dense_mla", rc)
    return (o, lse) if lse is not None else o


def dsa_indexer_topk_approx(q, w, kcache, seq_lens, cu_q_lens, cu_kv_lens, page_indices, *, k, max_kv, over=4,
                            topk=None, ws=None, dev_status=None):
    """Approximate token top-k: exact top-k of per-bin maxima over
    ``min(n, over * k)`` strided bins of each score row (ascending
    positions, -1 padded)."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    _need(w, "w", torch.float32, dev, 2)
    _need(kcache, "kcache", torch.bfloat16, dev, 3)
    S, PTW = _meta(dev, seq_lens, cu_q_lens, cu_kv_lens, page_indices)
    T, Hi, Di = q.shape
    P, ps, _ = kcache.shape
    if topk is None:
        topk = torch.empty((T, k), dtype=torch.int32, device=dev)
    if ws is None:
        nb = lib().dsa_indexer_topk_approx_workspace_size(T, S, max_kv, ps, k, over)
        ws = torch.empty(max(1, nb), dtype=torch.uint8, device=dev)
    rc = lib().dsa_indexer_topk_approx(_stream(dev), _ptr(q), _ptr(w), _ptr(kcache), _ptr(seq_lens), _ptr(cu_q_lens),
                                       _ptr(cu_kv_lens), _ptr(page_indices), T, S, P, PTW, ps, Hi, Di, int(max_kv),
                                       int(k), int(over), _ptr(topk), _ptr(ws), ws.numel(), _ptr(dev_status))
    _check("dsa_indexer_topk_approx", rc)
    return topk


def dsa_selftest_wait_timeout(dev_status, limit_clocks=2_000_000):
    """Run one bounded wait that is bound to run out (a barrier nothing
    arrives on); the device status word gets DSA_STATUS_TIMEOUT."""
    _need(dev_status, "dev_status", torch.int32, dev_status.device, 1)
    rc = lib().dsa_selftest_wait_timeout(_stream(dev_status.device), int(limit_clocks), _ptr(dev_status))
    _check("dsa_selftest_wait_timeout", rc)


# ------------------------------------------- the steps around the attention
# These calls are short, so what their checks cost counts: each check reads
# every property of a tensor once, and the raw stream handle is taken without
# building a torch.cuda.Stream (2 us of a call's 10, measured).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _launch(dev, name, *args):
    """Call a device entry point on ``dev``'s current stream (whatever device
    is current) and raise on an error code."""
    if dev.type != "cuda":
        raise ValueError(f"{name}: tensors must be on a CUDA device, got {dev}")
    fn = getattr(_lib or lib(), name)
    i = dev.index
    if torch.cuda.current_device() == i:
        rc = fn(_raw_stream(i) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream, *args)
    else:
        with torch.cuda.device(dev):
            rc = fn(torch.cuda.current_stream(dev).cuda_stream, *args)
    if rc:
        raise DSAError(name, rc)


def _addr(t):
    return None if t is None else t.data_ptr()


def _i32(t, name, dev):
    """The address of a contiguous 1-D int32 tensor."""
    if type(t) is torch.Tensor and t.dtype is torch.int32 and t.dim() == 1 and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    _need(t, name, torch.int32, dev, 1)
    return t.data_ptr()


def _ragged(dev, seq_lens, cu_q_lens, cu_kv_lens, page_indices):
    meta = (_i32(seq_lens, "seq_lens", dev), _i32(cu_q_lens, "cu_q_lens", dev), _i32(cu_kv_lens, "cu_kv_lens", dev),
            _i32(page_indices, "page_indices", dev))
    S = seq_lens.numel()
    if cu_q_lens.numel() != S + 1 or cu_kv_lens.numel() != S + 1:
        raise ValueError(f"cu_q_lens and cu_kv_lens need {S + 1} entries for {S} requests")
    return S, page_indices.numel(), meta


def _status(dev_status, dev):
    if dev_status is None:
        return None
    p = _i32(dev_status, "dev_status", dev)
    if dev_status.numel() < 1:
        raise ValueError("dev_status must hold one word")
    return p


def _shape(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


class PageTables(NamedTuple):
    """What :func:`dsa_build_page_tables` writes (int32)."""

    cu_q_lens: torch.Tensor     # [S + 1]
    cu_kv_lens: torch.Tensor    # [S + 1]
    page_indices: torch.Tensor  # [PTW], -1 behind the last page
    token_seq: torch.Tensor     # [T], -1 behind the last token
    positions: torch.Tensor     # [T]
    slots: torch.Tensor         # [T], page * ps + row
    n_taken: torch.Tensor       # [1], pages taken from the free list


def dsa_build_page_tables(q_lens, seq_lens, block_table, free_pages=None, *, T, PTW, ps=64, free_state=None,
                          out=None, dev_status=None):
    """A step's ragged metadata and slot map from its requests' lengths.

    ``q_lens`` [S] new tokens and ``seq_lens`` [S] positions with them;
    ``block_table`` [S, W] holds each request's pages and is extended in place
    by the pages that the new tokens are the first to need, taken in order
    from ``free_pages`` [F]. ``T`` and ``PTW`` may be upper bounds of the
    tokens and page-table entries (the rest is -1); with ``T`` the number of
    tokens, ``(seq_lens, out.cu_q_lens, out.cu_kv_lens, out.page_indices)`` is
    the metadata of every other call. ``out``: a :class:`PageTables` to write
    into.

    A call takes from the first entry of ``free_pages`` on. For a sequence of
    steps over one list pass ``free_state``, int32 [3 + 2 S], zeros before the
    first (dsa_build_page_tables_next): each step then takes the pages behind
    those of the steps before, and a step with the last one's lengths is that
    step again."""
    dev = q_lens.device
    a_q, a_seq = _i32(q_lens, "q_lens", dev), _i32(seq_lens, "seq_lens", dev)
    S = q_lens.numel()
    if seq_lens.numel() != S:
        raise ValueError(f"seq_lens must have {S} entries like q_lens, got {seq_lens.numel()}")
    if not isinstance(block_table, torch.Tensor) or block_table.dtype != torch.int32 or block_table.dim() != 2:
        raise TypeError("block_table must be an int32 tensor [S, W]")
    rows, W = block_table.shape
    bt_stride, one = block_table.stride()
    if block_table.device != dev or rows != S:
        raise ValueError(f"block_table must be on {dev} with {S} rows")
    if S and W and (W > 1 and one != 1 or S > 1 and bt_stride < W):
        raise ValueError("block_table rows must be contiguous and must not overlap")
    F, a_free = 0, None
    if free_pages is not None:
        F, a_free = free_pages.numel(), _i32(free_pages, "free_pages", dev)
    entry, state = "dsa_build_page_tables", ()
    if free_state is not None:
        entry, state = "dsa_build_page_tables_next", (_i32(free_state, "free_state", dev),)
        _shape(free_state, "free_state", (3 + 2 * S,))
    T, PTW = int(T), int(PTW)
    if T < 0 or PTW < 0:
        raise ValueError("T and PTW must not be negative")
    if out is None:
        # one allocation; the page table first, on a 16-byte boundary
        buf = torch.empty(PTW + 2 * (S + 1) + 3 * T + 1, dtype=torch.int32, device=dev)
        pages, cu_q, cu_kv, seq, pos, slots, taken = buf.split_with_sizes((PTW, S + 1, S + 1, T, T, T, 1))
        out = PageTables(cu_q, cu_kv, pages, seq, pos, slots, taken)
    else:
        for name, n in (("cu_q_lens", S + 1), ("cu_kv_lens", S + 1), ("page_indices", PTW), ("token_seq", T),
                        ("positions", T), ("slots", T), ("n_taken", 1)):
            _need(getattr(out, name), f"out.{name}", torch.int32, dev, 1)
            _shape(getattr(out, name), f"out.{name}", (n,))
    cu_q, cu_kv, pages, seq, pos, slots, taken = out
    _launch(dev, entry, a_q, a_seq, block_table.data_ptr(), max(W, bt_stride) if S > 1 else W, W,
            a_free, F, *state, S, T, PTW, int(ps), cu_q.data_ptr(), cu_kv.data_ptr(), pages.data_ptr(), seq.data_ptr(),
            pos.data_ptr(), slots.data_ptr(), taken.data_ptr(), _status(dev_status, dev))
    return out


_ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
_ROPE_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_ROPE_SCALINGS = {"none": 0, "linear": 1, "yarn": 2}


class RopeTarget:
    """Rows to rotate in one :func:`dsa_rope` call: ``x`` [T, H, D] (bf16 or
    fp32, any strides with contiguous columns), turned in columns ``rot_off``
    .. ``rot_off + rot_dim - 1`` (all after ``rot_off`` by default) into ``y``
    of the same shape, or in place without one. ``layout``: "interleaved"
    pairs (2i, 2i+1) or "half" pairs (i, i + rot_dim/2). ``scale`` multiplies
    the rotated columns. Holds its tensors and may be kept and used again:
    a call packs it anew when their storage, shape or strides have changed
    since it was made (resize_, set_, .data)."""

    __slots__ = ("x", "y", "rot_dim", "args", "c", "shape", "xp", "xs", "yp", "ys")

    def __init__(self, x, y=None, *, rot_off=0, rot_dim=None, layout="half", scale=1.0):
        if y is None:
            y = x
        if not isinstance(x, torch.Tensor) or not isinstance(y, torch.Tensor) or x.dim() != 3:
            raise TypeError("x and y must be tensors [T, H, D]")
        dtype, shape, lay = _ROPE_DTYPES.get(x.dtype), x.shape, _ROPE_LAYOUTS.get(layout)
        if dtype is None:
            raise TypeError(f"x must be bf16 or fp32, got {x.dtype}")
        if y is not x and (y.dtype is not x.dtype or y.shape != shape or y.device != x.device):
            raise ValueError("y must have the type, device and shape of x")
        if lay is None:
            raise ValueError(f"layout must be one of {sorted(_ROPE_LAYOUTS)}, got {layout!r}")
        _, H, D = shape
        xt, xh, xd = xs = x.stride()
        yt, yh, yd = ys = y.stride()
        if D > 1 and (xd != 1 or yd != 1):
            raise ValueError("the columns of x and y must be contiguous")
        xp, yp = x.data_ptr(), y.data_ptr()
        self.x, self.y, self.args = x, y, (rot_off, rot_dim, layout, scale)
        self.rot_dim = D - rot_off if rot_dim is None else rot_dim
        self.c = _rope_target(xp, yp, xt, xh, yt, yh, H, D, rot_off, lay, dtype, scale)
        self.shape, self.xp, self.xs, self.yp, self.ys = shape, xp, xs, yp, ys

    def repack(self):
        """Pack the tensors as they are now, with the checks of a new target."""
        off, dim, layout, scale = self.args
        self.__init__(self.x, self.y, rot_off=off, rot_dim=dim, layout=layout, scale=scale)


def dsa_rope(targets, positions, freqs, *, inverse=False):
    """Rotate the rows of one or several :class:`RopeTarget` in one launch.
    ``positions`` int32 [T] (rows with a negative one are left alone),
    ``freqs`` fp64 [rot_dim / 2] as :func:`dsa_rope_freqs` makes them.
    ``inverse`` turns back, which is also the gradient. Returns the rotated
    tensors, one or a list as ``targets`` came."""
    one = isinstance(targets, RopeTarget)
    ts = [targets] if one else list(targets)
    dev = positions.device
    a_pos = _i32(positions, "positions", dev)
    _need(freqs, "freqs", torch.float64, dev, 1)
    T, rot = positions.numel(), 2 * freqs.numel()
    for g in ts:
        x, y = g.x, g.y
        if (x.data_ptr() != g.xp or x.stride() != g.xs or x.shape != g.shape or
                y is not x and (y.data_ptr() != g.yp or y.stride() != g.ys or y.shape != g.shape)):
            g.repack()
        if x.device != dev or g.shape[0] != T:
            raise ValueError(f"a target needs {T} rows on {dev}, got {tuple(x.shape)} on {x.device}")
        if g.rot_dim != rot:
            raise ValueError(f"a target rotates {g.rot_dim} columns, freqs are for {rot}")
    _launch(dev, "dsa_rope", b"".join([g.c for g in ts]), len(ts), T, rot, a_pos, freqs.data_ptr(), 1 if inverse else 0)
    return ts[0].y if one else [g.y for g in ts]


def dsa_rope_freqs(rot_dim, *, base=10000.0, scaling="none", factor=1.0, orig_max_pos=4096, beta_fast=32.0,
                   beta_slow=1.0, device=None):
    """Frequencies (fp64 [rot_dim / 2], radians per position) of the rotary
    pairs, scaled for long contexts: "none", "linear" (all divided by
    ``factor``) or "yarn" (by parts); and YaRN's factor 0.1 ln(factor) + 1 (or
    1), the scale of queries and keys whose columns all rotate. For the heads
    here, of which 64 of 576 columns rotate, see
    :func:`dsa_rope_attention_scales`."""
    if scaling not in _ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_SCALINGS)}, got {scaling!r}")
    freqs = torch.empty(max(0, int(rot_dim) // 2), dtype=torch.float64)
    ms = ctypes.c_double(1.0)
    rc = lib().dsa_rope_freqs(int(rot_dim), float(base), _ROPE_SCALINGS[scaling], float(factor), int(orig_max_pos),
                              float(beta_fast), float(beta_slow), _addr(freqs), ctypes.byref(ms))
    _check("dsa_rope_freqs", rc)
    return (freqs if device is None else freqs.to(device)), ms.value


def dsa_rope_attention_scales(factor, *, mscale=1.0, mscale_all_dim=1.0):
    """YaRN's factors for a head of which a part rotates: the scale of the
    rotated columns of queries and keys (:class:`RopeTarget`), and what
    ``sm_scale`` is multiplied by. ``mscale`` and ``mscale_all_dim``: the
    model's coefficients."""
    rotated, logits = ctypes.c_double(), ctypes.c_double()
    rc = lib().dsa_rope_attention_scales(float(factor), float(mscale), float(mscale_all_dim), ctypes.byref(rotated),
                                         ctypes.byref(logits))
    _check("dsa_rope_attention_scales", rc)
    return rotated.value, logits.value


def _rows576(t, name, dev):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.dim() != 2:
        raise TypeError(f"{name} must be a bf16 tensor [N, W]")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    n, w = t.shape
    stride, one = t.stride()
    if w < 576 or one != 1:
        raise ValueError(f"{name} needs at least 576 contiguous columns")
    return n, stride if n > 1 else 576


def _cache4(cache, dev):
    _need(cache, "cache", torch.uint8, dev, 3)
    P, ps, row = cache.shape
    if row != Q4_ROW_BYTES:
        raise ValueError(f"a 4-bit cache is [P, ps, {Q4_ROW_BYTES}], got {tuple(cache.shape)}")
    return P, ps


def dsa_q4_write_back(rows, cache, seq_lens, cu_q_lens, cu_kv_lens, page_indices, *, dev_status=None):
    """Quantise each query token's latent row (``rows`` [T, >= 576]) into its
    slot of the 4-bit ``cache`` [P, ps, 416] (uint8), in place."""
    dev = cache.device
    P, ps = _cache4(cache, dev)
    T, stride = _rows576(rows, "rows", dev)
    S, PTW, meta = _ragged(dev, seq_lens, cu_q_lens, cu_kv_lens, page_indices)
    _launch(dev, "dsa_q4_write_back", rows.data_ptr(), stride, cache.data_ptr(), *meta, T, S, P, PTW, ps,
            _status(dev_status, dev))
    return cache


def dsa_q4_read_rows(cache, slots, *, out=None, dev_status=None):
    """The bf16 values [N, 576] of the rows in ``slots`` (page * ps + row) of a
    4-bit cache; a negative slot gives zeros."""
    dev = cache.device
    P, ps = _cache4(cache, dev)
    a_slots = _i32(slots, "slots", dev)
    N = slots.numel()
    if out is None:
        out = torch.empty((N, 576), dtype=torch.bfloat16, device=dev)
    rows, stride = _rows576(out, "out", dev)
    if rows != N:
        raise ValueError(f"out needs {N} rows")
    _launch(dev, "dsa_q4_read_rows", cache.data_ptr(), P, ps, a_slots, N, out.data_ptr(), stride,
            _status(dev_status, dev))
    return out


def _attend_out(dev, T, H, Dv, o, lse, want_lse):
    if o is None:
        o = torch.empty((T, H, Dv), dtype=torch.bfloat16, device=dev)
    else:
        _need(o, "o", torch.bfloat16, dev, 3)
        _shape(o, "o", (T, H, Dv))
    if want_lse and lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    elif lse is not None:
        _need(lse, "lse", torch.float32, dev, 2)
        _shape(lse, "lse", (T, H))
    return o, lse


def dsa_sparse_mla_decode_q4(q, cache, seq_lens, cu_q_lens, cu_kv_lens, page_indices, sel, *, unit, sm_scale, o=None,
                             lse=None, want_lse=False, ws=None, dev_status=None, Dv=512):
    """:func:`dsa_sparse_mla_decode` over the 4-bit latent ``cache``
    [P, ps, 416] that :func:`dsa_q4_write_back` fills. Needs no workspace
    (``ws`` is taken as there and not used); ``q`` may have padding rows behind
    the last token, whose outputs are left as they are."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    P, ps = _cache4(cache, dev)
    _need(sel, "sel", torch.int32, dev, 2)
    T, H, Dk = q.shape
    S, PTW, meta = _ragged(dev, seq_lens, cu_q_lens, cu_kv_lens, page_indices)
    K = sel.shape[1]
    _shape(sel, "sel", (T, K))
    o, lse = _attend_out(dev, T, H, Dv, o, lse, want_lse)
    _launch(dev, "dsa_sparse_mla_decode_q4", _addr(q), _addr(cache), *meta, _addr(sel), K, int(unit), T, S, P, PTW, ps,
            H, Dk, Dv, float(sm_scale), _addr(o), _addr(lse), None, 0, _status(dev_status, dev))
    return (o, lse) if lse is not None else o


def dsa_window_mla(q, kv, seq_lens, cu_q_lens, cu_kv_lens, page_indices, *, max_kv, sm_scale, sliding_window,
                   num_sinks=0, soft_cap=0.0, o=None, lse=None, want_lse=False, ws=None, dev_status=None, Dv=512):
    """Causal absorbed-MLA over the ``sliding_window`` most recent positions
    and the first ``num_sinks`` ones. Needs no workspace (``ws`` is taken as in
    :func:`dsa_dense_mla` and not used); ``q`` may have padding rows behind the
    last token, whose outputs are left as they are."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    _need(kv, "kv", torch.bfloat16, dev, 3)
    T, H, Dk = q.shape
    P, ps, row_stride = kv.shape
    S, PTW, meta = _ragged(dev, seq_lens, cu_q_lens, cu_kv_lens, page_indices)
    o, lse = _attend_out(dev, T, H, Dv, o, lse, want_lse)
    _launch(dev, "dsa_window_mla", _addr(q), _addr(kv), row_stride, *meta, int(max_kv), T, S, P, PTW, ps, H, Dk, Dv,
            float(sm_scale), int(sliding_window), int(num_sinks), float(soft_cap), _addr(o), _addr(lse), None, 0,
            _status(dev_status, dev))
    return (o, lse) if lse is not None else o
