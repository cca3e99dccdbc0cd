"""dsa_prefix_mla's refusals, by the entry point and by the wrapper: no call
here reaches a kernel."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE, ALIGNMENT = -1, -2, -3, -7
OK = dict(q=16, kv=16, row_stride=576, seq=16, cu_q=16, cu_kv=16, pages=16, prefix=16, groups=16, G=2, max_kv=100, T=3,
          S=2, P=4, PTW=4, ps=64, H=16, Dk=576, Dv=512, scale=1.0, o=16, lse=None, ws=256, ws_bytes=1 << 40, status=None)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    from deepseek_sparse_attention_score_gb300 import abi

    return abi.lib()


def _call(lib, **bad):
    a = {**OK, **bad}
    p = lambda k: ctypes.c_void_p(a[k]) if a[k] else None
    return lib.dsa_prefix_mla(None, p("q"), p("kv"), a["row_stride"], p("seq"), p("cu_q"), p("cu_kv"), p("pages"),
                              p("prefix"), p("groups"), a["G"], a["max_kv"], a["T"], a["S"], a["P"], a["PTW"], a["ps"],
                              a["H"], a["Dk"], a["Dv"], a["scale"], p("o"), p("lse"), p("ws"), a["ws_bytes"],
                              p("status"))


@pytest.mark.parametrize("bad,rc", [
    (dict(q=None), INVALID), (dict(kv=None), INVALID), (dict(o=None), INVALID), (dict(seq=None), INVALID),
    (dict(cu_q=None), INVALID), (dict(cu_kv=None), INVALID), (dict(pages=None), INVALID), (dict(prefix=None), INVALID),
    (dict(groups=None), INVALID), (dict(G=0), INVALID), (dict(G=-1), INVALID), (dict(G=(1 << 20) + 1), UNSUPPORTED),
    (dict(max_kv=0), INVALID), (dict(max_kv=(1 << 30) + 1), UNSUPPORTED), (dict(T=-1), INVALID), (dict(S=0), INVALID),
    (dict(T=65536), UNSUPPORTED), (dict(T=65535, H=32768), UNSUPPORTED), (dict(ps=16), UNSUPPORTED),
    # key tiles of all row tiles together: at most 2^31, which four million keys keep here
    (dict(T=65535, H=128, max_kv=1 << 23), UNSUPPORTED), (dict(T=65535, H=128, max_kv=4000000, ws=None), WORKSPACE),
    (dict(T=300, H=1, max_kv=1 << 30), UNSUPPORTED), (dict(T=1, H=1, max_kv=1 << 30, ws=None, G=1), UNSUPPORTED),
    (dict(P=1 << 26), UNSUPPORTED), (dict(H=-1), INVALID), (dict(Dk=512), UNSUPPORTED), (dict(Dv=576), UNSUPPORTED),
    (dict(row_stride=600), UNSUPPORTED), (dict(q=8), ALIGNMENT), (dict(kv=24), ALIGNMENT), (dict(o=4), ALIGNMENT),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=3e38), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE), (dict(ws=264), ALIGNMENT),
])
def test_refused(lib, bad, rc):
    assert _call(lib, **bad) == rc


def test_nothing_to_do(lib):
    assert _call(lib, T=0, S=0, P=0, PTW=0, prefix=None, ws=None, ws_bytes=0) == 0
    assert _call(lib, H=0, ws=None) == 0


def test_workspace_size(lib):
    size = lib.dsa_prefix_mla_workspace_size
    assert size(0, 16, 1) == 0 and size(4, 0, 1) == 0 and size(4, 16, 0) == 0
    assert 0 < size(4, 16, 1) <= size(4000, 128, 1) <= size(4000, 128, 4000) < 1 << 30
    need = size(3, 16, 2)
    assert _call(lib, ws_bytes=need - 1) == WORKSPACE


def test_wrapper_refusals():
    import deepseek_sparse_attention_score_gb300 as dsa

    q, kv = torch.zeros(2, 3, 576, dtype=torch.bfloat16), torch.zeros(4, 64, 576, dtype=torch.bfloat16)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    meta = (i32(2), i32(3), i32(3), i32(4))
    call = lambda q=q, kv=kv, meta=meta, prefix=i32(1), groups=None, **kw: dsa.dsa_prefix_mla(
        q, kv, *meta, prefix, groups, max_kv=100, sm_scale=1.0, **kw)
    for bad, err in ((dict(q=q.float()), TypeError), (dict(q=q[0]), ValueError), (dict(kv=kv[:, :, ::2]), ValueError),
                     (dict(meta=(i32(2), i32(2), i32(3), i32(4))), ValueError), (dict(prefix=i32(2)), ValueError),
                     (dict(prefix=i32(1).long()), TypeError), (dict(groups=i32(3)), ValueError),
                     (dict(groups=i32(2).float()), TypeError), (dict(o=q), ValueError),
                     (dict(lse=torch.zeros(3, 2)), ValueError), (dict(ws=torch.zeros(8)), ValueError),
                     (dict(dev_status=i32(0)), ValueError), (dict(), ValueError)):  # the last: not on a GPU
        with pytest.raises(err):
            call(**bad)
