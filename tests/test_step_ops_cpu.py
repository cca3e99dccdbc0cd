"""Refusals and host-only parts of the operators around the attention; no
GPU: every call here must be turned away before anything is enqueued."""
import ctypes
import math

import numpy as np
import pytest
import torch

import steps_ref as R

OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, -1, -2, -7


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


def _p(addr=4096):
    return ctypes.c_void_p(addr)


def _args(base, kw):
    base.update(kw)
    return list(base.values())


def _tables(**kw):
    return _args(dict(stream=None, q_lens=_p(), seq_lens=_p(), block_table=_p(), bt_stride=8, width=8, free=_p(), F=4,
                      S=3, T=3, PTW=9, ps=64, cu_q=_p(), cu_kv=_p(), pages=_p(), seq=_p(), pos=_p(), slots=_p(),
                      taken=_p(), status=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), INVALID), (dict(T=-1), INVALID), (dict(PTW=-1), INVALID), (dict(F=-1), INVALID),
    (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(PTW=(1 << 30) + 1), UNSUPPORTED),
    (dict(width=-1), INVALID), (dict(bt_stride=7), INVALID), (dict(ps=48), UNSUPPORTED), (dict(ps=0), UNSUPPORTED),
    (dict(S=16385), UNSUPPORTED), (dict(width=1 << 25, bt_stride=1 << 25), UNSUPPORTED),
    (dict(q_lens=None), INVALID), (dict(seq_lens=None), INVALID), (dict(block_table=None), INVALID),
    (dict(free=None), INVALID), (dict(cu_q=None), INVALID), (dict(cu_kv=None), INVALID), (dict(pages=None), INVALID),
    (dict(seq=None), INVALID), (dict(pos=None), INVALID), (dict(slots=None), INVALID), (dict(taken=None), INVALID),
])
def test_page_tables_host_checks(dsa, kw, code):
    assert dsa.lib().dsa_build_page_tables(*_tables(**kw)) == code


def _rope(n=1, T=4, rot=64, pos=_p(), freqs=_p(), **kw):
    from deepseek_sparse_attention_score_gb300.abi import _rope_target
    f = dict(x=4096, y=8192, x_stride_t=64, x_stride_h=64, y_stride_t=64, y_stride_h=64, H=1, D=64, rot_off=0,
             layout=0, dtype=0, scale=1.0)
    f.update(kw)
    return [None, _rope_target(*[v or 0 for v in f.values()]) * max(1, n), n, T, rot, pos, freqs, 0]


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), INVALID), (dict(n=9), UNSUPPORTED), (dict(T=-1), INVALID), (dict(rot=0), INVALID),
    (dict(rot=63), INVALID), (dict(rot=514, D=600), UNSUPPORTED), (dict(rot=66), INVALID), (dict(rot_off=1), INVALID),
    (dict(rot_off=-1), INVALID), (dict(H=-1), INVALID), (dict(layout=2), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(scale=math.nan), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(x=4097), ALIGNMENT),
    (dict(y=8194, dtype=1), ALIGNMENT), (dict(y=4096, y_stride_t=128), INVALID), (dict(pos=None), INVALID),
    (dict(y_stride_t=0), INVALID), (dict(y_stride_t=63), INVALID),  # rows of y on top of each other
    (dict(H=2, y_stride_t=64), INVALID), (dict(H=2, y_stride_t=127), INVALID),
    (dict(H=2, y_stride_h=256, y_stride_t=64, T=5), INVALID), (dict(H=2, y_stride_h=0, y_stride_t=128), INVALID),
    (dict(D=4097), UNSUPPORTED), (dict(H=65537), UNSUPPORTED),
    (dict(freqs=None), INVALID), (dict(H=1 << 26), UNSUPPORTED), (dict(T=0), OK), (dict(T=0, x=None), OK),
])
def test_rope_host_checks(dsa, kw, code):
    assert dsa.lib().dsa_rope(*_rope(**kw)) == code


def _write(**kw):
    return _args(dict(stream=None, rows=_p(), src_stride=576, cache=_p(), seq=_p(), cu_q=_p(), cu_kv=_p(), pages=_p(),
                      T=4, S=4, P=16, PTW=16, ps=64, status=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(src_stride=575), UNSUPPORTED), (dict(src_stride=580), UNSUPPORTED), (dict(src_stride=512), UNSUPPORTED),
    (dict(rows=None), INVALID), (dict(cache=None), INVALID), (dict(rows=_p(4104)), ALIGNMENT),
    (dict(cache=_p(4100)), ALIGNMENT), (dict(ps=16), UNSUPPORTED), (dict(pages=None), INVALID), (dict(T=-1), INVALID),
    (dict(P=1 << 25), UNSUPPORTED), (dict(S=0), INVALID), (dict(T=0), OK),
])
def test_q4_write_back_host_checks(dsa, kw, code):
    assert dsa.lib().dsa_q4_write_back(*_write(**kw)) == code


def _read(**kw):
    return _args(dict(stream=None, cache=_p(), P=4, ps=64, slots=_p(), N=3, rows=_p(), stride=576, status=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), INVALID), (dict(P=-1), INVALID), (dict(ps=100), UNSUPPORTED), (dict(P=1 << 26), UNSUPPORTED),
    (dict(stride=584 - 1), UNSUPPORTED), (dict(stride=568), UNSUPPORTED), (dict(slots=None), INVALID),
    (dict(rows=None), INVALID), (dict(cache=None), INVALID), (dict(rows=_p(4098)), ALIGNMENT), (dict(N=0), OK),
])
def test_q4_read_rows_host_checks(dsa, kw, code):
    assert dsa.lib().dsa_q4_read_rows(*_read(**kw)) == code


def _attend(**kw):
    return _args(dict(stream=None, q=_p(), cache=_p(), seq=_p(), cu_q=_p(), cu_kv=_p(), pages=_p(), sel=_p(), K=64,
                      unit=1, T=4, S=4, P=16, PTW=16, ps=64, H=128, Dk=576, Dv=512, sm_scale=0.1, o=_p(), lse=None,
                      ws=_p(), ws_bytes=1 << 20, status=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(ps=48), UNSUPPORTED), (dict(Dv=256), UNSUPPORTED), (dict(Dk=512), UNSUPPORTED), (dict(unit=32), INVALID),
    (dict(K=0), INVALID), (dict(K=(1 << 30) + 1), UNSUPPORTED), (dict(sel=None), INVALID),
    (dict(sm_scale=math.inf), INVALID),
    (dict(sm_scale=3e36), INVALID), (dict(cache=_p(4104)), ALIGNMENT), (dict(cache=None), INVALID),
    (dict(o=None), INVALID), (dict(T=65536, S=65536), UNSUPPORTED), (dict(T=65535, H=32769), UNSUPPORTED), (dict(H=-1), INVALID), (dict(H=0), OK),
    (dict(T=0, S=0, P=0, PTW=0), OK),
])
def test_decode_q4_host_checks(dsa, kw, code):
    assert dsa.lib().dsa_sparse_mla_decode_q4(*_attend(**kw)) == code


def _window(**kw):
    return _args(dict(stream=None, q=_p(), kv=_p(), row_stride=576, seq=_p(), cu_q=_p(), cu_kv=_p(), pages=_p(),
                      max_kv=1024, T=4, S=4, P=16, PTW=16, ps=64, H=128, Dk=576, Dv=512, sm_scale=0.1, window=8,
                      sinks=4, cap=0.0, o=_p(), lse=None, ws=_p(), ws_bytes=1 << 20, status=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(cap=-1.0), INVALID), (dict(cap=math.inf), INVALID),
    (dict(max_kv=0), INVALID), (dict(ps=100), UNSUPPORTED), (dict(kv=_p(4100)), ALIGNMENT),
    (dict(T=65535, H=32769), UNSUPPORTED), (dict(row_stride=600), UNSUPPORTED), (dict(sm_scale=math.nan), INVALID), (dict(T=0, S=0, P=0, PTW=0), OK),
])
def test_window_host_checks(dsa, kw, code):
    assert dsa.lib().dsa_window_mla(*_window(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rot_dim=0), INVALID), (dict(rot_dim=7), INVALID), (dict(base=1.0), INVALID), (dict(base=math.nan), INVALID),
    (dict(scaling="yarn", factor=0.5), INVALID), (dict(scaling="linear", factor=math.inf), INVALID),
    (dict(scaling="yarn", factor=2.0, orig_max_pos=0), INVALID),
    (dict(scaling="yarn", factor=2.0, beta_fast=1.0, beta_slow=2.0), INVALID),
])
def test_rope_freqs_host_checks(dsa, kw, code):
    kw = dict(dict(rot_dim=64), **kw)
    with pytest.raises(dsa.DSAError) as e:
        dsa.dsa_rope_freqs(**kw)
    assert e.value.rc == code


def test_rope_freqs(dsa):
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    got, m = dsa.dsa_rope_freqs(64)
    np.testing.assert_allclose(got.numpy(), f, rtol=1e-14)
    assert m == 1.0
    got, m = dsa.dsa_rope_freqs(64, scaling="linear", factor=8.0)
    np.testing.assert_allclose(got.numpy(), f / 8, rtol=1e-14)
    assert m == 1.0
    # YaRN by hand: a pair turns orig * f / (2 pi) times within the trained
    # length; those of more than 32 turns stay, those of less than one are
    # divided, and between the weights fall by equal steps
    got, m = dsa.dsa_rope_freqs(64, scaling="yarn", factor=40.0, orig_max_pos=4096)
    turns = 4096 * f / (2 * np.pi)
    keep = (got.numpy() / f - 1 / 40) / (1 - 1 / 40)
    assert np.allclose(keep[turns > 32 * 1.4], 1, atol=1e-12) and np.allclose(keep[turns < 1 / 1.4], 0, atol=1e-12)
    mid = keep[(keep > 1e-9) & (keep < 1 - 1e-9)]
    assert len(mid) > 5 and np.allclose(np.diff(mid), np.diff(mid)[0], atol=1e-12) and np.diff(mid)[0] < 0
    assert abs(m - (0.1 * math.log(40.0) + 1)) < 1e-15
    got, m = dsa.dsa_rope_freqs(64, scaling="yarn", factor=1.0)
    np.testing.assert_allclose(got.numpy(), f, rtol=1e-14)
    assert m == 1.0
    got, _ = dsa.dsa_rope_freqs(2)
    assert got.tolist() == [1.0]


def test_wrappers_refuse_bad_tensors(dsa):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on a GPU
        dsa.dsa_build_page_tables(i32(2), i32(2), i32(2, 4), T=2, PTW=2)
    with pytest.raises(TypeError):
        dsa.dsa_build_page_tables(i32(2).long(), i32(2), i32(2, 4), T=2, PTW=2)
    with pytest.raises(ValueError):
        dsa.dsa_build_page_tables(i32(2), i32(3), i32(2, 4), T=2, PTW=2)
    with pytest.raises(ValueError):
        dsa.dsa_build_page_tables(i32(2), i32(2), i32(3, 4), T=2, PTW=2)
    with pytest.raises(ValueError):
        dsa.dsa_build_page_tables(i32(2), i32(2), i32(4, 2).t(), T=2, PTW=2)
    with pytest.raises(ValueError):
        dsa.dsa_build_page_tables(i32(2), i32(2), i32(1, 4).expand(2, 4), T=2, PTW=2)
    x = torch.zeros(3, 2, 64)
    with pytest.raises(TypeError):
        dsa.RopeTarget(x.half())
    with pytest.raises(TypeError):
        dsa.RopeTarget(x[0])
    with pytest.raises(ValueError):
        dsa.RopeTarget(x, x.bfloat16().new_zeros(3, 2, 64))
    with pytest.raises(ValueError):
        dsa.RopeTarget(x, layout="quarter")
    with pytest.raises(ValueError):
        dsa.RopeTarget(x.transpose(1, 2))
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        dsa.dsa_rope(dsa.RopeTarget(x), i32(4), f)
    with pytest.raises(ValueError):
        dsa.dsa_rope(dsa.RopeTarget(x, rot_dim=32), i32(3), f)
    with pytest.raises(TypeError):
        dsa.dsa_rope(dsa.RopeTarget(x), i32(3), f.float())
    cache = torch.zeros(2, 64, 416, dtype=torch.uint8)
    rows = torch.zeros(1, 576, dtype=torch.bfloat16)
    meta = (i32(1), i32(2), i32(2), i32(1))
    with pytest.raises(ValueError):
        dsa.dsa_q4_write_back(rows[:, :512], cache, *meta)
    with pytest.raises(ValueError):
        dsa.dsa_q4_write_back(rows, cache[:, :, :400].contiguous(), *meta)
    with pytest.raises(ValueError):
        dsa.dsa_q4_write_back(rows, cache, i32(1), i32(3), i32(2), i32(1))
    with pytest.raises(ValueError):
        dsa.dsa_q4_read_rows(cache, i32(3), out=rows)
    q = torch.zeros(1, 2, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # one selection row per token
        dsa.dsa_sparse_mla_decode_q4(q, cache, *meta, i32(2, 4), unit=1, sm_scale=1.0)
    with pytest.raises(ValueError):
        dsa.dsa_sparse_mla_decode_q4(q, cache, *meta, i32(1, 4), unit=1, sm_scale=1.0, o=q[:, :1, :512].contiguous())
    with pytest.raises(ValueError):
        dsa.dsa_window_mla(q, torch.zeros(2, 64, 576, dtype=torch.bfloat16), *meta, max_kv=64, sm_scale=1.0,
                           sliding_window=4, lse=torch.zeros(1, 3))


def test_reference_quantiser():
    """The tests' own 4-bit reference, by hand: scale 1 keeps the e2m1 values,
    ties go to the even code, the row's bytes are where the header says."""
    x = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -6, -.26, -.74, -1.26, 0, -0.0, .5, 4])
    c, s = R.q4_group(x)
    assert R.E4M3[s] == 1.0
    assert c.tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 15, 9, 9, 11, 0, 8, 1, 6]
    row = torch.zeros(1, 576, dtype=torch.bfloat16)
    row[0, :16] = torch.from_numpy(x).to(torch.bfloat16)
    row[0, 512] = 1.0
    b = R.q4_pack(row)[0]
    # word 0: dims 0 2 4 6 in nibbles 0..3, dims 1 3 5 7 above
    assert b[:4].tolist() == [7 | 2 << 4, 4 | 6 << 4, 0 | 2 << 4, 4 | 6 << 4]
    assert b[256] == s and (b[257:288] == 0).all() and b[288:290].tolist() == [0x80, 0x3F]
    v = R.q4_values(b)
    assert v[:8].tolist() == [6, 0, 1, 1, 2, 2, 4, 4] and v[512] == 1.0
    assert R.q4_group(np.r_[np.nan, np.zeros(15)])[1] == 0x7F and R.q4_group(np.full(16, 6 * 2.0 ** -10))[1] == 0
