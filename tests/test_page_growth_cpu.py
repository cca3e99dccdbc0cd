"""Refusals of dsa_build_page_tables_next and of its binding; no GPU."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


def _args(**kw):
    p = ctypes.c_void_p(4096)
    a = dict(stream=None, q_lens=p, seq_lens=p, block_table=p, bt_stride=8, width=8, free=p, F=4, state=p, S=3, T=3,
             PTW=9, ps=64, cu_q=p, cu_kv=p, pages=p, seq=p, pos=p, slots=p, taken=p, status=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), INVALID), (dict(F=-1), INVALID), (dict(free=None), INVALID), (dict(ps=48), UNSUPPORTED),
    (dict(S=16385), UNSUPPORTED), (dict(bt_stride=7), INVALID), (dict(taken=None), INVALID), (dict(q_lens=None), INVALID),
])
def test_host_checks(dsa, kw, code):
    assert dsa.lib().dsa_build_page_tables_next(*_args(**kw)) == code


@pytest.mark.parametrize("state,error", [
    (torch.zeros(6, dtype=torch.int32), ValueError), (torch.zeros(8, dtype=torch.int32), ValueError),
    (torch.zeros(7, dtype=torch.int64), TypeError), (torch.zeros(14, dtype=torch.int32)[::2], ValueError),
    (torch.zeros(1, 7, dtype=torch.int32), ValueError), ([0] * 7, TypeError),
])
def test_binding_refuses_a_bad_state(dsa, state, error):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(error):
        dsa.dsa_build_page_tables(i32(2), i32(2), i32(2, 4), T=2, PTW=2, free_state=state)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.dsa_build_page_tables(i32(2), i32(2), i32(2, 4), T=2, PTW=2, free_state=i32(7))
