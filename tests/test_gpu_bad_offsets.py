"""Offsets that do not start at zero (invalid metadata): the tokens in front of
the first request have no slot, and no lookup leaves the arrays."""
import numpy as np
import pytest
import torch

import dsa_inputs as DI
import steps_ref as R
from gpu_util import meta_to

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BAD_METADATA = 0x2


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


@pytest.mark.parametrize("S", [2, 40, 1100])
def test_tokens_before_the_first_request(dsa, S):
    """cu_q_lens = [3, 4, ...]: tokens 0, 1 and 2 belong to no request, tokens
    3 .. S + 2 to requests 0 .. S - 1."""
    wl = DI.random_small(61, [1] * S, [64 + 7 * (s % 9) for s in range(S)], H=16)
    rg = wl.rg
    seq, cu_q, cu_kv, pages = meta_to(rg, DEV)
    # a buffer with other integers in front, where a lookup below index 0 would show
    off = torch.full((S + 65,), 2**30, dtype=torch.int32, device=DEV)[64:]
    off.copy_(cu_q + 3)
    rows = torch.randn(S + 3, 576, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    cache = torch.full((rg.num_pages, 64, 416), 9, dtype=torch.uint8, device=DEV)
    dsa.dsa_q4_write_back(rows, cache, seq, off, cu_kv, pages, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == BAD_METADATA
    pos = rg.token_pos()
    slots = rg.page_indices[rg.cu_kv_lens[np.arange(S)] // 64 + pos // 64].astype(np.int64) * 64 + pos % 64
    want = np.full((rg.num_pages * 64, 416), 9, np.uint8)
    want[slots] = R.q4_pack(rows[3:].cpu())
    assert np.array_equal(cache.cpu().numpy().reshape(-1, 416), want)
    # and the attention over them: the requests' tokens as with valid offsets
    q = torch.randn(S + 3, 16, 576, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    o, lse = dsa.dsa_window_mla(q, wl.kv[0].to(DEV), seq, off, cu_kv, pages, max_kv=rg.max_kv, sm_scale=wl.sm_scale,
                                sliding_window=40, num_sinks=2, want_lse=True)
    torch.cuda.synchronize()

    def seen(t):
        j = np.arange(pos[t] + 1)
        return j[(j > pos[t] - 40) | (j < 2)]
    flat = R.f64(wl.kv[0]).reshape(-1, 576)
    R.check_attend(o[3:], lse[3:], R.attend(R.f64(q)[3:], R.token_keys(rg, flat, seen), wl.sm_scale), f"{S} requests")
