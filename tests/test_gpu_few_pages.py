"""Page lists and windows shorter than the splits that their keys would fill:
pages are dealt out whole, so some splits are empty or there is only one."""
import numpy as np
import pytest
import torch

import dsa_inputs as DI
import steps_ref as R
from gpu_util import meta_to

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


@pytest.mark.parametrize("K", [1, 2, 3, 5, 9])
@pytest.mark.parametrize("ps", [64, 128])
@pytest.mark.parametrize("H", [16, 128])
def test_page_selections(dsa, ps, K, H):
    wl = DI.random_small(91 + K, [1, 1, 1], [10 * ps + 5, 3, 1200], H=H, page_size=ps)
    rg = wl.rg
    cache = torch.zeros((rg.num_pages, ps, 416), dtype=torch.uint8, device=DEV)
    N = rg.num_pages * ps
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    dsa.dsa_q4_write_back(wl.kv[0].view(N, 576).to(DEV), cache, i32(N), i32(0, N), i32(0, N),
                          torch.arange(rg.num_pages, dtype=torch.int32, device=DEV))
    rng = np.random.default_rng(K)
    sel = np.full((3, K), -1, np.int32)
    for s in range(3):
        n = -(-int(rg.seq_lens[s]) // ps)
        m = min(n, K)
        sel[s, :m] = np.sort(rng.permutation(n)[:m])
    st = i32(0)
    o, lse = dsa.dsa_sparse_mla_decode_q4(wl.q[0].to(DEV), cache, *meta_to(rg, DEV), torch.from_numpy(sel).to(DEV), unit=ps,
                                          sm_scale=wl.sm_scale, want_lse=True, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    flat = R.q4_values(cache.cpu().numpy().reshape(-1, 416))
    of = lambda t: (sel[t][sel[t] >= 0].astype(np.int64)[:, None] * ps + np.arange(ps)).reshape(-1)
    R.check_attend(o, lse, R.attend(R.f64(wl.q[0]), R.token_keys(rg, flat, of), wl.sm_scale), f"{K} pages of {ps}")


@pytest.mark.parametrize("max_kv", [1, 128, 129, 600, 1200])
@pytest.mark.parametrize("H", [16, 128])
def test_windows(dsa, max_kv, H):
    wl = DI.random_small(95, [1, 1], [max_kv, max(1, max_kv // 2)], H=H, page_size=128)
    rg, st = wl.rg, torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = dsa.dsa_window_mla(wl.q[0].to(DEV), wl.kv[0].to(DEV), *meta_to(rg, DEV), max_kv=max_kv, sm_scale=wl.sm_scale,
                                sliding_window=500, num_sinks=4, want_lse=True, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    pos = rg.token_pos()

    def seen(t):
        j = np.arange(pos[t] + 1)
        return j[(j > pos[t] - 500) | (j < 4)]
    flat = R.f64(wl.kv[0]).reshape(-1, 576)
    R.check_attend(o, lse, R.attend(R.f64(wl.q[0]), R.token_keys(rg, flat, seen), wl.sm_scale), f"{max_kv} keys")
