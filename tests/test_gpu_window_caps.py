"""dsa_window_mla at the ends of the logit cap's and the scale's range: caps
whose reciprocal overflows, caps that leave every logit as it is, and scales
that the kernel's own factor would overflow."""
import ctypes
import math

import numpy as np
import pytest
import torch

import dsa_inputs as DI
import steps_ref as R

INVALID = -1


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


@pytest.mark.parametrize("sm_scale", [3e38, -3e38, math.inf, math.nan])
def test_scale_past_the_range_is_refused(dsa, sm_scale):
    p = ctypes.c_void_p(4096)
    assert dsa.lib().dsa_window_mla(None, p, p, 576, p, p, p, p, 1024, 0, 4, 16, 16, 64, 128, 576, 512, sm_scale, 8, 4,
                                    0.0, p, None, None, 0, None) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [1e-40, 1e-30, 2.0 ** 59, 2.0 ** 60, 1e30, 3e38])
@pytest.mark.parametrize("H", [16, 128])
def test_caps_at_the_ends(dsa, cap, H):
    from gpu_util import meta_to

    dev = torch.device("cuda")
    wl = DI.random_small(71, [1, 5], [200, 90], H=H)
    rg = wl.rg
    q = wl.q[0].clone()
    q[0, 0] = 0     # logits of zero: the cap's factor times zero
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    o, lse = dsa.dsa_window_mla(q.to(dev), wl.kv[0].to(dev), *meta_to(rg, dev), max_kv=rg.max_kv, sm_scale=wl.sm_scale,
                                sliding_window=70, num_sinks=3, soft_cap=cap, want_lse=True, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    pos = rg.token_pos()

    def seen(t):
        j = np.arange(pos[t] + 1)
        return j[(j > pos[t] - 70) | (j < 3)]
    # a cap of 2^59 and more changes no logit of this size in 64 bits
    ref = R.attend(R.f64(q), R.token_keys(rg, R.f64(wl.kv[0]).reshape(-1, 576), seen), wl.sm_scale,
                   cap if cap <= 2.0 ** 59 else 0.0)
    R.check_attend(o, lse, ref, f"cap {cap}")
