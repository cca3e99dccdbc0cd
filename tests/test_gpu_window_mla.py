"""dsa_window_mla inside element-wise error bounds: windows and sinks that
are apart, touch, overlap or end inside a page; one token and many; splits;
the logit cap; dropped pages between the sinks and the window."""
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


def _visible(rg, window, sinks):
    pos = rg.token_pos()

    def of(t):
        j = np.arange(pos[t] + 1)
        return j if window == 0 else j[(j > pos[t] - window) | (j < sinks)]
    return of


def _run(dsa, wl, window, sinks, cap=0.0, kv=None, meta=None, **kw):
    rg, st = wl.rg, torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = dsa.dsa_window_mla(wl.q[0].to(DEV), (wl.kv[0] if kv is None else kv).to(DEV), *(meta or meta_to(rg, DEV)),
                                max_kv=max(1, rg.max_kv), sm_scale=wl.sm_scale, sliding_window=window,
                                num_sinks=sinks, soft_cap=cap, want_lse=True, dev_status=st, **kw)
    torch.cuda.synchronize()
    return o, lse, st.item()


def _check(dsa, wl, window, sinks, cap=0.0, **kw):
    rg = wl.rg
    o, lse, st = _run(dsa, wl, window, sinks, cap, **kw)
    assert st == 0
    flat = R.f64(wl.kv[0]).reshape(-1, 576)
    ref = R.attend(R.f64(wl.q[0]), R.token_keys(rg, flat, _visible(rg, window, sinks)), wl.sm_scale, cap)
    R.check_attend(o, lse, ref, f"window {window} sinks {sinks} cap {cap}")
    return o, lse


@pytest.mark.parametrize("ps", [32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(100, 4), (1, 1), (64, 64), (33, 130), (257, 37), (5000, 8), (1, 0), (0, 4),
                                          (150, 2**30), (2**31 - 1, 3)])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [700, 64, 301]), ([1, 21, 0, 7], [500, 130, 40, 333])])
def test_matches_64_bit(dsa, ps, window, sinks, q_lens, kv_lens):
    _check(dsa, DI.random_small(ps + window % 97, q_lens, kv_lens, H=16, page_size=ps), window, sinks)


@pytest.mark.parametrize("H", [1, 128, 130])
def test_heads_and_one_token(dsa, H):
    _check(dsa, DI.random_small(H, [1], [1], H=H), 3, 2)
    _check(dsa, DI.random_small(H + 1, [2], [900], H=H), 333, 5)


@pytest.mark.parametrize("H", [1, 3, 43, 64, 65])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 1), (100, 4), (0, 0), (300, 70)])
def test_neighbouring_tokens_share_a_block(dsa, H, window, sinks):
    """Up to 64 heads: runs of 128 / H tokens, at the ends of requests shorter
    ones; a row sees its own window only."""
    _check(dsa, DI.random_small(40 + H, [70, 3, 0, 131, 1], [400, 3, 64, 131, 200], H=H, page_size=32), window, sinks)


def test_many_requests_of_two_tokens(dsa):
    n = 1030  # past the requests that a block searches: one token each
    wl = DI.random_small(45, [2] * n, [2 + s % 40 for s in range(n)], H=2, page_size=32)
    _check(dsa, wl, 8, 2)
    wl = DI.random_small(46, [3] * 200, [3 + s % 40 for s in range(200)], H=2, page_size=32)
    _check(dsa, wl, 8, 2)


@pytest.mark.parametrize("window,sinks", [(1000, 4), (700, 200), (64, 64)])
def test_split_over_ctas(dsa, window, sinks):
    wl = DI.random_small(11, [1, 1], [2600, 1500], H=24)
    o, lse = _check(dsa, wl, window, sinks)
    o2, lse2, _ = _run(dsa, wl, window, sinks)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H", [1, 33, 64, 65])
@pytest.mark.parametrize("S,window,sinks,cap", [(12, 1100, 4, 0.0), (24, 450, 70, 0.0), (48, 66, 1, 2.0), (90, 10, 0, 0.0),
                                                (160, 64, 9, 0.0)])
def test_many_requests_of_one_token(dsa, S, window, sinks, cap, H):
    """More requests than run at once in two CTAs each: up to 64 heads take
    one, over 8, 4, 2 and 1 splits."""
    kv = [1 + 97 * s % (window + 200) for s in range(S)]
    _check(dsa, DI.random_small(50 + S, [1] * S, kv, H=H), window, sinks, cap=cap)


@pytest.mark.parametrize("sinks", [0, 9])
def test_logit_cap(dsa, sinks):
    _check(dsa, DI.random_small(12, [1, 6], [400, 200], H=16), 90, sinks, cap=2.0)


def test_row_stride_640(dsa):
    wl = DI.random_small(13, [1, 9], [700, 300], H=16)
    wide = torch.full((wl.rg.num_pages, 64, 640), float("nan"), dtype=torch.bfloat16)
    wide[:, :, :576] = wl.kv[0]
    o, lse = _check(dsa, wl, 200, 4)
    o2, lse2, st = _run(dsa, wl, 200, 4, kv=wide)
    assert st == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 0), (200, 4)])
def test_padding_rows_are_left_alone(dsa, window, sinks):
    """T as an upper bound: queries and outputs of 3 rows more than tokens."""
    wl = DI.random_small(17, [1, 9, 0], [700, 300, 64], H=16)
    o, lse = _check(dsa, wl, window, sinks)
    q = torch.cat([wl.q[0], torch.full((3, 16, 576), float("nan"), dtype=torch.bfloat16)]).to(DEV)
    o2, lse2 = torch.full((13, 16, 512), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((13, 16), 7.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dsa.dsa_window_mla(q, wl.kv[0].to(DEV), *meta_to(wl.rg, DEV), max_kv=700, sm_scale=wl.sm_scale,
                       sliding_window=window, num_sinks=sinks, o=o2, lse=lse2, dev_status=st)
    assert st.item() == 0 and (o2[10:] == 7).all() and (lse2[10:] == 7).all()
    R.check_attend(o2[:10], lse2[:10], R.attend(R.f64(wl.q[0]), R.token_keys(
        wl.rg, R.f64(wl.kv[0]).reshape(-1, 576), _visible(wl.rg, window, sinks)), wl.sm_scale), "padded")


@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_scales_of_zero_and_below(dsa, scale):
    wl = DI.random_small(18, [2], [300], H=16)
    wl.sm_scale = scale
    _check(dsa, wl, 100, 4)


def test_pages_between_sinks_and_window_are_not_read(dsa):
    """They may be dropped from the table and hold anything."""
    wl = DI.random_small(14, [1, 2], [900, 640], H=16)
    rg = wl.rg
    o, lse = _check(dsa, wl, 130, 4)
    meta = meta_to(rg, DEV)
    kv, pages = wl.kv[0].clone(), rg.page_indices.copy()
    for s, first in ((0, (900 - 130) // 64), (1, (639 - 130) // 64)):
        base = rg.cu_kv_lens[s] // 64
        kv[rg.page_indices[base + 1: base + first]] = float("nan")
        pages[base + 1: base + first] = -1
    meta[3] = torch.from_numpy(pages).to(DEV)
    o2, lse2, st = _run(dsa, wl, 130, 4, kv=kv, meta=meta)
    assert st == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


def test_offsets_past_32_bits(dsa):
    """A cache of 4.8 GB whose requests lie at its end."""
    wl = DI.random_small(19, [1, 3], [400, 200], H=16)
    rg, P = wl.rg, 65536
    big = torch.zeros((P, 64, 576), dtype=torch.bfloat16, device=DEV)
    assert big.numel() * 2 > 2**32
    big[P - rg.num_pages:] = wl.kv[0].to(DEV)
    meta = meta_to(rg, DEV)
    meta[3] = meta[3] + (P - rg.num_pages)
    o, lse = _check(dsa, wl, 100, 4)
    o2, lse2, st = _run(dsa, wl, 100, 4, kv=big, meta=meta)
    assert st == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)
