"""The 4-bit latent cache: quantising write-back and read (bytes and values
equal to the plain quantiser), special values, and the sparse attention over
it inside element-wise error bounds: units, page sizes, heads, splits, masks
that leave a row empty, bad pages, NaN in rows that are not selected."""
import numpy as np
import pytest
import torch

import dsa_inputs as DI
import steps_ref as R
from gpu_util import meta_to

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


DEV = torch.device("cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _slots(rg):
    s, p = rg.token_seq(), rg.token_pos()
    ent = rg.cu_kv_lens[s] // rg.page_size + p // rg.page_size
    return rg.page_indices[ent].astype(np.int64) * rg.page_size + p % rg.page_size


def _rows(n, seed=0):
    """Rows of unlike size, with ties, zeros and the format's ends among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, 576), generator=g)
    x[:, :512] *= torch.exp(2 * torch.randn((n, 32), generator=g)).repeat_interleave(16, 1)
    x = x.to(torch.bfloat16)
    ties = torch.tensor([6, .25, -.25, .75, -.75, 1.25, 1.75, 2.5, -2.5, 3.5, 5, -5, 0, -0.0, .5, 4])
    for i in range(min(n, 8)):
        x[i, :16] = (ties * 2.0 ** (i - 4)).to(torch.bfloat16)
        x[i, 16:32] = 0
        x[i, 32:48] = (ties * 2.0 ** -(7 + i)).to(torch.bfloat16)   # scales down to where they vanish
        x[i, 48:64] = (ties * 2.0 ** (4 + i)).to(torch.bfloat16)    # and up to where they saturate
        x[i, 64:80] = torch.randn(16, generator=g).to(torch.bfloat16) * (3.3e38 if i == 1 else 1.0)
        x[i, 80] = 6 * (1 + (2 * i + 1) / 16)                       # the scale itself ties
    return x.to(DEV)


@pytest.mark.parametrize("q_lens,kv_lens,ps", [
    ([1], [1], 64), ([1, 1, 1], [700, 64, 65], 32), ([130], [130], 128), ([1, 45, 0, 7], [500, 300, 40, 1000], 64),
])
def test_write_back_and_read(dsa, q_lens, kv_lens, ps):
    rg = DI.make_ragged(q_lens, kv_lens, ps, master_seed=3, spare_pages=2)
    rows, st = _rows(rg.T, 5), _status()
    cache = torch.randint(0, 255, (rg.num_pages, ps, 416), dtype=torch.uint8, device=DEV)
    before = cache.cpu().numpy().reshape(-1, 416)
    dsa.dsa_q4_write_back(rows, cache, *meta_to(rg, DEV), dev_status=st)
    slots = _slots(rg)
    got = cache.cpu().numpy().reshape(-1, 416)
    want = before.copy()
    want[slots] = R.q4_pack(rows)
    assert np.array_equal(got, want)  # the rows' bytes, and every other row as it was
    sl = torch.from_numpy(np.concatenate([slots, [-1, 0]]).astype(np.int32)).to(DEV)
    out = dsa.dsa_q4_read_rows(cache, sl, dev_status=st)
    vals = R.q4_values(got[np.concatenate([slots, [0]])])
    assert np.array_equal(R.f64(out)[:-2], vals[:-1], equal_nan=True) and (out[-2] == 0).all()
    assert np.array_equal(R.f64(out)[-1], vals[-1], equal_nan=True)
    assert st.item() == 0


def test_strided_rows(dsa):
    rg = DI.make_ragged([9], [40], 64, master_seed=1)
    wide = torch.randn(9, 640, device=DEV).to(torch.bfloat16)
    a, b = (torch.zeros(rg.num_pages, 64, 416, dtype=torch.uint8, device=DEV) for _ in range(2))
    dsa.dsa_q4_write_back(wide[:, :576], a, *meta_to(rg, DEV))
    dsa.dsa_q4_write_back(wide[:, :576].contiguous(), b, *meta_to(rg, DEV))
    assert torch.equal(a, b) and a.any()
    out = torch.full((9, 640), 7.0, dtype=torch.bfloat16, device=DEV)
    sl = torch.from_numpy(_slots(rg).astype(np.int32)).to(DEV)
    dsa.dsa_q4_read_rows(a, sl, out=out)
    assert torch.equal(out[:, :576], dsa.dsa_q4_read_rows(a, sl)) and (out[:, 576:] == 7).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_not_finite_groups_read_as_nan(dsa, bad):
    rg = DI.make_ragged([2], [2], 64, master_seed=1)
    rows = _rows(2)
    rows[1, 100] = bad      # group 6
    rows[1, 575] = bad      # a rotary dim: copied
    cache = torch.zeros(rg.num_pages, 64, 416, dtype=torch.uint8, device=DEV)
    dsa.dsa_q4_write_back(rows, cache, *meta_to(rg, DEV))
    out = R.f64(dsa.dsa_q4_read_rows(cache, torch.from_numpy(_slots(rg).astype(np.int32)).to(DEV)))
    x = R.f64(rows)  # group 4 of row 1 overflowed to infinities when it was made
    want = np.isnan(x)
    want[:, :512] = (~np.isfinite(x[:, :512])).reshape(2, 32, 16).any(2).repeat(16, 1)
    assert want[1, 96:112].all() and np.array_equal(np.isnan(out), want)
    assert bad != bad or out[1, 575] == bad


def test_write_back_outside_the_cache_is_skipped(dsa):
    rg = DI.make_ragged([1, 1, 1], [100, 70, 64], 64, master_seed=2)
    meta = meta_to(rg, DEV)
    meta[3] = meta[3].clone()
    meta[3][1] = rg.num_pages      # request 0's second page
    meta[3][3] = -1                # request 1's
    cache = torch.zeros(rg.num_pages, 64, 416, dtype=torch.uint8, device=DEV)
    st = _status()
    dsa.dsa_q4_write_back(_rows(3), cache, *meta, dev_status=st)
    assert st.item() == 0x2
    assert cache.view(-1, 416).any(1).sum().item() == 1
    st.zero_()
    out = dsa.dsa_q4_read_rows(cache, torch.tensor([rg.num_pages * 64, 2**31 - 1], dtype=torch.int32, device=DEV),
                               dev_status=st)
    assert st.item() == 0x4 and (out == 0).all()


# ---------------------------------------------------------------- attention
def _batch(q_lens, kv_lens, ps, H, seed=0):
    rg = DI.make_ragged(q_lens, kv_lens, ps, master_seed=seed + 1, spare_pages=2)
    g = torch.Generator().manual_seed(seed)
    pool = R.q4_pack(torch.randn((500, 576), generator=g).to(torch.bfloat16))
    rows = np.random.default_rng(seed).integers(0, len(pool), rg.num_pages * ps)
    cache = torch.from_numpy(pool[rows]).view(rg.num_pages, ps, 416)
    q = torch.randn((rg.T, H, 576), generator=g).to(torch.bfloat16)
    return rg, cache, q


def _select(rg, K, unit, rng, empty=()):
    n = rg.token_pos() + 1
    sel = np.full((rg.T, K), -1, np.int32)
    for t in range(rg.T):
        m = int(n[t]) if unit == 1 else -(-int(n[t]) // unit)
        pick = rng.permutation(m)[:K]
        sel[t, rng.permutation(K)[: len(pick)]] = pick  # any order, -1 anywhere
    for t in empty:
        sel[t] = -1
    return sel


def _positions(sel, unit):
    def of(t):
        j = sel[t][sel[t] >= 0].astype(np.int64)
        return j if unit == 1 else (j[:, None] * unit + np.arange(unit)).reshape(-1)
    return of


def _run(dsa, rg, cache, q, sel, unit, **kw):
    st = _status()
    o, lse = dsa.dsa_sparse_mla_decode_q4(q.to(DEV), cache.to(DEV), *meta_to(rg, DEV), torch.from_numpy(sel).to(DEV),
                                          unit=unit, sm_scale=DI.SM_SCALE, want_lse=True, dev_status=st, **kw)
    torch.cuda.synchronize()
    return o, lse, st.item()


def _check(dsa, rg, cache, q, sel, unit, what, **kw):
    o, lse, st = _run(dsa, rg, cache, q, sel, unit, **kw)
    assert st == 0
    flat = R.q4_values(cache.numpy().reshape(-1, 416))
    ref = R.attend(R.f64(q), R.token_keys(rg, flat, _positions(sel, unit)), DI.SM_SCALE)
    R.check_attend(o, lse, ref, what)
    return o, lse


@pytest.mark.parametrize("ps", [32, 64, 128])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("q_lens,kv_lens,H,K", [
    ([1], [1], 1, 1),
    ([1], [40], 16, 33),
    ([1, 1, 1], [300, 64, 129], 128, 70),
    ([1, 5, 0, 3], [200, 100, 40, 257], 7, 64),
    ([1, 1], [90, 400], 130, 257),     # two groups of heads
])
def test_attention(dsa, ps, paged, q_lens, kv_lens, H, K):
    rg, cache, q = _batch(q_lens, kv_lens, ps, H, seed=H + K)
    unit = ps if paged else 1
    sel = _select(rg, K if not paged else 1 + K // 16, unit, np.random.default_rng(K))
    _check(dsa, rg, cache, q, sel, unit, f"ps {ps} unit {unit}")


@pytest.mark.parametrize("K,unit", [(2048, 1), (2047, 1), (37, 64), (9, 64)])
def test_long_selections_split(dsa, K, unit):
    """One request: the selection is split over CTAs and merged, the same on
    every run."""
    rg, cache, q = _batch([1, 1], [2600, 1900], 64, 32, seed=4)
    sel = _select(rg, K, unit, np.random.default_rng(1))
    o, lse = _check(dsa, rg, cache, q, sel, unit, "split")
    for _ in range(3):
        o2, lse2, _ = _run(dsa, rg, cache, q, sel, unit)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H", [1, 33, 64, 65])
@pytest.mark.parametrize("S,K,unit", [(12, 1024, 1), (24, 512, 1), (24, 9, 64), (48, 130, 1), (90, 63, 1), (160, 1, 64)])
def test_many_requests(dsa, S, K, unit, H):
    """More requests than run at once in two CTAs each: up to 64 heads take one,
    over 8, 4, 2 and 1 splits. Some rows select nothing, one has a NaN query."""
    kv = [1 + (K * unit + 97 * s) % (K * unit + 64) for s in range(S)]
    rg, cache, q = _batch([1] * S, kv, 64, H, seed=S + H)
    sel = _select(rg, K, unit, np.random.default_rng(S), empty=(1, S - 1))
    o, lse = _check(dsa, rg, cache, q, sel, unit, f"{S} requests")
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    q[2, H // 2, 3] = float("nan")  # its own row only
    o2, lse2, st = _run(dsa, rg, cache, q, sel, unit)
    row = torch.zeros((S, H), dtype=torch.bool, device=DEV)
    row[2, H // 2] = True
    assert st == 0 and torch.isnan(o2[row]).all() and torch.isnan(lse2[row]).all()
    assert torch.equal(o[~row], o2[~row]) and torch.equal(lse[~row], lse2[~row])


@pytest.mark.parametrize("unit", [1, 64])
def test_rows_that_select_nothing(dsa, unit):
    rg, cache, q = _batch([1, 1, 1], [300, 500, 64], 64, 16, seed=5)
    sel = _select(rg, 40, unit, np.random.default_rng(2), empty=(0, 2))
    o, lse = _check(dsa, rg, cache, q, sel, unit, "empty rows")
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()
    sel[1] = 600 if unit == 1 else 9  # only positions past the request: nothing either
    o, lse, st = _run(dsa, rg, cache, q, sel, unit)
    assert st == 0 and (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("unit", [1, 64])
def test_entries_listed_twice_count_twice(dsa, unit):
    rg, cache, q = _batch([1, 2], [300, 200], 64, 16, seed=15)
    sel = _select(rg, 60 if unit == 1 else 3, unit, np.random.default_rng(5))
    sel[:, 1], sel[0, 2] = sel[:, 0], sel[0, 0]
    _check(dsa, rg, cache, q, sel, unit, "twice")


def test_padding_rows_are_left_alone(dsa):
    """T as an upper bound of the tokens: three rows behind the last request."""
    rg, cache, q = _batch([1, 4, 0], [300, 200, 64], 64, 16, seed=17)
    sel = _select(rg, 130, 1, np.random.default_rng(7))
    q2 = torch.cat([q, torch.full((3, 16, 576), float("nan"), dtype=torch.bfloat16)]).to(DEV)
    sel2 = torch.from_numpy(np.concatenate([sel, np.zeros((3, 130), np.int32)])).to(DEV)
    o, lse = torch.full((8, 16, 512), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((8, 16), 7.0, device=DEV)
    st = _status()
    dsa.dsa_sparse_mla_decode_q4(q2, cache.to(DEV), *meta_to(rg, DEV), sel2, unit=1, sm_scale=DI.SM_SCALE, o=o,
                                 lse=lse, dev_status=st)
    assert st.item() == 0 and (o[5:] == 7).all() and (lse[5:] == 7).all()
    flat = R.q4_values(cache.numpy().reshape(-1, 416))
    R.check_attend(o[:5], lse[:5], R.attend(R.f64(q), R.token_keys(rg, flat, _positions(sel, 1)), DI.SM_SCALE),
                   "padded")
    # and in the write-back: rows behind the last request go nowhere
    rows = _rows(8, 9)
    a, b = (torch.zeros_like(cache, device=DEV) for _ in range(2))
    dsa.dsa_q4_write_back(rows, a, *meta_to(rg, DEV), dev_status=st)
    dsa.dsa_q4_write_back(rows[:5], b, *meta_to(rg, DEV), dev_status=st)
    assert st.item() == 0 and torch.equal(a, b) and a.any()


@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_scales_of_zero_and_below(dsa, scale):
    rg, cache, q = _batch([1], [300], 64, 16, seed=16)
    sel = _select(rg, 130, 1, np.random.default_rng(6))
    o, lse = dsa.dsa_sparse_mla_decode_q4(q.to(DEV), cache.to(DEV), *meta_to(rg, DEV), torch.from_numpy(sel).to(DEV),
                                          unit=1, sm_scale=scale, want_lse=True)
    flat = R.q4_values(cache.numpy().reshape(-1, 416))
    R.check_attend(o, lse, R.attend(R.f64(q), R.token_keys(rg, flat, _positions(sel, 1)), scale), f"scale {scale}")


@pytest.mark.parametrize("unit", [1, 64])
def test_unselected_and_unwritten_rows_may_hold_anything(dsa, unit):
    rg, cache, q = _batch([1, 3], [300, 200], 64, 16, seed=6)
    sel = _select(rg, 100 if unit == 1 else 3, unit, np.random.default_rng(3))
    o, lse = _check(dsa, rg, cache, q, sel, unit, "clean")
    keep = np.zeros(rg.num_pages * 64, bool)
    seq, pos = rg.token_seq(), rg.token_pos()
    for t in range(rg.T):
        j = _positions(sel, unit)(t)
        j = j[j <= pos[t]]
        keep[rg.page_indices[rg.cu_kv_lens[seq[t]] // 64 + j // 64].astype(np.int64) * 64 + j % 64] = True
    dirty = cache.clone().view(-1, 416)
    dirty[torch.from_numpy(~keep)] = 0x7F  # NaN scales, NaN rotary dims
    o2, lse2, st = _run(dsa, rg, dirty.view_as(cache), q, sel, unit)
    assert st == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("unit", [1, 64])
def test_selected_nan_shows(dsa, unit):
    rg, cache, q = _batch([1], [64], 64, 16, seed=7)
    cache.view(-1, 416)[int(rg.page_indices[0]) * 64 + 5, 256 + 3] = 0x7F
    sel = np.zeros((1, 6), np.int32) if unit == 64 else np.arange(6, dtype=np.int32)[None]
    o, lse, _ = _run(dsa, rg, cache, q, sel, unit)
    assert torch.isnan(o).all() and torch.isnan(lse).all()


def test_bad_pages_are_skipped(dsa):
    rg, cache, q = _batch([1, 1], [200, 128], 64, 16, seed=8)
    meta = meta_to(rg, DEV)
    meta[3] = meta[3].clone()
    meta[3][1], meta[3][2] = rg.num_pages, -5
    st = _status()
    sel = np.tile(np.arange(200, dtype=np.int32), (2, 1))
    o, lse = dsa.dsa_sparse_mla_decode_q4(q.to(DEV), cache.to(DEV), *meta, torch.from_numpy(sel).to(DEV), unit=1,
                                          sm_scale=DI.SM_SCALE, want_lse=True, dev_status=st)
    assert st.item() == 0x2
    flat = R.q4_values(cache.numpy().reshape(-1, 416))
    live = [np.r_[0:64, 192:200], np.arange(128)]
    R.check_attend(o, lse, R.attend(R.f64(q), R.token_keys(rg, flat, lambda t: live[t]), DI.SM_SCALE), "bad pages")


def test_two_captured_graphs_at_once(dsa):
    rg, cache, q = _batch([1, 1], [1500, 900], 64, 16, seed=9)
    sel = _select(rg, 700, 1, np.random.default_rng(4))
    want, lse, _ = _run(dsa, rg, cache, q, sel, 1)
    dc, dq, ds, meta = cache.to(DEV), q.to(DEV), torch.from_numpy(sel).to(DEV), meta_to(rg, DEV)
    graphs = []
    for _ in range(2):
        o = torch.zeros_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dsa.dsa_sparse_mla_decode_q4(dq, dc, *meta, ds, unit=1, sm_scale=DI.SM_SCALE, o=o)
        graphs.append((g, o, torch.cuda.Stream()))
    for _ in range(5):
        for g, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for _, o, _ in graphs)


def test_offsets_past_32_bits(dsa):
    """A cache of 4.8 GB whose requests lie at its end."""
    P, ps = 90112, 128
    rg = DI.make_ragged([1, 130], [200, 300], ps, master_seed=3)
    rg.page_indices = (P - 1 - rg.page_indices).astype(np.int32)
    rg.num_pages = P
    cache = torch.zeros((P, ps, 416), dtype=torch.uint8, device=DEV)
    assert cache.numel() > 2**32
    g = torch.Generator().manual_seed(18)
    last = cache[-8:]
    pool = R.q4_pack(torch.randn((8 * ps, 576), generator=g).to(torch.bfloat16))
    last.copy_(torch.from_numpy(pool).view(8, ps, 416))
    rows, st = _rows(rg.T, 19), _status()
    dsa.dsa_q4_write_back(rows, cache, *meta_to(rg, DEV), dev_status=st)
    slots = _slots(rg)
    assert slots.min() * 416 > 2**32
    out = dsa.dsa_q4_read_rows(cache, torch.from_numpy(slots.astype(np.int32)).to(DEV), dev_status=st)
    flat = R.q4_values(last.cpu().numpy().reshape(-1, 416))
    assert np.array_equal(R.f64(out), R.q4_values(R.q4_pack(rows)), equal_nan=True)
    assert np.array_equal(R.f64(out), flat[slots - (P - 8) * ps], equal_nan=True)
    # attention over rows that were there before: positions below the new ones
    q = torch.randn((rg.T, 16, 576), generator=g).to(torch.bfloat16)
    sel = np.tile(np.arange(0, 165, 5, dtype=np.int32), (rg.T, 1))
    o, lse = dsa.dsa_sparse_mla_decode_q4(q.to(DEV), cache, *meta_to(rg, DEV), torch.from_numpy(sel).to(DEV), unit=1,
                                          sm_scale=DI.SM_SCALE, want_lse=True, dev_status=st)
    assert st.item() == 0
    rg.page_indices = (rg.page_indices - (P - 8)).astype(np.int32)
    R.check_attend(o, lse, R.attend(R.f64(q), R.token_keys(rg, flat, _positions(sel, 1)), DI.SM_SCALE), "far rows")
