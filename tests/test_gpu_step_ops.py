"""The operators around the attention as a step uses them together: lengths ->
page tables -> rotary positions -> (4-bit) write-back -> indexer -> attention,
through LayerRunner, against the plain references and the oracle; captured in
a graph; and chained without a layer for windowed attention."""
import numpy as np
import pytest
import torch

import dsa_inputs as DI
import oracle as O
import steps_ref as R
from gpu_util import check_topk_rows, f32, meta_np

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


def _rotated(x, pos, freqs, off, layout, scale):
    """bf16 tensor [T, H, D] with 64 columns turned in 64 bits and rounded."""
    y, _ = R.rope(R.f64(x), pos, freqs.numpy(), off, layout, scale, False)
    return torch.from_numpy(y).to(torch.bfloat16)


def _near(got, want):
    """Equal but for results that lie within the fp32 arithmetic's error of a
    rounding boundary (one bf16 step apart, rarely)."""
    d = (got.cpu().double() - want.double()).abs()
    assert (d <= 2.0 ** -7 * want.double().abs() + 1e-6).all()
    assert (d > 0).double().mean() < 1e-3


@pytest.mark.parametrize("case", ["decode", "budget", "prefill"])
@pytest.mark.parametrize("bits", [4, 16])
def test_step_from_lengths(dsa, case, bits):
    from deepseek_sparse_attention_score_gb300.layer import LayerRunner

    q_lens, kv_lens = ([1, 40, 0, 7], [400, 300, 64, 900]) if case == "prefill" else ([1, 1, 1], [700, 64, 1025])
    wl = DI.random_small(31, q_lens, kv_lens, H=16, k=96, k_pages=4)
    wl.QB = 32  # query blocks of the bf16 prefill path
    rg = wl.rg
    freqs, scale = dsa.dsa_rope_freqs(64, scaling="yarn", factor=4.0, orig_max_pos=256)
    run = LayerRunner(wl, DEV, page_budget=3 if case == "budget" else None, cache_bits=bits, tables=True,
                      rope=(freqs, scale, "interleaved"))
    run.meta[3].fill_(-9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # on a stream of its own
        run.step()
    side.synchronize()
    assert run.status.item() == 0
    # tables: the workload's own metadata, from its lengths
    for got, want in zip(run.meta, (rg.seq_lens, rg.cu_q_lens, rg.cu_kv_lens, rg.page_indices)):
        assert np.array_equal(got.cpu().numpy(), want)
    pos = rg.token_pos()
    assert np.array_equal(run.tables.positions.cpu().numpy(), pos)
    # rotary positions
    _near(run.q[0][:, :, 512:], _rotated(wl.q[0], pos, freqs, 512, "interleaved", scale)[:, :, 512:])
    assert torch.equal(run.q[0][:, :, :512].cpu(), wl.q[0][:, :, :512])
    _near(run.q_idx, _rotated(wl.q_idx, pos, freqs, 0, "half", 1.0))
    # the new rows in their slots, every other row as generated
    slots = run.tables.slots.cpu().numpy()
    assert np.array_equal(slots, rg.page_indices[rg.cu_kv_lens[rg.token_seq()] // 64 + pos // 64] * 64 + pos % 64)
    old = wl.kv[0].view(-1, 576)
    _near(run.new_kv[0], _rotated(old[slots][:, None], pos, freqs, 512, "interleaved", scale)[:, 0])
    rows = old.clone()
    rows[slots] = run.new_kv[0].cpu()
    if bits == 4:
        packed = R.q4_pack(rows)
        assert np.array_equal(run.kv4[0].cpu().numpy().reshape(-1, 416), packed)
        flat = R.q4_values(packed)
    else:
        assert torch.equal(run.kv[0].view(-1, 576).cpu(), rows)
        flat = R.f64(rows)
    # selections from the caches as written
    kc = wl.kcache[0].view(-1, 128).clone()
    kc[slots] = run.new_k[0].cpu()
    assert torch.equal(run.kcache[0].view(-1, 128).cpu(), kc)
    _, scores = O.indexer_topk(f32(run.q_idx), f32(wl.w), f32(kc).reshape(rg.num_pages, 64, 128), rg.seq_lens,
                               rg.cu_q_lens, rg.cu_kv_lens, rg.page_indices, wl.k)
    paged = case != "decode"
    if paged:
        scores = [O.page_scores_of_row(r, 64) for r in scores]
    sel = (run.topk_pages if paged else run.topk)[0].cpu().numpy()
    check_topk_rows(sel, O.topk_rows_of(scores, sel.shape[1]), sel.shape[1], scores)
    # attention over them
    live = lambda t: sel[t][sel[t] >= 0].astype(np.int64)
    of = (lambda t: (live(t)[:, None] * 64 + np.arange(64)).reshape(-1)) if paged else live
    o, lse, otol, _ = R.attend(R.f64(run.q[0]), R.token_keys(rg, flat, of), wl.sm_scale)
    e = np.abs(R.f64(run.o[0]) - o) - otol
    assert (e <= 0).all(), e.max()


def test_captured_step_follows_its_lengths(dsa):
    """One captured decode step, replayed while the requests grow over a page
    boundary: each replay equals an eager step of the new lengths."""
    from deepseek_sparse_attention_score_gb300.layer import LayerRunner

    wl = DI.random_small(32, [1, 1], [127, 300], H=16, k=64)
    run = LayerRunner(wl, DEV, cache_bits=4, tables=True)
    # room for the pages that growth takes
    run.PTW += 2
    grown = torch.full((2, run.block_table.shape[1] + 1), -1, dtype=torch.int32, device=DEV)
    grown[:, :-1] = run.block_table
    run.block_table = grown
    spare = sorted(set(range(wl.rg.num_pages)) - set(wl.rg.page_indices.tolist()))
    run.free_pages = torch.tensor(spare, dtype=torch.int32, device=DEV)
    pages = torch.empty(run.PTW, dtype=torch.int32, device=DEV)
    run.tables = run.tables._replace(page_indices=pages)
    run.meta[3] = pages
    run.max_kv += 8
    run.ws_idx = torch.empty(dsa.dsa_indexer_workspace_size(2, 2, run.max_kv, 64), dtype=torch.uint8, device=DEV)
    run.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run.step()
    cache0 = run.kv4[0].clone()
    for lens in ([127, 300], [128, 301], [129, 302]):  # request 0 enters its third page
        run.lens[1].copy_(torch.tensor(lens, dtype=torch.int32))
        run.kv4[0].copy_(cache0)
        run.step()
        torch.cuda.synchronize()
        want = [run.o[0].clone(), run.topk[0].clone(), run.kv4[0].clone(), pages.clone()]
        run.kv4[0].copy_(cache0)
        for x in (run.o[0], run.topk[0], pages):
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert run.status.item() == 0
        assert all(torch.equal(a, b) for a, b in zip(want, (run.o[0], run.topk[0], run.kv4[0], pages)))
    assert run.tables.n_taken.item() == 1 and pages[2].item() == spare[0]


def test_window_after_tables_and_rope(dsa):
    """A layer without an indexer: tables, rotation straight into the latent
    rows and queries, write-back, windowed attention with sinks."""
    wl = DI.random_small(33, [1, 30, 5], [500, 200, 333], H=16)
    rg = wl.rg
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a.astype(np.int32))).to(DEV)
    need = -(-rg.seq_lens // 64)
    bt = np.full((3, need.max()), -1)
    for s in range(3):
        bt[s, : need[s]] = rg.page_indices[rg.cu_kv_lens[s] // 64:][: need[s]]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    seq = to(rg.seq_lens)
    tb = dsa.dsa_build_page_tables(to(rg.q_lens), seq, to(bt), T=rg.T, PTW=rg.PTW, dev_status=st)
    # block tables that hold every page: the entries past the old ones are
    # taken from the (empty) free list, so they have to be there already
    assert st.item() == 0x20
    st.zero_()
    had = -(-(rg.seq_lens - rg.q_lens) // 64)
    free = np.concatenate([bt[s, had[s]: need[s]] for s in range(3)])
    tb = dsa.dsa_build_page_tables(to(rg.q_lens), seq, to(bt), to(free), T=rg.T, PTW=rg.PTW, dev_status=st)
    meta = (seq, tb.cu_q_lens, tb.cu_kv_lens, tb.page_indices)
    freqs, scale = dsa.dsa_rope_freqs(64, device=DEV)
    q, rows = wl.q[0].to(DEV), torch.randn(rg.T, 1, 576, device=DEV).to(torch.bfloat16)
    kv = wl.kv[0].to(DEV)
    dsa.dsa_rope([dsa.RopeTarget(q, rot_off=512), dsa.RopeTarget(rows, rot_off=512)], tb.positions, freqs)
    dsa.dsa_paged_write_back(rows[:, 0], kv, *meta, dev_status=st)
    o, lse = dsa.dsa_window_mla(q, kv, *meta, max_kv=500, sm_scale=wl.sm_scale, sliding_window=100, num_sinks=4,
                                want_lse=True, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    pos = rg.token_pos()
    flat = R.f64(wl.kv[0]).reshape(-1, 576)
    flat[tb.slots.cpu().numpy()] = R.f64(rows[:, 0])

    def seen(t):
        j = np.arange(pos[t] + 1)
        return j[(j > pos[t] - 100) | (j < 4)]
    R.check_attend(o, lse, R.attend(R.f64(q), R.token_keys(rg, flat, seen), wl.sm_scale), "step")


def test_runner_refusals(dsa):
    from deepseek_sparse_attention_score_gb300.layer import LayerRunner

    wl = DI.random_small(34, [1], [64], H=16)
    with pytest.raises(ValueError):
        LayerRunner(wl, DEV, cache_bits=8)
    with pytest.raises(ValueError):
        LayerRunner(wl, DEV, rope=(dsa.dsa_rope_freqs(64)[0], 1.0, "half"))
