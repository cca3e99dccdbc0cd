"""LayerRunner's forms that chain the operators around the attention over
several layers (IndexShare) and from host buffers: 4-bit caches, tables from
lengths, rotation. Every layer is checked against the plain references on the
rows that its cache holds."""
import numpy as np
import pytest
import torch

import dsa_inputs as DI
import oracle as O
import steps_ref as R
from gpu_util import check_topk_rows, f32

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


def _workload(kind, types=(0, 1, 0)):
    """Three layers: a full one, one that shares its selections, a full one."""
    lens = ([1, 40, 0, 7], [400, 300, 64, 900]) if kind == "prefill" else ([1, 1, 1], [700, 64, 1025])
    wl = DI.random_small(81, *lens, H=16, k=96, k_pages=4)
    bf = lambda t, seed, what: DI.randn(tuple(t.shape), seed, what).to(torch.bfloat16)
    for layer in range(1, len(types)):
        wl.q.append(bf(wl.q[0], 82 + layer, "q"))
        wl.kv.append(bf(wl.kv[0], 82 + layer, "kv"))
        if types[layer] == 0:
            wl.kcache.append(bf(wl.kcache[0], 82 + layer, "kcache"))
    wl.indexer_types = list(types)
    wl.QB = 32
    return wl


def _check_layers(run, wl, kind, pos, q=None):
    """Selections and outputs of every layer from the inputs that it had; `q`:
    the layers' queries where the runner's own are not what they attended."""
    rg, paged = wl.rg, kind == "prefill"
    for layer, ty in enumerate(wl.indexer_types):
        slot = run.src_slot[layer]
        sel = (run.topk_pages if paged else run.topk)[slot].cpu().numpy()
        if ty == 0:
            kc = f32(run.kcache[slot]).reshape(rg.num_pages, 64, 128)
            _, scores = O.indexer_topk(f32(run.q_idx), f32(run.w), kc, rg.seq_lens, rg.cu_q_lens, rg.cu_kv_lens,
                                       rg.page_indices, wl.k)
            if paged:
                scores = [O.page_scores_of_row(r, 64) for r in scores]
            check_topk_rows(sel, O.topk_rows_of(scores, sel.shape[1]), sel.shape[1], scores)
        live = lambda t: sel[t][sel[t] >= 0].astype(np.int64)
        of = (lambda t: (live(t)[:, None] * 64 + np.arange(64)).reshape(-1)) if paged else live
        flat = (R.q4_values(run.kv4[layer].cpu().numpy().reshape(-1, 416)) if run.cache_bits == 4
                else R.f64(run.kv[layer]).reshape(-1, 576))
        o, _, otol, _ = R.attend(R.f64(run.q[layer] if q is None else q[layer]), R.token_keys(rg, flat, of), wl.sm_scale)
        e = np.abs(R.f64(run.o[layer]) - o) - otol
        assert (e <= 0).all(), (layer, e.max())


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("bits", [4, 16])
def test_layers_that_share_selections(dsa, kind, bits):
    from deepseek_sparse_attention_score_gb300.layer import LayerRunner

    wl = _workload(kind)
    rg, pos = wl.rg, wl.rg.token_pos()
    freqs, _ = dsa.dsa_rope_freqs(64, scaling="yarn", factor=4.0, orig_max_pos=256)
    scale, logits = dsa.dsa_rope_attention_scales(4.0, mscale=1.0, mscale_all_dim=0.5)
    wl.sm_scale *= logits
    run = LayerRunner(wl, DEV, cache_bits=bits, tables=True, rope=(freqs, scale, "interleaved"))
    before = [c.clone() for c in (run.kv4 if bits == 4 else run.kv)]
    run.step()
    run.step()  # the same step again: rotation starts from the rows that are not rotated
    torch.cuda.synchronize()
    assert run.status.item() == 0
    slots = run.tables.slots.cpu().numpy()
    for layer in range(3):
        # rotated queries and rows of every layer, shared ones too
        for got, raw, off in ((run.q[layer], wl.q[layer], 512),
                              (run.new_kv[layer][:, None], wl.kv[layer].view(-1, 576)[slots][:, None], 512)):
            want, mag = R.rope(R.f64(raw), pos, freqs.numpy(), off, "interleaved", scale, False)
            err = np.abs(R.f64(got) - want) - R.rope_tol(want, mag, torch.bfloat16)
            assert (err[..., off:] <= 0).all(), layer
            assert torch.equal(got[..., :off].cpu(), raw[..., :off])
        # the cache: the new rows where they belong, the others as they were
        cache = (run.kv4 if bits == 4 else run.kv)[layer]
        want = before[layer].cpu().view(rg.num_pages * 64, -1).clone()
        new = run.new_kv[layer].cpu()
        want[slots] = torch.from_numpy(R.q4_pack(new)) if bits == 4 else new
        assert torch.equal(cache.cpu().view(rg.num_pages * 64, -1), want)
    _check_layers(run, wl, kind, pos)
    if bits == 4:  # buffers of the forms that this runner never takes
        assert not any(hasattr(run, a) for a in ("ws_att", "units", "member", "counts"))


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("bits,tables", [(4, False), (16, True), (4, True)])
def test_step_from_host_buffers(dsa, kind, bits, tables):
    """step_host over a 4-bit cache and from lengths: eager, then captured and
    replayed, equal to the resident step."""
    from deepseek_sparse_attention_score_gb300.layer import LayerRunner

    wl = _workload(kind)
    run = LayerRunner(wl, DEV, cache_bits=bits, tables=tables)
    pin = lambda t: t.detach().to("cpu").pin_memory()
    host = dict(q_idx=pin(run.q_idx), w=pin(run.w), q=[pin(x) for x in run.q],
                meta=[pin(m) for m in (run.lens if tables else run.meta)],
                topk=torch.empty(run.topk[0].shape, dtype=torch.int32).pin_memory(),
                o=[torch.empty(x.shape, dtype=torch.bfloat16).pin_memory() for x in run.o],
                new_kv=[pin(x) for x in run.new_kv], new_k=[pin(x) for x in run.new_k])
    run.step()
    torch.cuda.synchronize()
    assert run.status.item() == 0
    _check_layers(run, wl, kind, wl.rg.token_pos())
    ref_topk, ref_o = run.topk[0].cpu().clone(), [x.cpu().clone() for x in run.o]
    side = torch.cuda.Stream()

    def call():
        run.step_host(host["q_idx"], host["w"], host["q"], host["meta"], host["topk"], host["o"], side,
                      h_new_kv=host["new_kv"], h_new_k=host["new_k"])

    def clobber():
        for t in [run.q_idx, *run.q, *run.new_kv, *run.new_k]:
            t.zero_()
        if tables:  # everything that the lengths stand for has to be found again
            for t in [*run.lens, *run.meta[1:]]:
                t.fill_(-7)
        host["topk"].fill_(-5)
        for x in [*run.o, *host["o"]]:
            x.fill_(7.0)
        torch.cuda.synchronize()

    def same():
        torch.cuda.synchronize()
        assert run.status.item() == 0
        assert torch.equal(host["topk"], ref_topk)
        for a, b in zip(host["o"], ref_o):
            torch.testing.assert_close(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-4)

    clobber()
    call()
    same()
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s2):
        call()
    torch.cuda.synchronize()
    for _ in range(2):
        clobber()
        g.replay()
        same()


def test_host_step_refuses_rotation(dsa):
    from deepseek_sparse_attention_score_gb300.layer import LayerRunner

    wl = _workload("decode", (0,))
    run = LayerRunner(wl, DEV, tables=True, rope=(dsa.dsa_rope_freqs(64)[0], 1.0, "half"))
    with pytest.raises(ValueError):
        run.step_host(None, None, None, None, None, None, None)
