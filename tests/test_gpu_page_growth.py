"""A free list over a sequence of steps (dsa_build_page_tables with free_state,
LayerRunner(tables=True)): no page is handed out twice, a step that is repeated
takes the same pages, and a captured step goes on where the last one stopped."""
import numpy as np
import pytest
import torch

import dsa_inputs as DI
import steps_ref as R

pytestmark = pytest.mark.gpu
NO_PAGES = 0x20
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


class Steps:
    """Steps of S requests, on the GPU and by the plain loop."""

    def __init__(self, dsa, S, width, F, T, PTW, ps=64, seed=0):
        self.dsa, self.T, self.PTW, self.ps = dsa, T, PTW, ps
        self.free = np.random.default_rng(seed).permutation(F).astype(np.int32)
        self.bt = np.full((S, width), -1, np.int32)
        self.start, self.last, self.taken = 0, None, 0
        self.g_bt, self.g_free = _i32(self.bt), _i32(self.free)
        self.state = torch.zeros(3 + 2 * S, dtype=torch.int32, device=DEV)
        self.st = torch.zeros(1, dtype=torch.int32, device=DEV)

    def __call__(self, q, seq, new=None):
        """One step; `new`: whether it is (by default when its lengths are)."""
        q, seq = np.asarray(q, np.int32), np.asarray(seq, np.int32)
        lens = (q.tolist(), seq.tolist())
        if self.last is not None and (lens != self.last if new is None else new):
            self.start = min(len(self.free), self.start + self.taken)
        self.last = lens
        want, self.bt, status = R.page_tables(q, seq, self.bt, self.free[self.start:], self.T, self.PTW, self.ps)
        self.taken = min(int(want["n_taken"][0]), len(self.free) - self.start)
        self.st.zero_()
        got = self.dsa.dsa_build_page_tables(_i32(q), _i32(seq), self.g_bt, self.g_free, T=self.T, PTW=self.PTW,
                                             ps=self.ps, free_state=self.state, dev_status=self.st)
        torch.cuda.synchronize()
        for k, v in want.items():
            assert np.array_equal(getattr(got, k).cpu().numpy(), v), k
        assert np.array_equal(self.g_bt.cpu().numpy(), self.bt) and self.st.item() == status
        assert self.state.cpu().tolist() == [0, self.start, self.taken, *q.tolist(), *seq.tolist()]
        return status


@pytest.mark.parametrize("S,ps", [(1, 64), (3, 32), (40, 128), (2047, 64)])
def test_steps_take_pages_one_after_another(dsa, S, ps):
    rng = np.random.default_rng(S)
    n_steps, q_max = 8, 3 * ps
    run = Steps(dsa, S, width=n_steps * 3 + 1, F=n_steps * 4 * S, T=S * q_max + 7, PTW=S * (n_steps * 3 + 1) + 2, ps=ps,
                seed=S)
    seq = np.zeros(S, np.int64)
    for i in range(n_steps):
        q = np.where(rng.random(S) < 0.5, 1, rng.integers(0, q_max + 1, S))
        if i == 0:
            q[0] = 5  # lengths that are not all zeros
        seq = seq + q
        for _ in range(rng.integers(1, 4)):  # the step, and retries of it
            assert run(q, seq) == 0
        held = run.bt[run.bt >= 0]
        assert len(np.unique(held)) == len(held) == int((-(-seq // ps)).sum())


def test_the_list_runs_out_and_is_filled_anew(dsa):
    run = Steps(dsa, 2, width=8, F=5, T=200, PTW=16)
    assert run([64, 130], [64, 130]) == 0          # takes 1 + 3
    assert run([1, 63], [65, 193]) == NO_PAGES     # takes 2, one is left
    assert run([1, 63], [65, 193]) == NO_PAGES     # and again
    run.g_free.copy_(_i32(np.arange(50, 55)))
    run.free = np.arange(50, 55, dtype=np.int32)
    run.state.zero_()
    run.start, run.taken = 0, 0
    assert run([1, 63], [65, 193]) == 0
    assert run([64, 1], [129, 194]) == 0
    assert run.bt[:, :4].tolist()[0][1:3] == [50, 52] and run.bt[1, 3] == 51


def test_equal_lengths_as_a_new_step(dsa):
    """Two prompts of one length, one after the other, that both stay."""
    run = Steps(dsa, 1, width=4, F=8, T=100, PTW=4)
    assert run([100], [100]) == 0
    first = run.bt.copy()
    run.state[3:] = -1
    run.bt[:] = -1
    run.g_bt.fill_(-1)
    assert run([100], [100], new=True) == 0
    assert not set(first[0, :2].tolist()) & set(run.bt[0, :2].tolist())


def test_without_a_state_every_call_starts_at_the_front(dsa):
    bt = torch.full((1, 4), -1, dtype=torch.int32, device=DEV)
    free = _i32([9, 8, 7])
    for q, seq in ((64, 64), (64, 128)):
        dsa.dsa_build_page_tables(_i32([q]), _i32([seq]), bt, free, T=64, PTW=4)
    torch.cuda.synchronize()
    assert bt.cpu().tolist() == [[9, 9, -1, -1]]


def test_captured_layer_step_grows_over_many_pages(dsa):
    """A captured decode step over a 4-bit cache, replayed while one request
    enters its third, fourth and fifth page and the other its sixth: live pages
    stay distinct and the rows written before stay as they were."""
    from deepseek_sparse_attention_score_gb300.layer import LayerRunner

    wl = DI.random_small(32, [1, 1], [127, 300], H=16, k=64, spare_pages=6)
    spare = sorted(set(range(wl.rg.num_pages)) - set(wl.rg.page_indices.tolist()))
    run = LayerRunner(wl, DEV, cache_bits=4, tables=True, spare_pages=spare, max_kv=330)
    assert run.PTW == wl.rg.PTW + len(spare) and run.block_table.shape[1] == 6
    run.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run.step()
    written, pages_used = {}, 0
    for i, lens in enumerate([[127, 300], [128, 301], [129, 302], [129, 302], [192, 320], [193, 321], [256, 322],
                              [257, 330], [257, 330]]):
        run.lens[1].copy_(torch.tensor(lens, dtype=torch.int32))
        rows = torch.randn(2, 576, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16)
        run.new_kv[0].copy_(rows)
        if i % 2:
            g.replay()
        else:
            run.step()
        torch.cuda.synchronize()
        assert run.status.item() == 0
        # both requests' pages, from the block table and from the packed table
        need = [-(-n // 64) for n in lens]
        bt = run.block_table.cpu().numpy()
        live = np.concatenate([bt[s, : need[s]] for s in range(2)])
        assert (live >= 0).all() and len(set(live.tolist())) == len(live)
        assert np.array_equal(run.meta[3].cpu().numpy()[: len(live)], live)
        slots = run.tables.slots.cpu().tolist()
        assert slots == [int(bt[s, (n - 1) // 64]) * 64 + (n - 1) % 64 for s, n in enumerate(lens)]
        written.update(zip(slots, R.q4_pack(rows)))
        cache = run.kv4[0].cpu().numpy().reshape(-1, 416)
        for slot, row in written.items():
            assert np.array_equal(cache[slot], row), (i, slot)
        # attention over the selected positions of those pages
        pos = [n - 1 for n in lens]
        sel = run.topk[0].cpu().numpy()
        flat = R.q4_values(cache)
        o, _, otol, _ = R.attend(R.f64(run.q[0]), lambda t: flat[[
            int(bt[t, j // 64]) * 64 + j % 64 for j in sel[t] if 0 <= j <= pos[t]]], wl.sm_scale)
        assert (np.abs(R.f64(run.o[0]) - o) <= otol).all()
    assert run.free_state[:3].cpu().tolist() == [0, 3, 1]  # 129; 193 and 321; then 257


def test_runner_refusals(dsa):
    from deepseek_sparse_attention_score_gb300.layer import LayerRunner

    wl = DI.random_small(34, [1], [64], H=16)
    for kw in (dict(spare_pages=[1]), dict(PTW=4), dict(max_kv=100)):
        with pytest.raises(ValueError):
            LayerRunner(wl, DEV, **kw)
    for kw in (dict(PTW=0), dict(max_kv=63)):
        with pytest.raises(ValueError):
            LayerRunner(wl, DEV, tables=True, **kw)


def test_no_requests_and_the_largest_number(dsa):
    state, st = torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    out = dsa.dsa_build_page_tables(_i32([]), _i32([]), torch.zeros((0, 4), dtype=torch.int32, device=DEV), _i32([3]), T=2,
                                    PTW=2, free_state=state, dev_status=st)
    torch.cuda.synchronize()
    assert state.cpu().tolist() == [0, 0, 0] and st.item() == 0 and (out.slots == -1).all()
    S = 16384
    run = Steps(dsa, S, width=3, F=3 * S, T=S, PTW=3 * S)
    seq = np.arange(S) % 60 + 1
    assert run(np.ones(S), seq) == 0  # from an empty block table: a request's first page comes with its first tokens
    assert run(np.ones(S), seq + 1) == 0 and run(np.ones(S), seq + 1) == 0
    assert run(np.ones(S), np.full(S, 65)) == 0
    held = run.bt[run.bt >= 0]
    assert len(np.unique(held)) == len(held)


def test_a_list_that_is_not_given(dsa):
    """No free list: steps that take no page, and one that would."""
    run = Steps(dsa, 2, width=2, F=0, T=4, PTW=4)
    run.bt[:, 0] = [4, 7]
    run.g_bt.copy_(_i32(run.bt))
    run.g_free = None
    assert run([1, 1], [5, 64]) == 0 and run([1, 1], [6, 64]) == 0
    assert run([1, 1], [7, 65]) == NO_PAGES
