"""dsa_build_page_tables against a plain loop over requests, tokens and pages
(integers: equal), its in-place growth, padding, device conditions and use in
a captured graph."""
import numpy as np
import pytest
import torch

import steps_ref as R

pytestmark = pytest.mark.gpu
BAD_METADATA, NO_PAGES = 0x2, 0x20


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


def _inputs(q, seq, ps, seed=0, spare=5, width=None, stride=None):
    rng = np.random.default_rng(seed)
    q, seq = np.asarray(q, np.int32), np.asarray(seq, np.int32)
    had, need = -(-(seq - q) // ps), -(-seq // ps)
    W = int(max(1, need.max(initial=0))) if width is None else width
    ids = rng.permutation(int(np.clip(need, 0, None).sum()) + spare).astype(np.int32)
    bt = np.full((len(q), stride or W), -7, np.int32)
    k = 0
    for s in range(len(q)):
        n = int(np.clip(had[s], 0, W))
        bt[s, :n] = ids[k: k + n]
        k += n
    return q, seq, bt, ids[k:], W


def _run(dsa, q, seq, bt, free, W, ps, T, PTW):
    dev = torch.device("cuda")
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    table, st = to(bt), torch.zeros(1, dtype=torch.int32, device=dev)
    out = dsa.dsa_build_page_tables(to(q), to(seq), table[:, :W], to(free), T=T, PTW=PTW, ps=ps, dev_status=st)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out._asdict().items()}, table.cpu().numpy(), st.item()


def _check(dsa, q, seq, bt, free, W, ps, T, PTW):
    got, table, st = _run(dsa, q, seq, bt, free, W, ps, T, PTW)
    ref, rbt, rst = R.page_tables(q, seq, bt[:, :W], free, T, PTW, ps)
    for k, v in ref.items():
        assert np.array_equal(got[k], v), (k, np.argwhere(got[k] != v)[:5].tolist())
    assert np.array_equal(table[:, :W], rbt) and np.array_equal(table[:, W:], bt[:, W:])
    assert st == rst
    return got


@pytest.mark.parametrize("ps", [32, 64, 128])
@pytest.mark.parametrize("q,seq", [
    ([1], [1]),
    ([1, 1, 1], [700, 64, 65]),                    # the first takes no page, the last its second
    ([300], [300]),                                # everything new
    ([0, 5, 0, 0, 129, 1, 0], [0, 5, 77, 0, 129, 1025, 64]),  # empty and pausing requests
    ([4096, 1, 33], [9000, 128, 33]),
])
def test_matches_plain_loop(dsa, ps, q, seq):
    q, seq, bt, free, W = _inputs(q, seq, ps)
    need = int((-(-seq // ps)).sum())
    _check(dsa, q, seq, bt, free, W, ps, int(q.sum()), need)        # exact sizes
    _check(dsa, q, seq, bt, free, W, ps, int(q.sum()) + 9, need + 6)  # padded sizes


@pytest.mark.parametrize("S", [2, 31, 513, 2047, 4100])
def test_many_requests(dsa, S):
    rng = np.random.default_rng(S)
    q = rng.integers(0, 4, S)
    seq = q + rng.integers(0, 600, S) * (rng.random(S) < 0.8)
    q, seq, bt, free, W = _inputs(q, seq, 64, seed=S, stride=23)
    _check(dsa, q, seq, bt, free, min(W, 23), 64, int(q.sum()) + 3, int((-(-seq // 64)).sum()) + 1)


def test_largest_number_of_requests(dsa):
    S = 16384
    q, seq, bt, free, W = _inputs(np.ones(S), np.arange(S) % 200 + 1, 64)
    _check(dsa, q, seq, bt, free, W, 64, S, int((-(-seq // 64)).sum()))


def test_no_requests(dsa):
    got, _, st = _run(dsa, np.zeros(0, np.int32), np.zeros(0, np.int32), np.zeros((0, 4), np.int32),
                      np.zeros(3, np.int32), 4, 64, 5, 7)
    assert st == 0 and got["cu_q_lens"].tolist() == [0] and got["n_taken"].tolist() == [0]
    assert (got["slots"] == -1).all() and (got["page_indices"] == -1).all()


def test_running_out_of_pages(dsa):
    q, seq, bt, free, W = _inputs([100, 200, 1], [100, 500, 129], 64)
    got = _check(dsa, q, seq, bt, free[:4], W, 64, 301, 14)  # takes 2 + 3 + 1, has 4
    assert got["n_taken"].tolist() == [6] and (got["slots"] == -1).any()
    _, _, st = _run(dsa, q, seq, bt, free[:4], W, 64, 301, 14)
    assert st == NO_PAGES


@pytest.mark.parametrize("T,PTW", [(300, 14), (301, 12), (0, 14), (301, 0)])
def test_sizes_too_small(dsa, T, PTW):
    q, seq, bt, free, W = _inputs([100, 200, 1], [100, 500, 129], 64)
    _check(dsa, q, seq, bt, free, W, 64, T, PTW)
    assert _run(dsa, q, seq, bt, free, W, 64, T, PTW)[2] & BAD_METADATA


def test_impossible_lengths_count_as_empty(dsa):
    q = np.array([1, -3, 5, 1, 2, 1], np.int32)
    seq = np.array([70, 10, 4, 2**31 - 1, -2, 130], np.int32)  # negative q, q > seq, past the table, negative seq
    bt = np.arange(24, dtype=np.int32).reshape(6, 4)
    _check(dsa, q, seq, bt, np.arange(50, 60, dtype=np.int32), 4, 64, 9, 9)


def test_same_values_again_and_captured(dsa):
    dev = torch.device("cuda")
    q, seq, bt, free, W = _inputs([3, 1, 64], [67, 900, 64], 64)
    to = lambda a: torch.from_numpy(a).to(dev)
    tq, tseq, tbt, tfree = to(q), to(seq), to(bt), to(free)
    first = dsa.dsa_build_page_tables(tq, tseq, tbt, tfree, T=70, PTW=20)
    torch.cuda.synchronize()
    ref = [x.clone() for x in first]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_build_page_tables(tq, tseq, tbt, tfree, T=70, PTW=20, out=first)
    for x in first:
        x.fill_(99)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, ref))
    # one token more: the captured step follows the lengths
    tq.copy_(to(np.array([4, 1, 1], np.int32)))
    tseq.copy_(to(np.array([71, 901, 65], np.int32)))
    g.replay()
    torch.cuda.synchronize()
    want, _, _ = R.page_tables(tq.cpu().numpy(), tseq.cpu().numpy(), tbt.cpu().numpy(), free, 70, 20, 64)
    assert all(np.array_equal(getattr(first, k).cpu().numpy(), v) for k, v in want.items())
