"""dsa_prefix_mla where a prefix ends inside a page: what a request holds from
the prefix on, the first request of a group included, reaches its own outputs
alone, and requests that end between the prefix's last page and its end see the
right keys."""
import numpy as np
import pytest
import torch

from test_gpu_prefix_mla import Batch, _check, dsa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ps", [32, 64, 128])
@pytest.mark.parametrize("prefix", [1, 10, 31, 63, 65, 130, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rows_behind_the_prefix_stay_with_their_request(dsa, ps, prefix, bad):  # noqa: F811
    b = Batch([(prefix, [(1, 4), (2, 90), (1, 1)]), (prefix + 7, [(1, 200), (1, 3)]), (0, [(1, 5), (1, 70)])], 16, ps)
    o, lse = _check(dsa, b)
    first = np.cumsum([0] + b.q_lens)
    ends = [prefix] * 3 + [prefix + 7] * 2 + [0] * 2
    for s, end in enumerate(ends):
        # the first position behind the prefix, which lies in the page of the prefix's end, and the last one
        for at in sorted({end, b.seq[s] - 1}):
            page = b.kv[b.table[s][at // ps]]
            old = page[at % ps].clone()
            page[at % ps, 3:512:7] = bad
            o2, lse2 = b.call(dsa)
            torch.cuda.synchronize()
            page[at % ps] = old
            t0, t1 = int(first[s]), int(first[s + 1])
            others = torch.ones(b.T, dtype=torch.bool, device="cuda")
            others[t0:t1] = False
            assert torch.equal(o[others], o2[others]) and torch.equal(lse[others], lse2[others]), (s, at)
            seen = [t for t in range(t0, t1) if b.seq[s] - (t1 - t) >= at]  # tokens from that position on
            assert seen and not o2[seen].isfinite().all(-1).any(), (s, at)


@pytest.mark.parametrize("ps", [32, 64, 128])
@pytest.mark.parametrize("H", [5, 16, 128])
@pytest.mark.parametrize("groups", [
    [(100, [(1, 4), (1, -20), (5, -30), (20, 3), (1, -99)])],     # requests that end before the prefix does
    [(127, [(1, 1), (3, -1), (2, 0), (1, -62), (40, -63)])],
    [(193, [(1, 9)] + [(1, -k) for k in range(0, 60, 4)]), (31, [(1, 1), (1, 0), (2, -3)])],
], ids=str)
def test_requests_that_end_in_the_prefix_s_last_page(dsa, groups, H, ps):  # noqa: F811
    _check(dsa, Batch(groups, H, ps))
