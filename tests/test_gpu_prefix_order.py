"""dsa_prefix_mla and groups that are out of order or out of range: the call is
flagged, their rows are not written, and those of the other groups are right."""
import pytest
import torch

from test_gpu_prefix_mla import Batch, dsa  # noqa: F401

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _check_rows(dsa, b, want, wl, good, left):  # noqa: F811
    """Rows of the tokens in ``good`` as in ``want``, those in ``left`` as they were."""
    H = b.H
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full((b.T, H, 512), 7.0, dtype=BF, device="cuda")
    lse = torch.full((b.T, H), 7.0, device="cuda")
    b.call(dsa, dev_status=st, o=o, lse=lse)
    torch.cuda.synchronize()
    assert st.item() == 2
    assert (o[left] == 7).all() and (lse[left] == 7).all()
    if good:
        # in other row tiles than before: equal but for rounding
        assert (o[good].float() - want[good].float()).abs().max() < 2e-2 and (lse[good] - wl[good]).abs().max() < 1e-4


@pytest.mark.parametrize("groups,good,left", [
    ([0, 3, 1], [0, 1], [4]),  # the first one has the third request too
    ([0, 2, 9], [0, 1], [2, 3, 4]),
    ([0, 2, 3], [0, 1, 2, 3], [4]),
    ([1, 2, 4], [2, 3, 4], [0, 1]),
    ([0, -1, 4], [], [0, 1, 2, 3, 4]),
])
def test_groups(dsa, groups, good, left):  # noqa: F811
    b = Batch([(100, [(1, 30), (1, 60)]), (70, [(2, 20), (1, 1)])], 16)
    want, wl = b.call(dsa)
    b.groups.copy_(torch.tensor(groups, dtype=torch.int32))
    _check_rows(dsa, b, want, wl, good, left)


# requests of 2, 3, 1 and 2, 1, 4 new tokens: offsets 0 2 5 6 8 9 13, groups of three
@pytest.mark.parametrize("at,value,first", [
    (1, 6, True), (2, 1, True), (2, 1000, True), (1, -5, True), (2, -(1 << 31), True), (1, (1 << 31) - 1, True),
    (4, 5, False), (4, 10, False), (5, 7, False), (5, 0, False), (4, 100, False), (5, -7, False), (4, 1 << 30, False),
])
def test_tokens_inside_a_group(dsa, at, value, first):  # noqa: F811
    """Offsets that go down inside a group: the group is refused, whatever lies
    between its ends, and the other one's requests are found all the same."""
    b = Batch([(100, [(2, 30), (3, 60), (1, 5)]), (70, [(2, 20), (1, 1), (4, 300)])], 16)
    want, wl = b.call(dsa)
    b.meta[1][at] = value
    here, there = list(range(6)), list(range(6, 13))
    _check_rows(dsa, b, want, wl, there if first else here, here if first else there)


@pytest.mark.parametrize("S", [40, 3500])
@pytest.mark.parametrize("many", [False, True])
def test_one_group_of_many(dsa, S, many):  # noqa: F811
    """Few requests and groups, and more of them than the plan keeps in shared memory."""
    n = 5 if not many else S // 5  # groups
    sizes = [S // n] * n
    b = Batch([(40 + i % 30, [(2, 3)] * k) for i, k in enumerate(sizes)], 4, 32)
    want, wl = b.call(dsa)
    for bad in (0, n // 2, n - 1):
        a = bad * (S // n)
        at = a + 1 + (bad % max(1, S // n - 2))  # an offset inside the group
        old = b.meta[1][at].item()
        b.meta[1][at] = old - 3
        left = list(range(2 * a, 2 * (a + S // n)))
        _check_rows(dsa, b, want, wl, [t for t in range(b.T) if not 2 * a <= t < 2 * (a + S // n)], left)
        b.meta[1][at] = old
