"""dsa_rope_append's angles, where nothing else hides them: a pair (0, b) becomes
(-b sin, b cos), so that a small angle's own precision shows in the cache."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


# A turn fraction per position in 64 bits is off by 2^-65 at most, which for f radians per position is pi 2^-64 / f of
# it (2^-32 at f = 1e-9); the product's conversion to fp32 by 2^-24, the sine by 2^-22 (two units), the scaled sine and
# the product by 2^-24 each: below 2^-20 in all. The rounding to bf16 is 2^-8.
TOL = (1 + 2.0 ** -8) * (1 + 2.0 ** -20) - 1


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("queries", [False, True])  # rows by themselves, and in a launch with queries
@pytest.mark.parametrize("sign", [1, -1])
def test_small_angles(dsa, layout, queries, sign):
    R, T = 32, 48
    f = sign * np.logspace(-9, -3, R // 2)
    pos = np.concatenate([np.arange(1, 33), np.arange(1, 17) * 37])
    b = torch.linspace(1.0, 2.0, T * R // 2).to(BF).view(T, R // 2)
    x = torch.zeros(T, R, dtype=BF)
    ca, cb = (slice(0, R, 2), slice(1, R, 2)) if layout == "interleaved" else (slice(0, R // 2), slice(R // 2, R))
    x[:, cb] = b
    x, cache = x.cuda(), torch.zeros(2, 32, R, dtype=BF, device="cuda")
    i32 = lambda a: torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    freqs = torch.tensor(f, dtype=torch.float64, device="cuda")
    q = torch.zeros(T, 1, R, dtype=BF, device="cuda")
    dsa.dsa_rope_append(dsa.AppendTarget(x, cache, layout=layout), i32(pos), i32(np.arange(T)), freqs,
                        rotate=[dsa.RopeTarget(q)] if queries else [])
    got = cache.view(-1, R)[:T].double().cpu().numpy()
    want = -b.double().numpy() * np.sin(pos[:, None] * f)
    e = np.abs(got[:, ca] - want) / np.abs(want)
    assert (e <= TOL).all(), (e.max(), np.argwhere(e > TOL)[:4].tolist())


def test_angles_are_those_of_dsa_rope(dsa):
    """The largest step between the two ways is one of the result's rounding, at angles of all sizes."""
    R, T = 64, 4096
    freqs = torch.tensor(np.logspace(-9, 0, R // 2), dtype=torch.float64, device="cuda")
    rng = np.random.default_rng(1)
    pos = torch.from_numpy(np.exp(rng.uniform(0, np.log(2.0 ** 30), T)).astype(np.int32)).cuda()
    x = torch.zeros(T, R, dtype=BF, device="cuda")
    x[:, 1::2] = 1
    cache = torch.zeros(T // 32, 32, R, dtype=BF, device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    dsa.dsa_rope_append(dsa.AppendTarget(x, cache, layout="interleaved"), pos, slots, freqs)
    y = x[:, None].clone()
    dsa.dsa_rope(dsa.RopeTarget(y, layout="interleaved"), pos, freqs)
    got, want = cache.view(T, R).double(), y[:, 0].double()
    # Apart by: the fp64 product of dsa_rope, 2^-53 of 2^30 / 2 pi turns, or 1.2e-7 radians; fractions in fp32, 2^-26 of
    # a turn each, or 2e-7 radians; sines, 2^-23 each. Together 6e-7 < 2^-20. A step of bf16 is 2^-7.
    assert ((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -20).all()
    small = (pos.double()[:, None] * freqs) < 1.0  # there both angles keep fp32's relative precision
    d, w = (got - want).abs()[:, 0::2][small], want.abs()[:, 0::2][small]
    assert (d <= 2.0 ** -7 * w).all()
