"""Several targets of one rotation: on 16 bytes all of them (with columns that
pass through on both sides, bf16 beside fp32, padding rows), and beside a target
that is not, which takes a launch of its own and leaves the others theirs."""
import pytest
import torch

from test_gpu_rope import _check, _x, dsa  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def _targets(m, T, seed):
    """(target, out, in, old, rot_off, layout, scale) of aligned targets."""
    bf, f4 = torch.bfloat16, torch.float32
    out = []

    def add(x, y, off, layout, scale):
        x0, old = x.clone(), (x if y is None else y).clone()
        out.append((m.RopeTarget(x, y, rot_off=off, rot_dim=64, layout=layout, scale=scale), x if y is None else y, x0,
                    old, off, layout, scale))
    add(_x((T, 5, 128), bf, seed), None, 0, "half", 1.0)                                # in place
    add(_x((T, 6, 320), bf, seed + 1)[:, ::2, 64:256], _x((T, 3, 192), bf, seed + 2), 64, "interleaved", 1.5)
    add(_x((T, 2, 136), f4, seed + 3), _x((T, 4, 136), f4, seed + 4)[:, 1:3], 32, "half", 0.75)
    add(_x((3, T, 576), bf, seed + 5).transpose(0, 1), _x((T, 3, 576), bf, seed + 6), 512, "half", 1.0)
    add(_x((T, 1, 192), f4, seed + 7), None, 128, "interleaved", 2.0)
    return out


@pytest.mark.parametrize("T", [1, 19, 700])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("odd", [False, True])
def test_several_targets(dsa, T, inverse, odd):  # noqa: F811
    pos = torch.randint(0, 131072, (T,), generator=torch.Generator().manual_seed(T), dtype=torch.int32).cuda()
    if T > 4:
        pos[4] = pos[T - 1] = -1  # padding rows stay as they are
    freqs, _ = dsa.dsa_rope_freqs(64, scaling="linear", factor=4.0, device="cuda")
    ts = _targets(dsa, T, 10 * T)
    if odd:  # in the middle: rows of 2-byte alignment
        x = _x((T, 2, 131), torch.bfloat16, 3)[:, :, 1:130]
        y = _x((T, 2, 129), torch.bfloat16, 4)
        ts.insert(2, (dsa.RopeTarget(x, y, rot_off=7, rot_dim=64), y, x.clone(), y.clone(), 7, "half", 1.0))
    n = dsa.dsa_launch_count()
    res = dsa.dsa_rope([t[0] for t in ts], pos, freqs, inverse=inverse)
    assert dsa.dsa_launch_count() - n == (2 if odd else 1)
    torch.cuda.synchronize()
    for r, (_, y, x, old, off, layout, scale) in zip(res, ts):
        assert r is y
        _check(y, x, pos, freqs, off, layout, scale, inverse, old=old)


def test_only_unaligned_targets(dsa):  # noqa: F811
    T = 33
    pos = torch.arange(T, dtype=torch.int32).cuda()
    freqs, _ = dsa.dsa_rope_freqs(6, device="cuda")
    xs = [_x((T, 2, 10), torch.bfloat16, 1), _x((T, 1, 9), torch.float32, 2)]
    old = [x.clone() for x in xs]
    n = dsa.dsa_launch_count()
    dsa.dsa_rope([dsa.RopeTarget(x, rot_off=3, rot_dim=6) for x in xs], pos, freqs)
    assert dsa.dsa_launch_count() - n == 1
    for x, o in zip(xs, old):
        _check(x, o, pos, freqs, 3, "half", 1.0, False, old=o)
