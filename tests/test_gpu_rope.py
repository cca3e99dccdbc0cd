"""dsa_rope against 64-bit rotation: layouts, types, parts of the head, far
positions, strides and alignments, in place, padding rows, and its inverse as
the gradient (by the inner product and by differences)."""
import numpy as np
import pytest
import torch

import steps_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


def _x(shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def _check(y, x, positions, freqs, off, layout, scale, inverse, old=None):
    ref, mag = R.rope(R.f64(x), positions.cpu().numpy(), freqs.cpu().numpy(), off, layout, scale, inverse)
    pad = (positions < 0).cpu().numpy()
    if old is not None:
        ref[pad] = R.f64(old)[pad]
    e = np.abs(R.f64(y) - ref) - R.rope_tol(ref, mag, x.dtype)
    assert (e <= 0).all(), (np.argwhere(e > 0)[:4].tolist(), e.max())
    same = mag == 0
    assert np.array_equal(R.f64(y)[same], ref[same])  # columns that pass through, bit for bit


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H,D,off,rot", [
    (1, 1, 64, 0, 64), (3, 128, 64, 0, 64), (37, 5, 128, 0, 64), (5, 2, 576, 512, 64), (2, 3, 192, 64, 64),
    (4, 2, 10, 3, 6),     # nothing on 16 bytes
    (2, 1, 2, 0, 2), (700, 1, 576, 512, 64), (3, 2, 512, 0, 512),
])
def test_matches_64_bit(dsa, dtype, layout, T, H, D, off, rot):
    x = _x((T, H, D), dtype, T + D)
    pos = torch.randint(0, 131072, (T,), generator=torch.Generator().manual_seed(T), dtype=torch.int32).cuda()
    freqs, scale = dsa.dsa_rope_freqs(rot, scaling="yarn", factor=40.0, device="cuda")
    for inverse in (False, True):
        y = torch.empty_like(x)
        out = dsa.dsa_rope(dsa.RopeTarget(x, y, rot_off=off, rot_dim=rot, layout=layout, scale=scale), pos, freqs,
                           inverse=inverse)
        torch.cuda.synchronize()
        assert out is y
        _check(y, x, pos, freqs, off, layout, scale, inverse)
        z = x.clone()  # in place: the same values
        dsa.dsa_rope(dsa.RopeTarget(z, rot_off=off, rot_dim=rot, layout=layout, scale=scale), pos, freqs,
                     inverse=inverse)
        assert torch.equal(z, y)


def test_far_positions(dsa):
    """Angles up to 2^31 turns of the fastest pair keep fp32 accuracy."""
    pos = torch.tensor([0, 1, 2**20 + 1, 2**24 + 3, 2**30 + 7, 2**31 - 1], dtype=torch.int32).cuda()
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    x = _x((6, 2, 64), torch.float32)
    y = dsa.dsa_rope(dsa.RopeTarget(x, torch.empty_like(x)), pos, freqs)
    _check(y, x, pos, freqs, 0, "half", 1.0, False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_views_and_several_targets(dsa, dtype):
    T, H = 19, 6
    pos = torch.arange(100, 100 + T, dtype=torch.int32).cuda()
    pos[4] = pos[18] = -1  # padding rows stay as they are
    freqs, scale = dsa.dsa_rope_freqs(64, scaling="linear", factor=4.0, device="cuda")
    proj, q = _x((T, H, 192), dtype, 1), _x((T, H, 576), dtype, 2)
    k = _x((T, 1, 576), dtype, 3)
    qi = _x((H, T, 128), dtype, 4).transpose(0, 1)  # tokens are not the outer dimension
    odd = _x((T, 2, 131), dtype, 5)[:, :, 1:130]    # odd strides, unaligned
    q0, k0, odd0 = q.clone(), k.clone(), odd.clone()
    qi_out, odd_out = _x((T, H, 128), dtype, 6), _x((T, 2, 129), dtype, 7)
    qi_old, odd_old = qi_out.clone(), odd_out.clone()
    R4 = dsa.RopeTarget
    dsa.dsa_rope([R4(proj[:, :, 128:], q[:, :, 512:], layout="interleaved", scale=1.5),
                  R4(k, rot_off=512, layout="interleaved"), R4(qi, qi_out, rot_dim=64),
                  R4(odd, odd_out, rot_off=7, rot_dim=64)], pos, freqs)
    torch.cuda.synchronize()
    assert torch.equal(q[:, :, :512], q0[:, :, :512])
    _check(q[:, :, 512:], proj[:, :, 128:], pos, freqs, 0, "interleaved", 1.5, False, old=q0[:, :, 512:])
    _check(k, k0, pos, freqs, 512, "interleaved", 1.0, False, old=k0)
    _check(qi_out, qi, pos, freqs, 0, "half", 1.0, False, old=qi_old)
    _check(odd_out, odd0, pos, freqs, 7, "half", 1.0, False, old=odd_old)


def test_no_rows_and_no_heads(dsa):
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    dsa.dsa_rope(dsa.RopeTarget(torch.empty(0, 4, 64, device="cuda")), none, freqs)
    pos = torch.ones(3, dtype=torch.int32, device="cuda")
    x = _x((3, 1, 64), torch.float32)
    y = torch.empty_like(x)
    dsa.dsa_rope([dsa.RopeTarget(torch.empty(3, 0, 64, device="cuda")), dsa.RopeTarget(x, y)], pos, freqs)
    _check(y, x, pos, freqs, 0, "half", 1.0, False)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_inverse_is_the_gradient(dsa, layout):
    T, H, D, off, scale = 9, 3, 96, 16, 1.25
    pos = torch.randint(0, 50000, (T,), dtype=torch.int32).cuda()
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    x, g = _x((T, H, D), torch.float32, 1), _x((T, H, D), torch.float32, 2)
    t = lambda a, inv: dsa.dsa_rope(dsa.RopeTarget(a, torch.empty_like(a), rot_off=off, rot_dim=64, layout=layout,
                                                   scale=scale), pos, freqs, inverse=inv)
    dx = t(g, True)
    # the formula: the transpose of the turn, in 64 bits
    _check(dx, g, pos, freqs, off, layout, scale, True)
    # differences of f(x) = <rope(x), g>, which is linear: exact but for
    # rounding, 2^-20 of the magnitudes in f at both ends
    f = lambda a: float((t(a, False).double() * g.double()).sum())
    for c in [(0, 0, 0), (3, 1, off), (5, 2, off + 63), (8, 0, off + 31), (2, 2, 95)]:
        e = torch.zeros_like(x)
        e[c] = 64.0
        diff = (f(x + e) - f(x - e)) / 128.0
        row = lambda a: float(a[c[0], c[1]].abs().sum())
        tol = 2.0 ** -20 * (row(x) + 64.0) * row(g) * scale * 2 / 64.0 + 2.0 ** -22 * row(x) * row(g) * scale
        assert abs(diff - float(dx[c])) <= tol, (c, diff, float(dx[c]), tol)


def test_frequencies(dsa):
    f, m = dsa.dsa_rope_freqs(64)
    want = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    assert m == 1.0 and np.allclose(f.numpy(), want, rtol=1e-15, atol=0)


def test_offsets_past_32_bits(dsa):
    """Rows 2^31 + 64 elements apart in both tensors."""
    buf = torch.zeros(2**31 + 256, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((2, 1, 64), (2**31 + 64, 64, 1))
    far.copy_(_x((2, 1, 64), torch.bfloat16, 3))
    x = far.clone()
    pos = torch.tensor([77, 1234], dtype=torch.int32, device="cuda")
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    dsa.dsa_rope(dsa.RopeTarget(far), pos, freqs)
    _check(far, x, pos, freqs, 0, "half", 1.0, False)


def test_two_streams_at_once(dsa):
    """Calls on two streams share nothing."""
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    pos = torch.arange(500, dtype=torch.int32, device="cuda")
    xs = [_x((500, 8, 64), torch.bfloat16, k) for k in range(2)]
    ys = [torch.empty_like(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, x, y in zip(streams, xs, ys):
            with torch.cuda.stream(s):
                dsa.dsa_rope(dsa.RopeTarget(x, y), pos, freqs)
    torch.cuda.synchronize()
    for x, y in zip(xs, ys):
        _check(y, x, pos, freqs, 0, "half", 1.0, False)
