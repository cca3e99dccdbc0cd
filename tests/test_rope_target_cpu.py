"""A kept RopeTarget follows its tensors: what a call hands to the library is
their address, shape and strides at that call, not at the target's making."""
import struct

import pytest
import torch

FIELDS = struct.Struct("=QQqqqqiiiiif")


@pytest.fixture
def calls(monkeypatch):
    import __graft_entry__

    __graft_entry__.build()
    from deepseek_sparse_attention_score_gb300 import abi

    got = []
    monkeypatch.setattr(abi, "_launch", lambda dev, name, c, n, *a: got.append(
        [FIELDS.unpack(c[i * FIELDS.size: (i + 1) * FIELDS.size]) for i in range(n)]))
    return abi, got


def _expect(x, y, off):
    xs, ys = x.stride(), y.stride()
    return (x.data_ptr(), y.data_ptr(), xs[0], xs[1], ys[0], ys[1], x.shape[1], x.shape[2], off)


def _resize(t):
    t.resize_(4, 64, 96)


def _set(t):
    t.set_(torch.zeros(4, 4, 200)[:, ::2, 40:136])


def _data(t):
    t.data = torch.zeros(2, 4, 96).transpose(0, 1)


def _same_address(t):
    t.as_strided_((4, 2, 96), (96, 384, 1))


@pytest.mark.parametrize("change", [_resize, _set, _data, _same_address])
@pytest.mark.parametrize("which", ["x", "y", "both", "in place"])
def test_a_kept_target_follows_its_tensors(calls, change, which):
    abi, got = calls
    x = torch.zeros(4, 2, 96)
    y = x if which == "in place" else torch.zeros(4, 2, 96)
    pos, freqs = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    g, other = abi.RopeTarget(x, y, rot_off=8, rot_dim=64), abi.RopeTarget(torch.zeros(4, 1, 64))
    abi.dsa_rope([other, g], pos, freqs)
    assert got[-1][1][:9] == _expect(x, y, 8)
    for t in {"x": [x], "y": [y], "both": [x, y], "in place": [x]}[which]:
        change(t)
    if x.shape == y.shape:
        assert abi.dsa_rope([other, g], pos, freqs)[1] is y
        assert got[-1][1][:9] == _expect(x, y, 8)
        assert got[-1][0][:9] == _expect(other.x, other.y, 0)
    else:
        with pytest.raises(ValueError):
            abi.dsa_rope([other, g], pos, freqs)
        assert len(got) == 1


def test_a_target_that_no_longer_fits_is_refused(calls):
    abi, got = calls
    pos, freqs = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    x = torch.zeros(4, 2, 64)
    g = abi.RopeTarget(x)
    for change, error in ((lambda: x.resize_(5, 2, 64), ValueError), (lambda: x.resize_(4, 2, 96), ValueError),
                          (lambda: x.resize_(4, 128), TypeError), (lambda: x.resize_(4, 64, 4).transpose_(1, 2), ValueError)):
        change()
        with pytest.raises(error):
            abi.dsa_rope(g, pos, freqs)
    assert not got
    x.resize_(4, 2, 64)
    abi.dsa_rope(g, pos, freqs)
    assert got[-1][0][:9] == _expect(x, x, 0)
