"""dsa_rope_append's refusals, by the entry point and by the wrapper: no call
here reaches a kernel."""
import ctypes
import struct

import pytest
import torch

INVALID, UNSUPPORTED, ALIGNMENT = -1, -2, -7
TARGET = struct.Struct("=QQQqqqiiiif4x")
ROTATE = struct.Struct("=QQqqqqiiiiif")
OK = dict(x=4096, x_rot=0, cache=8192, x_stride=576, x_rot_stride=0, cache_stride=576, D=576, rot_off=512, layout=0,
          format=0, scale=1.0)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    from deepseek_sparse_attention_score_gb300 import abi

    return abi.lib()


def _call(lib, targets=({},), n=None, rotate=None, n_rotate=0, T=3, rot=64, pos=16, slots=16, freqs=16, P=2, ps=64,
          given=True):
    packed = b"".join(TARGET.pack(*{**OK, **t}.values()) for t in targets)
    p = lambda a: ctypes.c_void_p(a) if a else None
    return lib.dsa_rope_append(None, packed if given else None, len(targets) if n is None else n, rotate, n_rotate, T,
                               rot, p(pos), p(slots), p(freqs), P, ps, None)


def test_struct_size():
    assert TARGET.size == 72


@pytest.mark.parametrize("bad,rc", [
    (dict(given=False), INVALID), (dict(n=0), INVALID), (dict(n=-1), INVALID), (dict(T=-1), INVALID),
    (dict(targets=({},) * 5), UNSUPPORTED), (dict(n_rotate=1), INVALID), (dict(n_rotate=-1), INVALID),
    (dict(P=-1), INVALID), (dict(ps=48), UNSUPPORTED), (dict(P=1 << 25, ps=64), UNSUPPORTED),
    (dict(rot=0), INVALID), (dict(rot=63), INVALID), (dict(rot=24), UNSUPPORTED), (dict(rot=528), UNSUPPORTED),
    (dict(pos=0), INVALID), (dict(slots=0), INVALID), (dict(freqs=0), INVALID),
])
def test_refused_calls(lib, bad, rc):
    assert _call(lib, **bad) == rc


@pytest.mark.parametrize("bad,rc", [
    (dict(rot_off=-8), INVALID), (dict(rot_off=520), INVALID), (dict(D=48, rot_off=0), INVALID),
    (dict(layout=2), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(format=2), UNSUPPORTED), (dict(format=1, D=640, x_stride=640), UNSUPPORTED),
    (dict(format=1, rot_off=0), UNSUPPORTED), (dict(D=580, x_stride=584, cache_stride=584), UNSUPPORTED),
    (dict(rot_off=508), UNSUPPORTED), (dict(D=4104, x_stride=4104, cache_stride=4104), UNSUPPORTED),
    (dict(x=0), INVALID), (dict(cache=0), INVALID), (dict(x_stride=568), INVALID), (dict(x_stride=580), UNSUPPORTED),
    (dict(cache_stride=568), INVALID), (dict(cache_stride=580), UNSUPPORTED), (dict(x=4098), ALIGNMENT),
    (dict(cache=8200), ALIGNMENT), (dict(x_rot=4100, x_rot_stride=64), ALIGNMENT),
    (dict(x_rot=4096, x_rot_stride=56), INVALID), (dict(x_rot=4096, x_rot_stride=68), UNSUPPORTED),
])
def test_refused_targets(lib, bad, rc):
    assert _call(lib, targets=(bad,)) == rc
    assert _call(lib, targets=(dict(cache=16384), bad)) == rc


def test_refused_pairs_and_rotations(lib):
    assert _call(lib, targets=({}, {})) == INVALID  # two targets for one cache
    r = dict(x=4096, y=4096, xt=192, xh=64, yt=192, yh=64, H=3, D=64, off=0, layout=0, dtype=0, scale=1.0)
    for bad, rc in ((dict(off=1), INVALID), (dict(x=0), INVALID), (dict(layout=5), INVALID), (dict(dtype=2), UNSUPPORTED),
                    (dict(H=-1), INVALID), (dict(x=4097, y=8192), ALIGNMENT), (dict(y=8193), ALIGNMENT),
                    (dict(yt=64, x=4096, y=8192), INVALID)):
        assert _call(lib, rotate=ROTATE.pack(*{**r, **bad}.values()), n_rotate=1) == rc, bad
    assert _call(lib, rotate=ROTATE.pack(*r.values()) * 9, n_rotate=9) == UNSUPPORTED


def test_no_tokens(lib):
    assert _call(lib, T=0, pos=0, slots=0, freqs=0, targets=(dict(x=0, cache=0),)) == 0


def test_wrapper_refusals():
    import deepseek_sparse_attention_score_gb300 as dsa

    A = dsa.AppendTarget
    x, cache = torch.zeros(3, 128, dtype=torch.bfloat16), torch.zeros(2, 32, 128, dtype=torch.bfloat16)
    i32, f = torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    g = A(x, cache, rot_dim=64)
    for make, err in ((lambda: A(x.float(), cache), TypeError), (lambda: A(x[0], cache), TypeError),
                      (lambda: A(x, cache.float()), TypeError), (lambda: A(x, cache[0]), TypeError),
                      (lambda: A(x, cache[:, :, :64]), ValueError), (lambda: A(x.t(), cache), ValueError),
                      (lambda: A(x, cache, layout="quarter"), ValueError),
                      (lambda: A(x, cache, x_rot=x[:2]), ValueError),
                      (lambda: A(x[:, :64], cache, x_rot=x[:, 64:], rot_dim=32), ValueError),
                      (lambda: A(x, cache, x_rot=x), ValueError),  # 256 columns into rows of 128
                      (lambda: A(x, torch.zeros(2, 32, 400, dtype=torch.uint8)), ValueError),
                      (lambda: dsa.dsa_rope_append(g, i32, i32[:2], f), ValueError),
                      (lambda: dsa.dsa_rope_append(g, i32, i32.long(), f), TypeError),
                      (lambda: dsa.dsa_rope_append(g, i32, i32, f.float()), TypeError),
                      (lambda: dsa.dsa_rope_append(g, i32, i32, f[:16]), ValueError),
                      (lambda: dsa.dsa_rope_append([], i32, i32, f), ValueError),
                      (lambda: dsa.dsa_rope_append(g, i32[:2], i32[:2], f), ValueError),
                      (lambda: dsa.dsa_rope_append([g, A(x, cache[:1], rot_dim=64)], i32, i32, f), ValueError),
                      (lambda: dsa.dsa_rope_append(g, i32, i32, f, rotate=dsa.RopeTarget(x[:, None], rot_dim=32)),
                       ValueError),
                      (lambda: dsa.dsa_rope_append(g, i32, i32, f), ValueError)):  # not on a GPU
        with pytest.raises(err):
            make()


def test_a_kept_target_follows_its_tensors(monkeypatch):
    from deepseek_sparse_attention_score_gb300 import abi

    got = []
    monkeypatch.setattr(abi, "_launch", lambda dev, name, c, n, *a: got.append(TARGET.unpack(c[: TARGET.size])))
    x, cache = torch.zeros(3, 128, dtype=torch.bfloat16), torch.zeros(2, 32, 128, dtype=torch.bfloat16)
    i32, f = torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    g = abi.AppendTarget(x, cache, rot_dim=64)
    for change in (lambda: None, lambda: x.set_(torch.zeros(3, 256, dtype=torch.bfloat16)[:, 64:192]),
                   lambda: cache.set_(torch.zeros(5, 64, 136, dtype=torch.bfloat16))):
        change()
        abi.dsa_rope_append(g, i32, i32, f)
        assert got[-1][:8] == (x.data_ptr(), 0, cache.data_ptr(), x.stride(0), 0, cache.shape[2], 128, 0)
