"""dsa_rope_append refuses calls in which one part writes what another reads or
writes: their threads would race. No call here reaches a kernel; what may share
rows is in test_gpu_append_overlap.py."""
import ctypes
import os
import random
import subprocess

import pytest

from test_rope_append_cpu import ROTATE, _call, lib  # noqa: F401

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deepseek_sparse_attention_score_gb300",
                    "csrc")
INVALID = -1
CACHE = 2 * 64 * 576 * 2  # bytes of the calls' caches
FAR = 1 << 24
SPLIT = dict(x_rot=FAR, x_stride=512, x_rot_stride=64)
TURN = dict(x=4 * FAR, y=4 * FAR, xt=576, xh=576, yt=576, yh=576, H=1, D=576, off=512, layout=0, dtype=0, scale=1.0)


def _turn(**kw):
    t = {**TURN, **kw}
    return dict(rotate=ROTATE.pack(*t.values()), n_rotate=1)


@pytest.mark.parametrize("targets", [
    # the second cache starts inside the first, with the same rows and with others
    (dict(x=FAR, cache=8192), dict(x=FAR, cache=8192 + 5 * 1152)),
    (dict(x=FAR, cache=8192), dict(x=FAR, cache=8192 + CACHE - 16)),
    (dict(x=FAR, cache=8192 + 1040), dict(x=FAR, cache=8192)),
    (dict(x=FAR, cache=8192), dict(x=FAR, cache=8192 + 160, D=128, rot_off=0, cache_stride=128)),
    (dict(x=FAR, cache=8192), dict(x=FAR, cache=8192 + 160, format=1)),
    (dict(x=FAR, cache=8192, format=1), dict(x=FAR, cache=8192 + 2 * 64 * 416 - 16, format=1)),
    (dict(x=FAR, cache=8192, D=128, rot_off=0, cache_stride=640),
     dict(x=FAR, cache=8192 + 1280 + 128, D=128, rot_off=0, cache_stride=640)),
    # rows that lie in a cache, their own or another's
    (dict(x=8192),), (dict(x=8192 + CACHE - 16),), (dict(x=8192 - 3 * 1152 + 16),),
    (dict(x=FAR, x_stride=FAR // 2, cache=3 * FAR + 16),),
    (dict(x=8192 + 1152, x_stride=640),),
    (dict(x=FAR), dict(x=8192 + 4608, cache=1 << 20)),
    (dict(x=FAR, **{**SPLIT, "x_rot": 8192 + 16}),),
    (dict(**{**SPLIT, "x": 8192 + 512}),),
    (dict(x=8192 + 416 * 5, format=1),),
], ids=str)
def test_targets_that_meet(lib, targets):  # noqa: F811
    assert _call(lib, targets=targets) == INVALID


@pytest.mark.parametrize("target,turn", [
    # rows that turn in place while they are appended, as a whole and in two parts
    (dict(x=FAR), dict(x=FAR, y=FAR)),
    (dict(x=2 * FAR, **SPLIT), dict(x=FAR, y=FAR, xt=64, xh=64, yt=64, yh=64, D=64, off=0)),
    # outputs on top of rows
    (dict(x=FAR), dict(y=FAR + 2 * 1152)),
    (dict(x=FAR), dict(y=FAR - 3 * 1152 + 16)),
    (dict(x=FAR, x_stride=584), dict(y=FAR + 16)),
    (dict(x=2 * FAR, **SPLIT), dict(y=2 * FAR + 512)),
    (dict(x=FAR, x_stride=4096), dict(y=FAR + 8192 + 1000, yt=4096)),       # the first columns of one row
    (dict(x=FAR, x_stride=4096), dict(y=FAR - 1024, yt=4096, yh=192, H=3, D=192, off=0)),  # a head's of each
    (dict(x=FAR, x_stride=4096), dict(y=FAR + 2 * 8192 + 1024, yt=192, yh=4096, xt=192, xh=4096, H=100, D=192, off=0)),
    # rows that turn backwards
    (dict(x=FAR), dict(y=FAR + 2 * 1152, x=4 * FAR, yt=-576)),
    # outputs in the cache, and what turns read from there
    (dict(x=FAR), dict(y=8192 + 1152)),
    (dict(x=FAR), dict(y=8192 + CACHE - 32)),
    (dict(x=FAR), dict(x=8192 + 1152)),
    (dict(x=FAR), dict(x=8192 + 64, y=8192 + 64)),
], ids=str)
def test_rotations_that_meet(lib, target, turn):  # noqa: F811
    assert _call(lib, targets=(target,), **_turn(**turn)) == INVALID


def test_rows_meet_as_sets_of_bytes_do(tmp_path):
    """The answer for rows of any counts and steps against sets of bytes."""
    so = tmp_path / "rows.so"
    src = tmp_path / "rows.cpp"
    src.write_text('#include "rows.h"\nextern "C" int meet(const long long* v) {\n'
                   "  return dsa::rows_meet({v[0], v[1], v[2], v[3]}, {v[4], v[5], v[6], v[7]}, v[8], v[9]);\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", CSRC, str(src), "-o", str(so)], check=True)
    meet = ctypes.CDLL(str(so)).meet
    rng = random.Random(5)
    for k in range(30000):
        a, b = ([rng.randrange(0, 60), rng.randrange(0, 6), rng.randrange(-12, 13), rng.randrange(0, 9)] for _ in "ab")
        if rng.random() < 0.4:
            b[2] = a[2]
        m, gap = (rng.randrange(0, 8), rng.randrange(-20, 21)) if k % 2 else (1, 0)
        x = {a[0] + i * a[2] + c for i in range(a[1]) for c in range(a[3])}
        y = {b[0] + h * gap + i * b[2] + c for h in range(m) for i in range(b[1]) for c in range(b[3])}
        assert bool(meet((ctypes.c_longlong * 10)(*a, *b, m, gap))) == bool(x & y), (a, b, m, gap)
    # steps and counts whose product passes 64 bits, and long walks that need not be taken
    far, long = 1 << 62, (1 << 31) - 1
    for v, want in (((0, long, far, 16, 8, 4, 576, 16, 1, 0), True), ((0, long, far, 16, 16, 4, 576, 16, 1, 0), False),
                    ((0, long, 1152, 1152, long * 1152 - 1, 3, -far, 2, 1, 0), True),
                    ((0, long, 1280, 1152, 1152, long, 1280, 128, 1, 0), False),
                    ((0, 3, 1152, 1152, 1 << 50, long, 1024, 512, 65536, 1024), False)):
        assert bool(meet((ctypes.c_longlong * 10)(*v))) == want, v
