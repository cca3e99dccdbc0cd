"""Tensors of one dsa_rope_append call that lie between one another's rows, as
the columns of a fused projection do, without sharing a byte: the call is taken
and gives what tensors of their own give."""
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


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32)).cuda()


@pytest.mark.parametrize("T", [1, 2, 77, 3001])
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("turn", ["heads in place", "whole rows in place", "other columns", "heads apart"])
def test_fused_rows(dsa, T, split, turn):
    """[T, 3 heads of 192 | 192 free | latent row 576 | 8 free], the heads' last 64 columns and the row's turn."""
    gen = torch.Generator().manual_seed(T)
    fused = torch.randn(T, 1352, generator=gen).to(BF).cuda()
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    P, ps = -(-T // 32) + 1, 32
    pos, slots = _i32(np.arange(T) * 3 + 1), _i32(np.random.default_rng(T).permutation(P * ps)[:T])

    def call(rows, src, out):
        """rows: what is appended; src: where the heads lie; out: where they go."""
        cache = torch.zeros(P, ps, 576, dtype=BF, device="cuda")
        kv = rows[:, 768:1344]
        if split:
            g = dsa.AppendTarget(kv[:, :512], cache, x_rot=kv[:, 512:], rot_off=512)
        else:
            g = dsa.AppendTarget(kv, cache, rot_off=512)
        if turn == "heads in place":
            r = dsa.RopeTarget(src[:, :576].view(T, 3, 192), rot_off=128)
        elif turn == "whole rows in place":  # of which only the first head's columns are touched
            r = dsa.RopeTarget(src[:, None], rot_off=128, rot_dim=64)
        elif turn == "other columns":
            r = dsa.RopeTarget(src[:, None, :192], out[:, None, 576:768], rot_off=128)
        else:
            r = dsa.RopeTarget(src[:, :192].view(T, 1, 192), out[:, None, 576:768], rot_off=64, rot_dim=64)
        dsa.dsa_rope_append(g, pos, slots, freqs, rotate=r)
        return cache

    a, b = fused.clone(), fused.clone()
    got = call(a, a, a)
    want = call(fused.clone(), b, b)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(a, b) and want.any() and not torch.equal(a, fused)


@pytest.mark.parametrize("T", [1, 40, 2000])
def test_caches_of_one_tensor(dsa, T):
    """A layer's caches one behind the other, and rows from the same allocation."""
    P, ps = -(-T // 64) + 1, 64
    n = P * ps * 576
    pool = torch.zeros(2 * n + T * 576 + 64, dtype=BF, device="cuda")
    kv = [pool[i * n: (i + 1) * n].view(P, ps, 576) for i in range(2)]
    x = pool[2 * n: 2 * n + T * 576].view(T, 576)
    x.copy_(torch.randn(T, 576, generator=torch.Generator().manual_seed(T)))
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    pos, slots = _i32(np.arange(T)), _i32(np.arange(T))
    own = torch.zeros(P, ps, 576, dtype=BF, device="cuda")
    dsa.dsa_rope_append(dsa.AppendTarget(x.clone(), own, rot_off=512), pos, slots, freqs)
    dsa.dsa_rope_append([dsa.AppendTarget(x, c, rot_off=512) for c in kv], pos, slots, freqs)
    torch.cuda.synchronize()
    assert torch.equal(kv[0], own) and torch.equal(kv[1], own) and own.any()


def test_rows_that_turn_in_place_are_refused(dsa):
    T = 5
    x, cache = torch.zeros(T, 576, dtype=BF, device="cuda"), torch.zeros(1, 32, 576, dtype=BF, device="cuda")
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    before = dsa.dsa_launch_count()
    with pytest.raises(dsa.DSAError):
        dsa.dsa_rope_append(dsa.AppendTarget(x, cache, rot_off=512), _i32(range(T)), _i32(range(T)), freqs,
                            rotate=dsa.RopeTarget(x[:, None], rot_off=512))
    assert dsa.dsa_launch_count() == before
