"""YaRN's factors where only a part of the head rotates: the temperature is
that of the whole logit, m(mscale_all_dim)^2, and the rotated columns carry the
ratio of the two factors."""
import math

import numpy as np
import pytest
import torch

import steps_ref as R

INVALID = -1


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


@pytest.mark.parametrize("factor", [1.0, 4.0, 40.0])
@pytest.mark.parametrize("c,call", [(1.0, 1.0), (0.707, 0.707), (1.0, 0.707), (1.0, 0.0)])
def test_factors(dsa, factor, c, call):
    m = lambda k: 0.1 * k * math.log(factor) + 1
    rotated, logits = dsa.dsa_rope_attention_scales(factor, mscale=c, mscale_all_dim=call)
    assert rotated == pytest.approx(m(c) / m(call), rel=1e-15) and logits == pytest.approx(m(call) ** 2, rel=1e-15)
    if c == call:
        assert rotated == 1.0
    # a head that rotates whole, with the factor on queries and keys: the frequencies' own factor
    if call == 0.0:
        assert rotated == dsa.dsa_rope_freqs(64, scaling="yarn", factor=factor)[1] and logits == 1.0


@pytest.mark.parametrize("kw", [dict(factor=0.5), dict(factor=math.nan), dict(factor=math.inf),
                                dict(factor=4.0, mscale=math.inf), dict(factor=4.0, mscale_all_dim=math.nan),
                                dict(factor=4.0, mscale_all_dim=-10.0)])
def test_refusals(dsa, kw):
    with pytest.raises(dsa.DSAError) as e:
        dsa.dsa_rope_attention_scales(**kw)
    assert e.value.rc == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("c,call", [(1.0, 1.0), (1.0, 0.707)])
def test_logits_of_a_head_that_rotates_in_part(dsa, c, call):
    """The log-sum over a single key is its logit: rotation, write-back and
    attention against the definition over all 576 columns."""
    from gpu_util import meta_to
    import dsa_inputs as DI

    dev, factor = torch.device("cuda"), 40.0
    wl = DI.random_small(51, [1, 1, 1], [700, 64, 301], H=16)
    rg, pos = wl.rg, wl.rg.token_pos()
    freqs, _ = dsa.dsa_rope_freqs(64, scaling="yarn", factor=factor)
    rotated, logits = dsa.dsa_rope_attention_scales(factor, mscale=c, mscale_all_dim=call)
    q, rows, kv = wl.q[0].to(dev), torch.randn(rg.T, 1, 576).to(torch.bfloat16).to(dev), wl.kv[0].to(dev)
    q0, k0 = R.f64(q), R.f64(rows)
    T = dsa.RopeTarget
    dsa.dsa_rope([T(q, rot_off=512, layout="interleaved", scale=rotated),
                  T(rows, rot_off=512, layout="interleaved", scale=rotated)],
                 torch.from_numpy(pos.astype(np.int32)).to(dev), freqs.to(dev))
    meta = meta_to(rg, dev)
    dsa.dsa_paged_write_back(rows[:, 0], kv, *meta)
    _, lse = dsa.dsa_window_mla(q, kv, *meta, max_kv=rg.max_kv, sm_scale=wl.sm_scale * logits, sliding_window=1,
                                want_lse=True)
    # the definition: every column unscaled, the logit times m(call)^2 for the
    # latent part and m(c)^2 for the rotary part
    m = lambda k: 0.1 * k * math.log(factor) + 1
    qr, qm = R.rope(q0, pos, freqs.numpy(), 512, "interleaved", 1.0, False)
    kr, km = R.rope(k0, pos, freqs.numpy(), 512, "interleaved", 1.0, False)
    part = lambda s: (qr[..., s] * kr[..., s]).sum(-1)
    want = wl.sm_scale * (m(call) ** 2 * part(slice(0, 512)) + m(c) ** 2 * part(slice(512, 576)))
    # rotated columns are rounded to bf16 once on each side, after fp32 turns
    # that are off by 2^-20 of |a| + |b|; 576 fp32 additions, and 2^-20 for the
    # factors and the log-sum
    mag = lambda s: (np.abs(qr[..., s]) * np.abs(kr[..., s])).sum(-1)
    turn = 2.0 ** -20 * (qm * np.abs(kr) + km * np.abs(qr))[..., 512:].sum(-1)
    tol = wl.sm_scale * (m(c) ** 2 * (2.02 * R.BF16_HALF * mag(slice(512, 576)) + 1.02 * turn) +
                         576 * 2.0 ** -23 * m(1.0) ** 2 * mag(slice(0, 576))) + 2.0 ** -20 * (1 + np.abs(want))
    assert (np.abs(R.f64(lse) - want) <= tol).all()
