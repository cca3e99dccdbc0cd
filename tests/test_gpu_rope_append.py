"""dsa_rope_append against 64-bit rotation and against the separate calls:
bf16 and 4-bit caches, rows from one tensor and from two, layouts, parts of the
row, strides, padding rows, bad slots, queries in the same launch, far
positions, large caches, graphs and streams."""
import numpy as np
import pytest
import torch

import dsa_inputs as DI
import steps_ref as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


def _rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _slots(T, rows, seed):
    return np.random.default_rng(seed).permutation(rows)[:T]


def _check_cache(cache, old, x, pos, slots, freqs, off, layout, scale):
    """Rows in their slots within the rounding of the rotation, every other
    element of the cache as it was."""
    D = x.shape[1]
    ref, mag = R.rope(R.f64(x)[:, None], pos, freqs.cpu().numpy(), off, layout, scale, False)
    want, tol = R.f64(old).reshape(-1, old.shape[-1]), np.zeros((old.numel() // old.shape[-1], old.shape[-1]))
    live = (slots >= 0) & (pos >= 0) & (slots < len(want))
    want[slots[live], :D] = ref[live, 0]
    tol[slots[live], :D] = R.rope_tol(ref, mag, BF)[live, 0] * (mag[live, 0] > 0)
    e = np.abs(R.f64(cache).reshape(want.shape) - want) - tol
    assert (e <= 0).all(), (np.argwhere(e > 0)[:4].tolist(), e.max())


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,D,off,rot,width,ps,split", [
    (1, 576, 512, 64, 576, 64, False), (1, 576, 512, 64, 640, 32, True), (5, 128, 0, 64, 128, 64, False),
    (37, 576, 512, 64, 640, 128, True), (130, 128, 0, 128, 128, 32, False), (3, 512, 0, 512, 512, 64, True),
    (9, 88, 40, 16, 104, 64, False), (9, 88, 40, 32, 104, 64, True), (2, 16, 0, 16, 16, 32, False),
    (700, 576, 0, 64, 576, 64, True), (4, 4096, 2048, 64, 4096, 32, False),
    # through shared memory
    (2501, 576, 512, 64, 640, 64, True), (2048, 128, 0, 64, 128, 32, False), (2100, 88, 40, 32, 104, 64, True),
    (1900, 512, 0, 512, 512, 64, True), (3000, 16, 0, 16, 16, 128, False), (1850, 2048, 1024, 256, 2048, 64, False),
])
def test_matches_64_bit(dsa, layout, T, D, off, rot, width, ps, split):
    P = -(-T // ps) + 2
    x, cache = _rand((T, D), T + D), _rand((P, ps, width), 3)
    old = cache.clone()
    pos = np.random.default_rng(T).integers(0, 131072, T)
    slots = _slots(T, P * ps, D)
    if T > 4:
        slots[2] = -1
        pos[4] = -1  # either one makes a padding row
    if T > 1000:  # and runs of them
        slots[np.random.default_rng(1).random(T) < 0.3] = -1
        slots[1000:1200] = -1
    freqs, scale = dsa.dsa_rope_freqs(rot, scaling="yarn", factor=40.0, device="cuda")
    if split:  # the rotated columns from a slice of a wider tensor
        wide = torch.cat([_rand((T, 8), 9), x[:, off: off + rot], _rand((T, 24), 10)], 1)
        g = dsa.AppendTarget(torch.cat([x[:, :off], x[:, off + rot:]], 1), cache, x_rot=wide[:, 8: 8 + rot],
                             rot_off=off, layout=layout, scale=scale)
    else:
        wide = torch.cat([_rand((T, 16), 9), x, _rand((T, 8), 10)], 1)
        g = dsa.AppendTarget(wide[:, 16: 16 + D], cache, rot_off=off, rot_dim=rot, layout=layout, scale=scale)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert dsa.dsa_rope_append(g, _i32(pos), _i32(slots), freqs, dev_status=st) is cache
    torch.cuda.synchronize()
    assert st.item() == 0
    _check_cache(cache, old, x, pos, slots, freqs, off, layout, scale)


@pytest.mark.parametrize("T", [1, 33, 1000, 12999])
def test_is_the_rotation_and_the_write_back(dsa, T):
    """The same values as dsa_rope followed by the write-backs, 16-bit and
    4-bit, queries and all."""
    P, ps, H = -(-T // 64) + 1, 64, 3
    rows, keys, q, qi = _rand((T, 576), 1), _rand((T, 128), 2), _rand((T, H, 192), 3), _rand((T, 32, 128), 4)
    rows[:, :512] *= torch.exp(_rand((T, 1), 5))
    pos, slots = _i32(np.arange(T) * 7 + 3), _i32(np.arange(T))  # one request that owns the pages in order
    freqs, scale = dsa.dsa_rope_freqs(64, device="cuda")
    meta = (_i32([T]), _i32([0, T]), _i32([0, P * ps]), _i32(np.arange(P)))
    kv, kc = torch.zeros(P, ps, 576, dtype=BF, device="cuda"), torch.zeros(P, ps, 128, dtype=BF, device="cuda")
    kv4 = torch.zeros(P, ps, 416, dtype=torch.uint8, device="cuda")
    kv_, kc_, kv4_ = kv.clone(), kc.clone(), kv4.clone()
    A, RT = dsa.AppendTarget, dsa.RopeTarget
    qo, qio = _rand((T, H, 576), 6), torch.zeros_like(qi)
    qo_, qio_ = qo.clone(), qio.clone()
    # all three caches and two more targets in one call
    dsa.dsa_rope_append([A(rows, kv, rot_off=512, layout="interleaved"), A(keys, kc, rot_dim=64),
                         A(rows[:, :512], kv4, x_rot=rows[:, 512:], rot_off=512, layout="interleaved")], pos, slots,
                        freqs, rotate=[RT(q[:, :, 128:], qo[:, :, 512:], layout="interleaved"),
                                       RT(qi, qio, rot_dim=64)])
    turned, tk = rows.clone()[:, None], keys.clone()[:, None]
    dsa.dsa_rope([RT(turned, rot_off=512, layout="interleaved"), RT(tk, rot_dim=64),
                  RT(q[:, :, 128:], qo_[:, :, 512:], layout="interleaved"), RT(qi, qio_, rot_dim=64)], pos, freqs)
    dsa.dsa_paged_write_back_pair(turned[:, 0], kv_, tk[:, 0], kc_, *meta)
    dsa.dsa_q4_write_back(turned[:, 0], kv4_, *meta)
    torch.cuda.synchronize()
    assert torch.equal(qo, qo_) and torch.equal(qio, qio_)
    # the angles are formed another way: a result may lie a step apart where it
    # falls on a rounding boundary, and no more than rarely
    for a, b in ((kv, kv_), (kc, kc_), (kv4[:, :, 288:].contiguous().view(BF), kv4_[:, :, 288:].contiguous().view(BF))):
        d = (a.double() - b.double()).abs()
        assert (d <= 2.0 ** -7 * b.double().abs() + 1e-6).all() and (d > 0).double().mean() < 1e-3
    assert torch.equal(kv[:, :, :512], kv_[:, :, :512]) and torch.equal(kc[:, :, 64:], kc_[:, :, 64:])
    assert torch.equal(kv4[:, :, :288], kv4_[:, :, :288])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,D,off,rot,width,split", [
    (1, 576, 512, 64, 640, True), (37, 576, 512, 64, 576, False), (130, 128, 0, 128, 128, False),
    (9, 88, 40, 32, 104, True), (3, 512, 0, 512, 512, True), (2501, 576, 512, 64, 576, True),
    (1850, 1024, 512, 256, 1024, False), (2, 4096, 2048, 64, 4096, False), (700, 576, 512, 64, 416, False),
    (13, 576, 512, 64, 416, True),
])
def test_beside_other_targets(dsa, layout, T, D, off, rot, width, split):
    """Rows by themselves and with another tensor that turns in the same launch
    take different ways to the cache, with the same arithmetic: the same bytes."""
    ps, P = 32, -(-T // 32) + 1
    x = _rand((T, D), T)
    x[T // 2, 3] = float("inf")
    cache = _rand((P, ps, width), 2)
    if width == 416:
        cache = torch.full((P, ps, 416), 5, dtype=torch.uint8, device="cuda")
    slots = _slots(T, P * ps, 4)
    slots[np.random.default_rng(6).random(T) < 0.1] = -1
    pos, slots = _i32(np.random.default_rng(5).integers(0, 1 << 20, T)), _i32(slots)
    freqs, scale = dsa.dsa_rope_freqs(rot, device="cuda")
    q = _rand((T, 2, rot), 7)
    old, got = cache.clone(), []
    for rotate in ([], [dsa.RopeTarget(q, torch.empty_like(q))]):
        to = cache.clone()
        if split:
            g = dsa.AppendTarget(torch.cat([x[:, :off], x[:, off + rot:]], 1), to, x_rot=x[:, off: off + rot],
                                 rot_off=off, layout=layout, scale=scale)
        else:
            g = dsa.AppendTarget(x, to, rot_off=off, rot_dim=rot, layout=layout, scale=scale)
        dsa.dsa_rope_append(g, pos, slots, freqs, rotate=rotate)
        got.append(to.view(torch.uint8))
    torch.cuda.synchronize()
    assert torch.equal(got[0], got[1]) and (T < 9 or not torch.equal(got[0], old.view(torch.uint8)))


@pytest.mark.parametrize("times", [1, 1040])
def test_quantised_rows_of_every_kind(dsa, times):
    """4-bit groups with infinities, NaN, zeros, tiny and huge values, byte for
    byte as the reference packs them; the rotary part in its place; rows of
    padding between them."""
    T = 12
    x = _rand((T, 576), 8)
    x[0, :16], x[1, 5], x[2, 17], x[3, :512] = 0, float("inf"), float("nan"), 0
    x[4, :512] *= 2.0 ** -12
    x[5, :512] *= 2.0 ** 14
    rows = np.tile(R.q4_pack(x), (times, 1))
    x, T = x.repeat(times, 1), T * times
    P = -(-T // 64)
    pos, slots = np.zeros(T, np.int64), _slots(T, P * 64, 1)  # position 0: the rotation leaves the values
    slots[np.random.default_rng(2).random(T) < 0.2] = -1
    cache = torch.full((P, 64, 416), 77, dtype=torch.uint8, device="cuda")
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    dsa.dsa_rope_append(dsa.AppendTarget(x, cache, rot_off=512, layout="interleaved"), _i32(pos), _i32(slots), freqs)
    torch.cuda.synchronize()
    want = np.full((P * 64, 416), 77, np.uint8)
    want[slots[slots >= 0]] = rows[slots >= 0]
    got = cache.cpu().numpy().reshape(-1, 416)
    zero = (want[:, 288:].view(np.uint16) & 0x7FFF) == 0  # +0 and -0 are one value
    same = got == want
    same[:, 288:] |= np.repeat(zero & ((got[:, 288:].copy().view(np.uint16) & 0x7FFF) == 0), 2, 1)
    assert same.all(), np.argwhere(~same)[:4].tolist()


def test_slots_out_of_range(dsa):
    T = 6
    x, cache = _rand((T, 128), 1), _rand((2, 32, 128), 2)
    old = cache.clone()
    pos, slots = np.arange(T) + 5, np.array([3, 64, -5, 2 ** 31 - 1, 63, -1])
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_rope_append(dsa.AppendTarget(x, cache, rot_dim=64), _i32(pos), _i32(slots), freqs, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0x4
    _check_cache(cache, old, x, pos, slots, freqs, 0, "half", 1.0)


def test_queries_that_do_not_lie_on_16_bytes(dsa):
    """Those take the element-by-element launch; positions alone decide there."""
    T = 7
    x, cache = _rand((T, 128), 1), _rand((1, 32, 128), 2)
    q = _rand((T, 3, 67), 3)
    want, old = q.clone(), cache.clone()
    pos, slots = np.arange(T) * 1000, np.array([-1, 3, 2, 9, 30, 1, 0])
    pos[5] = -1
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    dsa.dsa_rope(dsa.RopeTarget(want, rot_off=3), _i32(pos), freqs)
    dsa.dsa_rope_append([dsa.AppendTarget(x, cache, rot_dim=64)], _i32(pos), _i32(slots), freqs,
                        rotate=dsa.RopeTarget(q, rot_off=3))
    torch.cuda.synchronize()
    assert torch.equal(q, want)
    _check_cache(cache, old, x, pos, slots, freqs, 0, "half", 1.0)


def test_far_positions(dsa):
    pos = np.array([0, 1, 2 ** 20 + 1, 2 ** 24 + 3, 2 ** 30 + 7, 2 ** 31 - 1])
    x, cache = _rand((6, 64), 4), torch.zeros(1, 32, 64, dtype=BF, device="cuda")
    old = cache.clone()
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    dsa.dsa_rope_append(dsa.AppendTarget(x, cache), _i32(pos), _i32(np.arange(6)), freqs)
    torch.cuda.synchronize()
    _check_cache(cache, old, x, pos, np.arange(6), freqs, 0, "half", 1.0)


@pytest.mark.parametrize("freqs", [[0.0] * 32, [-3.0] * 16 + [7.5] * 16, [3.141592653589793] * 32, [1e-9] * 32])
def test_any_frequencies(dsa, freqs):
    """Negative, zero, large and tiny ones; half a turn."""
    f = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    pos = np.array([0, 1, 2, 1001, 65535, 1 << 20])
    x, cache = _rand((6, 64), 4), torch.zeros(1, 32, 64, dtype=BF, device="cuda")
    old = cache.clone()
    dsa.dsa_rope_append(dsa.AppendTarget(x, cache, layout="interleaved"), _i32(pos), _i32(np.arange(6)), f)
    torch.cuda.synchronize()
    _check_cache(cache, old, x, pos, np.arange(6), f, 0, "interleaved", 1.0)


def test_rows_past_32_bit_offsets(dsa):
    P, ps = 58000, 64  # 4.3 GB of latent rows
    cache = torch.zeros(P, ps, 576, dtype=BF, device="cuda")
    x = _rand((3, 576), 5)
    pos, slots = np.array([9, 10, 11]), np.array([P * ps - 1, 0, P * ps - 64])
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    dsa.dsa_rope_append(dsa.AppendTarget(x, cache, rot_off=512), _i32(pos), _i32(slots), freqs)
    torch.cuda.synchronize()
    flat = cache.view(-1, 576)
    ref, mag = R.rope(R.f64(x)[:, None], pos, freqs.cpu().numpy(), 512, "half", 1.0, False)
    e = np.abs(R.f64(flat[torch.as_tensor(slots).cuda()]) - ref[:, 0]) - R.rope_tol(ref, mag, BF)[:, 0]
    assert (e <= 0).all()
    assert torch.count_nonzero(flat.abs().amax(1)).item() == 3


def test_nothing_to_append(dsa):
    none, freqs = _i32([]), dsa.dsa_rope_freqs(64, device="cuda")[0]
    cache = _rand((1, 32, 128), 2)
    before = dsa.dsa_launch_count()
    dsa.dsa_rope_append(dsa.AppendTarget(cache.new_zeros(0, 128), cache, rot_dim=64), none, none, freqs)
    assert dsa.dsa_launch_count() == before
    # an empty pool has no slot to write to
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_rope_append(dsa.AppendTarget(_rand((1, 128), 1), cache[:0], rot_dim=64), _i32([4]), _i32([0]), freqs,
                        dev_status=st)
    assert st.item() == 0x4


def test_captured_and_on_two_streams(dsa):
    """A captured call follows positions and slots that change between
    replays; two calls at once on streams of their own."""
    T = 50
    x = _rand((T, 576), 1)
    caches = [torch.zeros(2, 64, 576, dtype=BF, device="cuda") for _ in range(4)]
    pos, slots = _i32(np.arange(T)), _i32(_slots(T, 128, 0))
    freqs, _ = dsa.dsa_rope_freqs(64, device="cuda")
    call = lambda c: dsa.dsa_rope_append(dsa.AppendTarget(x, c, rot_off=512), pos, slots, freqs)
    call(caches[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(caches[0])
    pos.copy_(_i32(np.arange(T) + 999))
    slots.copy_(_i32(_slots(T, 128, 5)))
    caches[0].zero_()
    g.replay()
    call(caches[1])
    torch.cuda.synchronize()
    assert torch.equal(caches[0], caches[1]) and caches[0].any()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s, c in zip(streams, caches[2:]):
            with torch.cuda.stream(s):
                call(c)
    torch.cuda.synchronize()
    assert torch.equal(caches[2], caches[1]) and torch.equal(caches[3], caches[1])


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_layer_step(dsa, kind, bits):
    """LayerRunner with append: the caches and queries of the step that rotates
    and writes in separate calls, two full layers and one that shares."""
    from deepseek_sparse_attention_score_gb300.layer import LayerRunner

    lens = ([1, 40, 0, 7], [400, 300, 64, 900]) if kind == "prefill" else ([1, 1, 1], [700, 64, 1025])
    freqs, scale = dsa.dsa_rope_freqs(64, scaling="yarn", factor=4.0, orig_max_pos=256)
    runs = []
    for append in (False, True):
        wl = DI.random_small(81, *lens, H=16, k=96, k_pages=4)
        wl.QB = 32
        wl.q, wl.kv, wl.indexer_types = wl.q * 2, wl.kv * 2, [0, 1]
        run = LayerRunner(wl, DEV, cache_bits=bits, tables=True, rope=(freqs, scale, "interleaved"), append=append)
        raw = run.new_kv[0].clone()
        run.step()
        before = dsa.dsa_launch_count()
        run.step()
        runs.append((run, raw, dsa.dsa_launch_count() - before))
    torch.cuda.synchronize()
    (a, _, na), (b, raw, nb) = runs
    assert a.status.item() == 0 and b.status.item() == 0
    assert torch.equal(b.new_kv[0], raw)
    assert nb < na  # the write-backs' launches are gone
    assert torch.equal(a.q[0], b.q[0]) and torch.equal(a.q_idx, b.q_idx)
    near = lambda x, y: ((x.double() - y.double()).abs() <= 2.0 ** -7 * y.double().abs() + 1e-6).all()
    for layer in range(2):
        if bits == 4:
            assert torch.equal(a.kv4[layer][:, :, :288], b.kv4[layer][:, :, :288])
            assert near(a.kv4[layer][:, :, 288:].contiguous().view(BF), b.kv4[layer][:, :, 288:].contiguous().view(BF))
        else:
            assert near(a.kv[layer], b.kv[layer])
    assert near(a.kcache[0], b.kcache[0])
    with pytest.raises(ValueError):
        LayerRunner(DI.random_small(34, [1], [64], H=16), DEV, append=True)
