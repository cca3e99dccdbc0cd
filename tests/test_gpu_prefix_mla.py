"""dsa_prefix_mla against attention in 64 bits over each request's own page
table: groups of all kinds, prefixes that end inside pages and tiles, heads that
do not divide a tile, decode and extends, requests inside the prefix, empty
ones, padding rows; its refusals, flags, graphs and streams."""
import numpy as np
import pytest
import torch

import steps_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SCALE = 192 ** -0.5


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as m

    return m


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Batch:
    """``groups``: (prefix, [(new tokens, positions behind the prefix), ...]).
    A request with fewer positions than the prefix has a negative second
    number. Whole pages of the prefix are shared, its last rows are copied."""

    def __init__(self, groups, H, ps=64, stride=576, pad=0, seed=0):
        rng = np.random.default_rng(seed)
        self.H, self.ps = H, ps
        self.q_lens = [q for _, g in groups for q, _ in g]
        self.seq = [p + n for p, g in groups for _, n in g]
        pages = [-(-n // ps) for n in self.seq]
        P = sum(pages) + 5
        ids = iter(rng.permutation(P))
        kv = torch.randn((P, ps, stride), generator=torch.Generator().manual_seed(seed)).to(BF)
        self.table, s = [], 0
        for p, g in groups:
            for k, (_, n) in enumerate(g):
                own = [next(ids) for _ in range(pages[s] if k == 0 else max(0, pages[s] - p // ps))]
                if k:
                    own = lead[: min(p // ps, pages[s])] + own
                    tail = min(p, self.seq[s]) - p // ps * ps
                    if tail > 0:
                        kv[own[p // ps], :tail] = kv[lead[p // ps], :tail]
                else:
                    lead = own
                self.table.append(own)
                s += 1
        used = {x for t in self.table for x in t}
        for x in set(range(P)) - used:
            kv[x] = float("nan")  # pages of others
        self.T = sum(self.q_lens)
        self.kv = kv.cuda()
        self.q = torch.randn((self.T + pad, H, 576), generator=torch.Generator().manual_seed(seed + 1)).to(BF).cuda()
        self.meta = (_i32(self.seq), _i32(np.cumsum([0] + self.q_lens)), _i32(np.cumsum([0] + [n * ps for n in pages])),
                     _i32([x for t in self.table for x in t]))
        self.prefix = _i32([p for p, _ in groups])
        self.groups = _i32(np.cumsum([0] + [len(g) for _, g in groups]))
        self.max_kv = max(self.seq + [1])

    def call(self, dsa, sm_scale=SCALE, **kw):
        kw.setdefault("max_kv", self.max_kv)
        return dsa.dsa_prefix_mla(self.q, self.kv, *self.meta, self.prefix, self.groups, sm_scale=sm_scale,
                                  want_lse=True, **kw)

    def reference(self, sm_scale=SCALE):
        """As steps_ref.attend, a request at a time on the GPU."""
        out, t0 = [], 0
        for n, kv, pages in zip(self.q_lens, self.seq, self.table):
            k = self.kv[torch.tensor(np.array(pages, np.int64), device="cuda")].reshape(-1, self.kv.shape[2])[:kv, :576].double()
            for t in range(t0, t0 + n, 32):
                e = min(t0 + n, t + 32)
                q = self.q[t:e].double()
                pos = torch.arange(kv - n + t - t0, kv - n + e - t0, device="cuda")
                off = torch.arange(kv, device="cuda")[None, None] > pos[:, None, None]
                z = (q @ k.T * sm_scale).masked_fill(off, -np.inf)
                mag = (q.abs() @ k.abs().T).masked_fill(off, 0).amax(-1)
                d = 576 * 2.0 ** -23 * abs(sm_scale) * mag
                d = d + z.masked_fill(off, 0).abs().amax(-1) * 2.0 ** -22 + 2.0 ** -18
                lse = torch.logsumexp(z, -1)
                p = torch.exp(z - lse[..., None])
                o, a = p @ k[:, :512], p @ k[:, :512].abs()
                out.append((o, lse, (R.BF16_HALF + 4 * d[..., None]) * a + R.BF16_HALF * o.abs(),
                            2 * d + 2.0 ** -20 * lse.abs()))
            t0 += n
        return [torch.cat(x).cpu().numpy() for x in zip(*out)]


def _check(dsa, b, sm_scale=SCALE, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = b.call(dsa, sm_scale, dev_status=st, **kw)
    torch.cuda.synchronize()
    assert st.item() == 0
    R.check_attend(o[: b.T], lse[: b.T], b.reference(sm_scale))
    return o, lse


@pytest.mark.parametrize("H", [1, 16, 40, 128, 300])
@pytest.mark.parametrize("prefix", [1, 64, 100, 128, 500])
def test_decode(dsa, H, prefix):
    _check(dsa, Batch([(prefix, [(1, 1), (1, 5), (1, 200)])], H))


@pytest.mark.parametrize("ps", [32, 64, 128])
@pytest.mark.parametrize("stride", [576, 640])
def test_page_sizes_and_strides(dsa, ps, stride):
    _check(dsa, Batch([(333, [(1, 1), (3, 150), (1, 31)]), (128, [(1, 40)])], 24, ps, stride))


@pytest.mark.parametrize("groups", [
    [(0, [(1, 1)])],                                       # one token, nothing shared
    [(0, [(5, 5), (1, 300)])],                             # nothing shared
    [(1000, [(1, 1)])],                                    # nobody to share with
    [(700, [(40, 45), (1, 1), (130, 400)])],               # extends
    [(200, [(0, 10), (1, 7), (0, 0), (2, 9)])],            # requests without new tokens, the first among them
    [(300, [(1, 4), (5, -100), (1, -299), (20, 3)])],      # requests and new tokens inside the prefix
    [(100, [(1, 3)] * 3), (0, []), (260, [(2, 2)]), (64, [(1, 64)] * 5), (5, [(1, 1), (33, 60)])],
    [(64, [(1, 1)] * 90)],                                 # many requests in a tile
    [(129, [(1, 127), (1, 128), (1, 129), (1, 255), (1, 256), (1, 257)])],
], ids=str)
def test_groups(dsa, groups):
    _check(dsa, Batch(groups, 16))
    _check(dsa, Batch(groups, 7, 32, seed=4))


def test_all_requests_are_one_group_by_default(dsa):
    b = Batch([(150, [(1, 3), (2, 90)])], 16)
    o, lse = _check(dsa, b)
    o2, lse2 = dsa.dsa_prefix_mla(b.q, b.kv, *b.meta, b.prefix, max_kv=b.max_kv, sm_scale=SCALE, want_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H,keys", [(16, 20000), (128, 9000), (1, 70000)])
def test_long_lists_in_many_shares(dsa, H, keys):
    b = Batch([(keys, [(1, 1), (1, 77)])], H)
    o, lse = _check(dsa, b)
    for _ in range(3):
        o2, lse2 = b.call(dsa)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)  # bit for bit


@pytest.mark.parametrize("H,T", [(128, 301), (20, 2000)])
def test_many_row_tiles(dsa, H, T):
    """More lists than pairs: whole lists and divided ones."""
    _check(dsa, Batch([(150, [(T // 2, T // 2 + 3), (T - T // 2, T)])], H))


@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-30, 3.0])
def test_scales(dsa, scale):
    _check(dsa, Batch([(150, [(1, 3), (3, 90)])], 16), scale)


def test_logits_far_apart(dsa):
    """Prefix and own logits that differ by hundreds either way, and rows whose
    largest logit comes late."""
    for grow in (1, -1):
        b = Batch([(384, [(1, 300), (1, 20)])], 16)  # whole pages: no copies
        ramp = torch.linspace(0.02, 4.0, 64 * b.kv.shape[0], device="cuda").flip(0) if grow < 0 else torch.linspace(
            0.02, 4.0, 64 * b.kv.shape[0], device="cuda")
        order = torch.tensor(np.argsort(np.array(b.table[0] + [x for x in range(b.kv.shape[0]) if x not in b.table[0]])),
                             device="cuda")
        b.kv *= ramp.view(-1, 64)[order][:, :, None].to(BF)
        _check(dsa, b, 0.5)


def test_padding_rows_are_left(dsa):
    b = Batch([(90, [(1, 3), (2, 9)]), (64, [(1, 1)])], 16, pad=5)
    o = torch.full((b.T + 5, 16, 512), 7.0, dtype=BF, device="cuda")
    lse = torch.full((b.T + 5, 16), 7.0, device="cuda")
    _check(dsa, b, o=o, lse=lse)
    assert (o[b.T:] == 7).all() and (lse[b.T:] == 7).all()


def test_as_the_window_call(dsa):
    """The same attention as dsa_window_mla without a window."""
    b = Batch([(500, [(1, 4), (9, 70), (1, 200)]), (77, [(30, 30), (1, 5)])], 32)
    o, lse = _check(dsa, b)
    o2, lse2 = dsa.dsa_window_mla(b.q, b.kv, *b.meta, max_kv=b.max_kv, sm_scale=SCALE, sliding_window=0, want_lse=True)
    assert (o.float() - o2.float()).abs().max() < 2e-2 and (lse - lse2).abs().max() < 1e-4


def test_nan_queries_stay_in_their_rows(dsa):
    b = Batch([(130, [(1, 3), (3, 90)])], 16)
    o, lse = _check(dsa, b)
    b.q[1, 3, 5] = float("nan")
    o2, lse2 = b.call(dsa)
    torch.cuda.synchronize()
    assert o2[1, 3].isnan().all() and lse2[1, 3].isnan()
    o2[1, 3], lse2[1, 3] = o[1, 3], lse[1, 3]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("groups,H", [
    ([(130, [(1, 3), (1, 90), (1, 600), (2, 40)])], 16), ([(0, [(1, 30), (1, 300), (1, 5)])], 40),
    ([(64, [(1, 500)] * 7), (300, [(1, 9)] * 3)], 5), ([(256, [(1, 200), (1, 200)])], 128),
    ([(10, [(1, 4000), (1, 3), (1, 4000)])], 16),  # lists that start with own keys
    ([(20, [(1, 1)] * 100)], 1),
], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_of_one_request_stay_with_it(dsa, groups, H, bad):
    """An infinity or a NaN among a request's own keys reaches its own outputs
    and none of the other requests', which share its row tile."""
    b = Batch(groups, H)
    o, lse = _check(dsa, b)
    first = np.cumsum([0] + b.q_lens)
    for s in {1, len(b.seq) - 1}:
        last = b.seq[s] - 1
        page = b.kv[b.table[s][last // 64]]
        old = page[last % 64].clone()
        page[last % 64, 3:512:7] = bad
        o2, lse2 = b.call(dsa)
        torch.cuda.synchronize()
        own = slice(int(first[s + 1]) - 1, int(first[s + 1]))  # its last token sees the position
        assert not o2[own].isfinite().all(-1).any()
        others = torch.ones(b.T, dtype=torch.bool, device="cuda")
        others[int(first[s]): int(first[s + 1])] = False
        assert torch.equal(o[others], o2[others]) and torch.equal(lse[others], lse2[others])
        page[last % 64] = old


def test_empty_calls(dsa):
    b = Batch([(130, [(1, 3)])], 16)
    before = dsa.dsa_launch_count()
    dsa.dsa_prefix_mla(b.q[:0], b.kv, *b.meta, b.prefix, max_kv=200, sm_scale=1.0)
    dsa.dsa_prefix_mla(b.q[:, :0].contiguous(), b.kv, *b.meta, b.prefix, max_kv=200, sm_scale=1.0)
    assert dsa.dsa_launch_count() == before
    # rows without tokens: nothing is written
    b = Batch([(130, [(0, 3), (0, 1)])], 16, pad=2)
    o = torch.full((2, 16, 512), 7.0, dtype=BF, device="cuda")
    b.call(dsa, o=o)
    assert (o == 7).all()


@pytest.mark.parametrize("what", ["long prefix", "negative prefix", "groups out of order", "groups past the end",
                                  "requests without a group", "bad page", "long request", "short request"])
def test_flags(dsa, what):
    b = Batch([(100, [(1, 30), (1, 60)]), (70, [(2, 20), (1, 1)])], 16)
    want, wl = b.call(dsa)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    same = np.ones(5, bool)  # tokens with the right output all the same
    if what == "long prefix":
        b.prefix[0] = 1000  # all of request 0 and as much of request 1
        b.kv[b.table[1][: len(b.table[0])]] = b.kv[b.table[0]]
        want, wl = b.call(dsa)
        st.zero_()
    elif what == "negative prefix":
        b.prefix[1] = -3
    elif what == "groups out of order":
        b.groups[1] = 3
        b.groups[2] = 1
        same[:] = False
    elif what == "groups past the end":
        b.groups[2] = 9
        same[2:] = False
    elif what == "requests without a group":
        b.groups[2] = 3
        same[4] = False
    elif what == "bad page":
        b.meta[3][1] = b.kv.shape[0]
        same[:2] = False
    elif what == "long request":
        b.meta[0][1] = 5000
        same[1] = False
    else:
        b.meta[0][2] = 1  # fewer positions than new tokens
        same[2:] = False
    o, lse = b.call(dsa, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() & 0x2
    ok = torch.from_numpy(same).cuda()
    if what == "long prefix":
        # through other pages and tiles: equal but for rounding
        assert (o.float() - want.float()).abs().max() < 2e-2 and (lse - wl).abs().max() < 1e-4
    elif same.any():
        assert (o[ok].float() - want[ok].float()).abs().max() < 2e-2 and (lse[ok] - wl[ok]).abs().max() < 1e-4


def test_captured_and_replayed(dsa):
    """A captured call follows lengths that grow between replays."""
    b = Batch([(200, [(1, 10), (1, 60)])], 16)
    ws = torch.empty(dsa.dsa_prefix_mla_workspace_size(b.T, 16, 1), dtype=torch.uint8, device="cuda")
    o, lse = b.call(dsa, ws=ws, max_kv=300)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.call(dsa, ws=ws, o=o, lse=lse, max_kv=300)
    for grow in (0, 1, 30):
        seq = [n + grow if len(t) * 64 >= n + grow else n for n, t in zip([210, 260], b.table)]
        b.meta[0].copy_(_i32(seq))
        b.seq = seq
        o.zero_()
        ws.fill_(255)  # nothing is kept there between calls
        g.replay()
        torch.cuda.synchronize()
        R.check_attend(o, lse, b.reference())


def test_two_streams(dsa):
    """Calls at once with a workspace each."""
    bs = [Batch([(900, [(1, 10), (1, 60)])], 16, seed=1), Batch([(300, [(40, 50)]), (64, [(1, 1)] * 9)], 40, seed=2)]
    want = [b.call(dsa) for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        got = []
        for s, b in zip(streams, bs):
            with torch.cuda.stream(s):
                got.append(b.call(dsa))
        torch.cuda.synchronize()
        for (o, l), (o2, l2) in zip(want, got):
            assert torch.equal(o, o2) and torch.equal(l, l2)


def test_cache_past_32_bit_offsets(dsa):
    b = Batch([(700, [(1, 10), (1, 100)])], 16)
    P = 60000  # 4.4 GB
    big = torch.zeros((P, 64, 576), dtype=BF, device="cuda")
    n = b.kv.shape[0]
    big[P - n:] = b.kv
    b.kv = big
    b.meta[3].add_(P - n)
    b.table = [[x + P - n for x in t] for t in b.table]
    _check(dsa, b)


@pytest.mark.parametrize("what", ["requests", "groups", "row tiles"])
def test_more_than_the_plan_keeps_in_shared_memory(dsa, what):
    """Thousands of requests (most of them paused), hundreds of groups, more
    than a thousand row tiles."""
    if what == "requests":
        groups = [(70, [(1 if i % 97 == 5 else 0, 1 + i % 5) for i in range(3500)]), (33, [(0, 1)] * 200 + [(2, 40)])]
        _check(dsa, Batch(groups, 16, 32))
    elif what == "groups":
        _check(dsa, Batch([(i % 70, [(i % 3, i % 3 + 1), (1, 1 + i % 40)][: 1 + i % 2]) for i in range(600)], 4, 32))
    else:
        _check(dsa, Batch([(40, [(700, 700), (1, 1), (1399, 1400)])], 128, 128))


def test_appended_then_attended(dsa):
    """A step as it is used: page tables from lengths, rows rotated on their way
    into the cache together with the queries, then attention over the shared
    prefix; eager, and captured and replayed while the requests grow."""
    own = (61, 70, 62)  # two requests enter their fourth page
    b = Batch([(130, [(1, own[0]), (1, own[1]), (3, own[2])])], 16)
    S, H, T = 3, 16, b.T
    freqs, scale = dsa.dsa_rope_freqs(64, scaling="yarn", factor=4.0, orig_max_pos=256, device="cuda")
    width = max(len(t) for t in b.table) + 1
    bt = torch.full((S, width), -1, dtype=torch.int32)
    for s, t in enumerate(b.table):
        bt[s, : len(t)] = torch.tensor(t)
    used = {x for t in b.table for x in t}
    free = _i32([x for x in range(b.kv.shape[0]) if x not in used])
    b.kv = b.kv.nan_to_num()  # pages that the list hands out are written in part
    PTW = sum(len(t) for t in b.table) + 4
    seq, qn = b.meta[0], _i32(b.q_lens)
    q_raw, rows = b.q.clone(), torch.randn(T, 576, device="cuda").to(BF)
    q = torch.empty_like(q_raw)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    state = torch.zeros(3 + 2 * S, dtype=torch.int32, device="cuda")
    bt, old = bt.cuda(), b.kv.clone()
    tb = dsa.dsa_build_page_tables(qn, seq, bt, free, T=T, PTW=PTW, free_state=state, dev_status=st)
    o, lse = torch.empty(T, H, 512, dtype=BF, device="cuda"), torch.empty(T, H, device="cuda")
    ws = torch.empty(dsa.dsa_prefix_mla_workspace_size(T, H), dtype=torch.uint8, device="cuda")

    def step():
        dsa.dsa_build_page_tables(qn, seq, bt, free, T=T, PTW=PTW, free_state=state, out=tb, dev_status=st)
        dsa.dsa_rope_append(dsa.AppendTarget(rows, b.kv, rot_off=512, layout="interleaved", scale=scale), tb.positions,
                            tb.slots, freqs, dev_status=st,
                            rotate=dsa.RopeTarget(q_raw, q, rot_off=512, layout="interleaved", scale=scale))
        dsa.dsa_prefix_mla(q, b.kv, seq, tb.cu_q_lens, tb.cu_kv_lens, tb.page_indices, b.prefix, max_kv=400,
                           sm_scale=SCALE, o=o, lse=lse, ws=ws, dev_status=st)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for grow in (0, 1, 2):
        b.kv.copy_(old)
        b.seq = [130 + n + grow for n in own]
        seq.copy_(_i32(b.seq))
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert st.item() == 0
        pos = np.concatenate([np.arange(n - k, n) for n, k in zip(b.seq, b.q_lens)])
        assert np.array_equal(tb.positions.cpu().numpy(), pos)
        x, mag = R.rope(R.f64(rows)[:, None], pos, freqs.cpu().numpy(), 512, "interleaved", scale, False)
        got = R.f64(b.kv.view(-1, 576)[tb.slots.long()])
        assert (np.abs(got - x[:, 0]) <= R.rope_tol(x, mag, BF)[:, 0]).all()
        y, mag = R.rope(R.f64(q_raw), pos, freqs.cpu().numpy(), 512, "interleaved", scale, False)
        assert (np.abs(R.f64(q) - y) <= R.rope_tol(y, mag, BF)).all()
        cu = tb.cu_kv_lens.cpu().numpy() // 64
        pages = tb.page_indices.cpu().numpy()
        b.table = [pages[a: c].tolist() for a, c in zip(cu, cu[1:])]
        b.q = q
        R.check_attend(o, lse, b.reference())
