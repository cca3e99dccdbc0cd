"""Measured cases of two operators between a layer's projections and its attention's output: appending rows to the
paged caches with the rotary positions applied on the way, and attention of requests that share a long prefix, whose
keys are read once for all of them.

Every case has a plain form (elementary torch operations, ``own = False``) and the framework's calls
(``own = True``) on the same inputs; ``exact`` restates each operator in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
NOPE, ROPE = 512, 64          # latent row: 512 value dims, 64 rotary dims
DK = NOPE + ROPE
IDX_HEADS, IDX_DIM = 32, 128  # indexer queries and keys, of which the first 64 columns rotate
GROUP = 16                    # 4-bit codes that share a scale
ROW4 = NOPE // 2 + NOPE // GROUP + 2 * ROPE  # bytes of a 4-bit cache row
SM_SCALE = 1.0 / math.sqrt(192.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of one layer: 64 new tokens, their queries and indexer queries rotated by the same call
        dict(name="append_decode", op="append", T=64, pad=0, H=128, bits=16, layout="interleaved", split=False,
             max_pos=131072, ps=64),
        # a decode step into the 4-bit cache, the latent part and the rotary part from two tensors
        dict(name="append_decode_4bit", op="append", T=48, pad=5, H=0, bits=4, layout="interleaved", split=True,
             max_pos=131072, ps=64),
        # a prefill's rows
        dict(name="append_prefill", op="append", T=8192, pad=0, H=0, bits=16, layout="interleaved", split=True,
             max_pos=131072, ps=64),
        # ragged extends into the 4-bit cache, padded for a captured step
        dict(name="append_extend_4bit", op="append", T=12289, pad=95, H=0, bits=4, layout="half", split=False,
             max_pos=32768, ps=32),
        # the rows of a whole batch of long prompts
        dict(name="append_prompts", op="append", T=65537, pad=0, H=0, bits=16, layout="half", split=False,
             max_pos=65537, ps=128),
        # the smallest: two requests behind one system prompt
        dict(name="prefix_tiny", op="prefix", G=1, S=2, q_total=2, H=16, prefix=512, own_max=32, ps=64),
        # decode of a busy batch behind one long document, the heads of one of eight ranks
        dict(name="prefix_decode_16", op="prefix", G=1, S=64, q_total=64, H=16, prefix=32768, own_max=1024, ps=64),
        # the same with all heads
        dict(name="prefix_decode_128", op="prefix", G=1, S=32, q_total=32, H=128, prefix=16384, own_max=512, ps=64),
        # a few samples of one very long prompt
        dict(name="prefix_long", op="prefix", G=1, S=4, q_total=4, H=128, prefix=131072, own_max=2048, ps=64),
        # several prompts in one batch, ends inside pages, groups of unlike size
        dict(name="prefix_groups", op="prefix", G=5, S=37, q_total=60, H=40, prefix=9001, own_max=700, ps=32),
        # ragged extends behind a shared prompt
        dict(name="prefix_extend", op="prefix", G=1, S=6, q_total=500, H=16, prefix=8191, own_max=600, ps=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    ps = rng.choice([32, 64, 128])
    if rng.random() < 0.4:
        heads = rng.random() < 0.4
        T = _log_int(rng, 1, 512 if heads else 65537)
        return dict(op="append", T=T, pad=rng.choice([0, 1, 37]), H=_log_int(rng, 1, 128) if heads else 0,
                    bits=rng.choice([4, 16]), layout=rng.choice(["interleaved", "half"]), split=rng.random() < 0.5,
                    max_pos=max(T, _log_int(rng, 8192, 131072)), ps=ps)
    G = rng.choice([1, 1, 1, 2, 5])
    S = _log_int(rng, G, 64)
    H = _log_int(rng, 1, 128)
    q_total = S if rng.random() < 0.6 else _log_int(rng, S, max(S, 8192 // H))
    own_max = _log_int(rng, 1, 4096)
    # no more (query row, key) pairs than the largest listed case has
    most = max(64, (1 << 26) // (q_total * H) - own_max)
    return dict(op="prefix", G=G, S=S, q_total=q_total, H=H, prefix=_log_int(rng, 1, min(131072, most)),
                own_max=own_max, ps=ps)


# ------------------------------------------------------------- 4-bit format
# A row: 256 bytes of e2m1 codes, 32 e4m3 scales (one per 16 dims), 64 bf16 rotary dims. Dim 8*w + j sits in
# 32-bit word w; the even dims of a word are its nibbles 0..3, the odd ones its nibbles 4..7.
NIBBLE = (0, 4, 1, 5, 2, 6, 3, 7)  # nibble of dim j of a word
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pack(rows):
    """bf16 rows [N, 576] as bytes [N, 416]: scale = max / 6 in e4m3, codes to the nearest, ties to the even one."""
    x = rows[:, :NOPE].float().view(-1, NOPE // GROUP, GROUP)
    s = (x.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.float()[..., None]
    t = torch.where(d > 0, x.abs() / d, torch.zeros_like(x))
    code = torch.zeros_like(t, dtype=torch.uint8)
    for limit, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (t >= limit if up else t > limit).to(torch.uint8)
    code = (code | (torch.signbit(x).to(torch.uint8) << 3)).view(-1, NOPE // 8, 8)[:, :, [0, 2, 4, 6, 1, 3, 5, 7]]
    by = (code[:, :, 0::2] | (code[:, :, 1::2] << 4)).reshape(-1, NOPE // 2)
    return torch.cat([by, s.view(torch.uint8), rows[:, NOPE:].contiguous().view(torch.uint8).view(-1, 2 * ROPE)], 1)


def _unpack(b):
    """cache rows [N, 416] -> the values they stand for, fp32 [N, 576]"""
    by = b[:, : NOPE // 2].view(-1, NOPE // 8, 4)
    nib = torch.stack([by & 15, by >> 4], -1).view(-1, NOPE // 8, 8)[:, :, list(NIBBLE)].reshape(-1, NOPE)
    mag = torch.tensor(E2M1, device=b.device)[(nib & 7).long()]
    s = b[:, NOPE // 2: NOPE // 2 + NOPE // GROUP].contiguous().view(torch.float8_e4m3fn).float()
    v = (torch.where(nib >= 8, -mag, mag).view(-1, NOPE // GROUP, GROUP) * s[..., None]).view(-1, NOPE)
    return torch.cat([v, b[:, NOPE // 2 + NOPE // GROUP:].contiguous().view(torch.bfloat16).float()], 1)


# ------------------------------------------------------------------- inputs
def _lens(case):
    """Per request: its group, new tokens and positions with them, and per group its prefix: the same for every seed.
    Groups are runs of requests; every request holds its group's prefix and up to own_max positions of its own."""
    rng, S, G = np.random.default_rng(11), case["S"], case["G"]
    cuts = np.sort(rng.permutation(np.arange(1, S))[: G - 1]) if G > 1 else np.zeros(0, np.int64)
    groups = np.concatenate([[0], cuts, [S]]).astype(np.int64)
    prefix = np.full(G, case["prefix"], np.int64)
    if G > 1:
        prefix[1:] = np.maximum(1, (case["prefix"] * rng.random(G - 1)).astype(np.int64))
    q = np.ones(S, np.int64)
    if case["q_total"] > S:
        q += rng.multinomial(case["q_total"] - S, rng.dirichlet(np.ones(S)))
    mine = q - 1 + rng.integers(1, case["own_max"] + 1, S)  # positions behind the prefix, the new tokens among them
    of = np.repeat(np.arange(G), np.diff(groups))
    return groups, prefix, of, q, prefix[of] + mine


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=dtype)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = {"case": dict(case)}
    if case["op"] == "append":
        T, pad, ps = case["T"], case["pad"], case["ps"]
        P = -(-T // ps) + 3
        # runs of new positions of several requests, each from a place of its own; padding rows behind them
        cut = np.unique(rng.integers(0, T, 5))
        start = rng.integers(0, case["max_pos"], T)[np.searchsorted(cut, np.arange(T), side="right")]
        pos = (start + np.arange(T)) % case["max_pos"]
        pages = rng.permutation(P)
        slot = pages[np.arange(T) // ps] * ps + np.arange(T) % ps
        none = np.full(pad, -1)
        st.update(positions=_ints(np.concatenate([pos, none])), slots=_ints(np.concatenate([slot, none])),
                  freqs=torch.from_numpy(10000.0 ** (-np.arange(0, ROPE, 2) / ROPE)).to(DEV))
        T += pad
        rows = _randn(gen, T, DK)
        rows[:, :NOPE] *= torch.exp(_randn(gen, T, 1, dtype=torch.float32)).bfloat16()  # rows of unlike size
        if case["split"]:  # the normalised latent is a tensor of its own, the rotary part a slice of the projection
            st.update(latent=rows[:, :NOPE].contiguous(), rotary=rows[:, NOPE:])
        else:
            st.update(rows=rows)
        st["k_idx"] = _randn(gen, T, IDX_DIM)
        st["cache"] = (torch.zeros(P, ps, ROW4, device=DEV, dtype=torch.uint8) if case["bits"] == 4 else
                       torch.zeros(P, ps, DK, device=DEV, dtype=torch.bfloat16))
        st["idx_cache"] = torch.zeros(P, ps, IDX_DIM, device=DEV, dtype=torch.bfloat16)
        if case["bits"] == 4:
            st["values"] = torch.empty(T, DK, device=DEV, dtype=torch.bfloat16)
        if case["H"]:
            st.update(q_proj=_randn(gen, T, case["H"], 128 + ROPE), q=_randn(gen, T, case["H"], DK),
                      q_idx=_randn(gen, T, IDX_HEADS, IDX_DIM),
                      q_idx_out=torch.zeros(T, IDX_HEADS, IDX_DIM, device=DEV, dtype=torch.bfloat16))
        return st
    S, ps = case["S"], case["ps"]
    groups, prefix, of, q, seq = _lens(case)
    base, pages = prefix[of] // ps, -(-seq // ps)
    P = int((prefix // ps).sum() + (pages - base).sum()) + 3
    ids = iter(rng.permutation(P))
    take = lambda n: [next(ids) for _ in range(int(n))]
    shared = [take(p // ps) for p in prefix]
    table = [shared[g] + take(pages[s] - base[s]) for s, g in enumerate(of)]
    kv = _randn(gen, P, ps, DK)
    for g in range(len(prefix)):  # a prefix that ends inside a page: every request holds a copy of its last rows
        tail, first = int(prefix[g] % ps), int(groups[g])
        for s in range(first + 1, int(groups[g + 1])):
            if tail:
                kv[table[s][base[s]], :tail] = kv[table[first][base[first]], :tail]
    T = int(q.sum())
    st.update(kv=kv, q=_randn(gen, T, case["H"], DK), seq_lens=_ints(seq), cu_q_lens=_ints(np.cumsum(np.r_[0, q])),
              cu_kv_lens=_ints(np.cumsum(np.r_[0, pages * ps])), page_indices=_ints(np.concatenate(table)),
              prefix_lens=_ints(prefix), group_offsets=_ints(groups), T=T, max_kv=int(seq.max()),
              lens=(groups, prefix, q, seq, table), o=torch.empty(T, case["H"], NOPE, device=DEV, dtype=torch.bfloat16))
    return st


# ------------------------------------------------------------------- passes
def run(st):
    append = st["case"]["op"] == "append"
    if own:
        return _own_append(st) if append else _own_prefix(st)
    return _plain_append(st) if append else _plain_prefix(st)


def _own_append(st):
    import deepseek_sparse_attention_score_gb300 as dsa
    case, A, R = st["case"], dsa.AppendTarget, dsa.RopeTarget
    lay = case["layout"]
    if case["split"]:
        rows = A(st["latent"], st["cache"], x_rot=st["rotary"], rot_off=NOPE, rot_dim=ROPE, layout=lay)
    else:
        rows = A(st["rows"], st["cache"], rot_off=NOPE, rot_dim=ROPE, layout=lay)
    keys = A(st["k_idx"], st["idx_cache"], rot_off=0, rot_dim=ROPE, layout="half")
    turn = []
    if case["H"]:
        turn = [R(st["q_proj"][:, :, 128:], st["q"][:, :, NOPE:], layout=lay),
                R(st["q_idx"], st["q_idx_out"], rot_dim=ROPE, layout="half")]
    dsa.dsa_rope_append([rows, keys], st["positions"], st["slots"], st["freqs"], rotate=turn)
    if case["bits"] == 4:
        dsa.dsa_q4_read_rows(st["cache"], st["slots"], out=st["values"])
    return _appended(st)


def _appended(st):
    out = [st["values"] if st["case"]["bits"] == 4 else st["cache"], st["idx_cache"]]
    return out + ([st["q"][:, :, NOPE:], st["q_idx_out"]] if st["case"]["H"] else [])


def _own_prefix(st):
    import deepseek_sparse_attention_score_gb300 as dsa
    return dsa.dsa_prefix_mla(st["q"], st["kv"], st["seq_lens"], st["cu_q_lens"], st["cu_kv_lens"], st["page_indices"],
                              st["prefix_lens"], st["group_offsets"], max_kv=st["max_kv"], sm_scale=SM_SCALE,
                              o=st["o"], want_lse=True)


def _plain_append(st):
    case, T = st["case"], st["case"]["T"]  # the rows behind the first T are padding
    pos, slots = st["positions"][:T].double(), st["slots"][:T].long()
    ang = pos[:, None, None] * st["freqs"]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()

    def turn(x, layout):  # the first ROPE columns of [T, h, w], in 32 bits
        y = x[:T].float()
        r = y[..., :ROPE]
        if layout == "half":
            a, b = r[..., : ROPE // 2], r[..., ROPE // 2:]
            y[..., :ROPE] = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            y[..., :ROPE] = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return y.bfloat16()

    lay = case["layout"]
    latent, rotary = ((st["latent"], st["rotary"]) if case["split"] else (st["rows"][:, :NOPE], st["rows"][:, NOPE:]))
    rows = torch.cat([latent[:T], turn(rotary[:, None], lay)[:, 0]], 1)
    st["idx_cache"].view(-1, IDX_DIM)[slots] = turn(st["k_idx"][:, None], "half")[:, 0]
    if case["bits"] == 4:
        flat = st["cache"].view(-1, ROW4)
        flat[slots] = _pack(rows)
        st["values"][:T] = _unpack(flat[slots]).bfloat16()
        st["values"][T:] = 0
    else:
        st["cache"].view(-1, DK)[slots] = rows
    if case["H"]:
        st["q"][:T, :, NOPE:] = turn(st["q_proj"][:, :, 128:], lay)
        st["q_idx_out"][:T] = turn(st["q_idx"], "half")
    return _appended(st)


def _plain_prefix(st):
    """Logits of a group's queries against the prefix in one product, those of a request's own positions in another;
    one softmax over both."""
    case, H, ps = st["case"], st["case"]["H"], st["case"]["ps"]
    groups, prefix, q_lens, seq, _ = st["lens"]
    cu_q = np.cumsum(np.r_[0, q_lens])
    cu_p = np.cumsum(np.r_[0, -(-seq // ps)])
    flat, table = st["kv"].view(-1, DK), st["page_indices"].long()
    lse = torch.empty(st["T"], H, device=DEV)

    def keys(s, lo, hi):
        j = torch.arange(lo, hi, device=DEV)
        return flat[table[int(cu_p[s]) + j // ps] * ps + j % ps].float()

    for g in range(len(prefix)):
        p0 = int(prefix[g])
        shared = keys(int(groups[g]), 0, p0)
        s = int(groups[g])
        while s < groups[g + 1]:
            e = s + 1  # requests whose logits fit beside each other
            while e < groups[g + 1] and (cu_q[e + 1] - cu_q[s]) * H * p0 <= 1 << 28:
                e += 1
            x = st["q"][int(cu_q[s]): int(cu_q[e])].float().view(-1, DK) * SM_SCALE
            z = x @ shared.T
            m = z.amax(1)
            mine = []
            for r in range(s, e):
                a, b = int(cu_q[r] - cu_q[s]) * H, int(cu_q[r + 1] - cu_q[s]) * H
                k = keys(r, p0, int(seq[r]))
                y = x[a:b] @ k.T
                pos = int(seq[r] - q_lens[r]) + torch.arange(int(q_lens[r]), device=DEV).repeat_interleave(H)
                y = torch.where(torch.arange(p0, int(seq[r]), device=DEV)[None] <= pos[:, None], y, -math.inf)
                m[a:b] = torch.maximum(m[a:b], y.amax(1))
                mine.append((a, b, k, y))
            z = torch.exp_(z.sub_(m[:, None]))
            total, out = z.sum(1), z @ shared[:, :NOPE]
            for a, b, k, y in mine:
                w = torch.exp(y - m[a:b, None])
                total[a:b] += w.sum(1)
                out[a:b] += w @ k[:, :NOPE]
            st["o"][int(cu_q[s]): int(cu_q[e])] = (out / total[:, None]).view(-1, H, NOPE).bfloat16()
            lse[int(cu_q[s]): int(cu_q[e])] = (m + torch.log(total)).view(-1, H)
            s = e
    return st["o"], lse


# --------------------------------------------------------------------- work
def work(case):
    if case["op"] == "append":
        T, H = case["T"], case["H"]
        rows = 2 * DK + (ROW4 if case["bits"] == 4 else 2 * DK) + 2 * 2 * IDX_DIM
        turned = 2 * 2 * (H * ROPE + IDX_HEADS * IDX_DIM) if H else 0
        # a 4-bit case reads its rows back: the values that they stand for
        back = T * (ROW4 + 2 * DK) if case["bits"] == 4 else 0
        return {"bytes": T * (rows + turned + 8) + back + 4 * ROPE,
                "flops": 3 * T * ROPE * (2 + (H + IDX_HEADS if H else 0))}
    H = case["H"]
    groups, prefix, of, q, seq = _lens(case)
    T = int(q.sum())
    rows = int(prefix.sum() + (seq - prefix[of]).sum())
    pairs = int(sum(n * (kv - n) + n * (n + 1) // 2 for n, kv in zip(q.tolist(), seq.tolist())))
    return {"bytes": rows * 2 * DK + T * H * (2 * (DK + NOPE) + 4), "flops": 2 * pairs * H * (DK + NOPE)}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """The operators' definitions in 64 bits."""
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "append" else _exact_prefix(st)


def _exact_append(st):
    """Each pair is a complex number, turned by exp(i * angle); 4-bit values by a search of the nearest."""
    case = st["case"]
    pos, slots = st["positions"].tolist(), st["slots"].long()
    live = torch.tensor([p >= 0 for p in pos], device=DEV)
    ang = st["positions"].double()[:, None] * st["freqs"][None]
    w = torch.polar(torch.ones_like(ang), ang)

    def turn(x, layout):
        x = x.double()
        if layout == "half":
            z = torch.complex(x[..., : ROPE // 2], x[..., ROPE // 2:])
        else:
            z = torch.view_as_complex(x.reshape(*x.shape[:-1], ROPE // 2, 2).contiguous())
        z = z * (w if z.dim() == 2 else w[:, None])
        return torch.cat([z.real, z.imag], -1) if layout == "half" else torch.view_as_real(z).flatten(-2)

    def scatter(cache, rows):
        out = cache.double().clone()
        out.view(-1, rows.shape[1])[slots[live]] = rows[live]
        return out

    lay = case["layout"]
    latent, rotary = (st["latent"], st["rotary"]) if case["split"] else st["rows"].split((NOPE, ROPE), 1)
    latent, rotary = latent.double(), turn(rotary, lay)
    keys = torch.cat([turn(st["k_idx"][:, :ROPE], "half"), st["k_idx"][:, ROPE:].double()], 1)
    if case["bits"] == 4:
        first = torch.cat([_nearest4(latent), rotary], 1) * live[:, None]
    else:
        first = scatter(st["cache"], torch.cat([latent, rotary], 1))
    out = [first, scatter(st["idx_cache"], keys)]
    if case["H"]:
        q, qi = st["q"][:, :, NOPE:].double().clone(), st["q_idx_out"].double().clone()
        q[live] = turn(st["q_proj"][:, :, 128:], lay)[live]
        qi[live] = torch.cat([turn(st["q_idx"][..., :ROPE], "half"), st["q_idx"][..., ROPE:].double()], -1)[live]
        out += [q, qi]
    return out


def _nearest4(x):
    g = x.reshape(-1, GROUP)
    e4m3 = torch.tensor([m * 2.0 ** -9 for m in range(8)] +
                        [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1],
                        dtype=torch.float64, device=DEV)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)

    def nearest(v, values):
        hi = torch.searchsorted(values, v.contiguous()).clamp(1, values.numel() - 1)
        low, high = v - values[hi - 1], values[hi] - v
        return torch.where((high < low) | ((high == low) & (hi % 2 == 0)), hi, hi - 1)  # ties: the even code

    s = e4m3[nearest(g.abs().amax(1) / 6.0, e4m3)][:, None]
    t = g.abs() / torch.where(s > 0, s, torch.ones_like(s))
    v = torch.where(s > 0, grid[nearest(t, grid)], torch.zeros_like(t)) * s
    return torch.copysign(v, g).reshape(x.shape)


def _exact_prefix(st):
    """Request by request over its own page table: causal attention over all of its positions."""
    ps, H = st["case"]["ps"], st["case"]["H"]
    _, _, q_lens, seq, table = st["lens"]
    outs, lses, t0 = [], [], 0
    for n, kv, pages in zip(q_lens.tolist(), seq.tolist(), table):
        k = st["kv"][torch.tensor(np.array(pages), device=DEV)].reshape(-1, DK)[:kv].double()
        for a in range(0, n, 64):
            b = min(n, a + 64)
            z = (st["q"][t0 + a: t0 + b].double() @ k.T) * SM_SCALE
            last = torch.arange(kv - n + a, kv - n + b, device=DEV)
            z = z.masked_fill(torch.arange(kv, device=DEV) > last[:, None, None], -math.inf)
            l = torch.logsumexp(z, -1)
            outs.append(torch.exp(z - l[..., None]) @ k[:, :NOPE])
            lses.append(l)
        t0 += n
    return torch.cat(outs), torch.cat(lses)
