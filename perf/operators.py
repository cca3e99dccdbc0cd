"""Measured cases of the operators around the sparse-attention path: a serving step's tables, the rotary
positions, the 4-bit latent cache (write, read, sparse attention) and windowed attention with sinks.

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
IDX_HEADS, IDX_DIM = 32, 128  # indexer queries and keys
GROUP = 16                    # 4-bit codes that share a scale
ROW4 = NOPE // 2 + NOPE // GROUP + 2 * ROPE  # bytes of a 4-bit cache row
SM_SCALE = 1.0 / math.sqrt(192.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's bookkeeping: 64 requests, one new token each
        dict(name="tables_decode", op="tables", S=64, q_max=1, q_total=64, kv_max=131072, ps=64),
        # a large mixed step: decodes beside chunked prefills, tables of half a million pages
        dict(name="tables_mixed", op="tables", S=2047, q_max=4096, q_total=60000, kv_max=32768, ps=64),
        # one decode batch's queries, keys, indexer queries and indexer keys
        dict(name="rope_decode", op="rope", T=32, H=128, dtype="bf16", layout="interleaved", yarn=True, inverse=False,
             max_pos=131072),
        # the same four tensors of a prefill of 8192 tokens
        dict(name="rope_prefill", op="rope", T=8192, H=128, dtype="bf16", layout="interleaved", yarn=True,
             inverse=False, max_pos=131072),
        # gradients of rotated tensors in fp32, halves layout, a ragged number of tokens
        dict(name="rope_gradient", op="rope", T=4001, H=24, dtype="fp32", layout="half", yarn=False, inverse=True,
             max_pos=16384),
        # a decode step's new rows into the 4-bit cache and back
        dict(name="q4_rows_decode", op="q4_rows", S=48, q_max=1, kv_max=8192, ps=64),
        # four extends of 4096 tokens
        dict(name="q4_rows_extend", op="q4_rows", S=4, q_max=4096, kv_max=32768, ps=64),
        # the smallest attention: one request of 1024 tokens, 16 heads, 256 selected tokens
        dict(name="q4_attend_tiny", op="q4_attend", S=1, H=16, kv_min=1024, kv_max=1024, K=256, unit="token", ps=64,
             empty=False),
        # batched decode, 2048 selected tokens a request
        dict(name="q4_attend_batched", op="q4_attend", S=32, H=128, kv_min=4096, kv_max=8192, K=2048, unit="token",
             ps=64, empty=False),
        # longer contexts, a budget of 32 pages a request
        dict(name="q4_attend_pages", op="q4_attend", S=64, H=128, kv_min=16384, kv_max=32768, K=32, unit="page",
             ps=64, empty=True),
        # decode of layers without an indexer: the last 4096 positions and the first 64
        dict(name="window_decode", op="window", S=32, q_total=32, H=128, kv_max=16384, window=4096, sinks=64, ps=64),
        # extends of layers without an indexer, ragged, a short window and four sinks
        dict(name="window_extend", op="window", S=3, q_total=2049, H=128, kv_max=8192, window=1024, sinks=4, ps=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "q4_rows", "q4_attend", "window"])
    ps = rng.choice([32, 64, 128])
    if op == "tables":
        S = _log_int(rng, 1, 2047)
        return dict(op=op, S=S, q_max=rng.choice([1, 37, 4096]), q_total=_log_int(rng, S, max(S, 60000)),
                    kv_max=_log_int(rng, 4200, 32768), ps=ps)
    if op == "rope":
        dtype = rng.choice(["bf16", "fp32"])
        return dict(op=op, T=_log_int(rng, 1, 8192 if dtype == "bf16" else 4096), H=_log_int(rng, 1, 128 if dtype == "bf16" else 64),
                    dtype=dtype, layout=rng.choice(["interleaved", "half"]), yarn=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, max_pos=_log_int(rng, 8192, 131072))
    if op == "q4_rows":
        S = _log_int(rng, 1, 48)
        return dict(op=op, S=S, q_max=_log_int(rng, 1, max(1, 16000 // S)), kv_max=_log_int(rng, 16384, 32768), ps=ps)
    if op == "q4_attend":
        kv_max = _log_int(rng, 64, 16384)
        unit = rng.choice(["token", "page"])
        K = _log_int(rng, 1, 2048) if unit == "token" else _log_int(rng, 1, 2048 // ps)
        return dict(op=op, S=_log_int(rng, 1, 48), H=_log_int(rng, 1, 128), kv_min=_log_int(rng, 1, kv_max),
                    kv_max=kv_max, K=K, unit=unit, ps=ps, empty=rng.random() < 0.5)
    S = _log_int(rng, 1, 24)
    return dict(op=op, S=S, q_total=_log_int(rng, S, max(S, 1000)), H=_log_int(rng, 1, 128),
                kv_max=_log_int(rng, 1100, 16384), window=_log_int(rng, 1, 1900), sinks=rng.choice([0, 1, 4, 37, 128]),
                ps=ps)


# ------------------------------------------------------------ 4-bit format
# A row: 256 bytes of e2m1 codes, 32 e4m3 scales (one per 16 dims), 64 bf16 rotary dims. Dim 8*w + j sits in
# 32-bit word w; the even dims of a word are its nibbles 0..3, the odd ones its nibbles 4..7.
NIBBLE = (0, 4, 1, 5, 2, 6, 3, 7)  # nibble of dim j of a word
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(rows):
    """bf16 rows [N, 576] -> codes 0..15 [N, 512] (uint8) and scales [N, 32] (e4m3 values in fp32)."""
    x = rows[:, :NOPE].float().view(-1, NOPE // GROUP, GROUP)
    amax = x.abs().amax(-1)
    s = (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    s = torch.where(torch.isfinite(amax), s, torch.full_like(s, float("nan")))
    t = torch.where(s[..., None] > 0, x.abs() / s[..., None], torch.zeros_like(x))
    # to the nearest code, ties to the code with the even mantissa
    code = ((t > 0.25).to(torch.uint8) + (t >= 0.75).to(torch.uint8) + (t > 1.25).to(torch.uint8)
            + (t >= 1.75).to(torch.uint8) + (t > 2.5).to(torch.uint8) + (t >= 3.5).to(torch.uint8)
            + (t > 5.0).to(torch.uint8))
    return (code | (torch.signbit(x).to(torch.uint8) << 3)).view(-1, NOPE), s


def _pack(rows):
    code, s = _quantise(rows)
    w = code.view(-1, NOPE // 8, 8)[:, :, [0, 2, 4, 6, 1, 3, 5, 7]]  # nibble order
    by = (w[:, :, 0::2] | (w[:, :, 1::2] << 4)).reshape(-1, NOPE // 2)
    sc = s.to(torch.float8_e4m3fn).view(torch.uint8)
    rope = rows[:, NOPE:].contiguous().view(torch.uint8).view(-1, 2 * ROPE)
    return torch.cat([by, sc, rope], 1)


def _unpack(b):
    """cache rows [N, 416] uint8 -> the values they stand for, fp32 [N, 576]"""
    by = b[:, : NOPE // 2].view(-1, NOPE // 8, 4)
    nib = torch.stack([by & 15, by >> 4], -1).view(-1, NOPE // 8, 8)[:, :, list(NIBBLE)].reshape(-1, NOPE)
    mag = torch.tensor(E2M1, device=b.device)[(nib & 7).long()]
    v = torch.where(nib >= 8, -mag, mag)
    s = b[:, NOPE // 2: NOPE // 2 + NOPE // GROUP].contiguous().view(torch.float8_e4m3fn).float()
    v = (v.view(-1, NOPE // GROUP, GROUP) * s[..., None]).view(-1, NOPE)
    rope = b[:, NOPE // 2 + NOPE // GROUP:].contiguous().view(torch.bfloat16).float()
    return torch.cat([v, rope], 1)


# ------------------------------------------------------------------ inputs
def _lens(case):
    """q_lens and seq_lens of a case: the same lengths for every seed, which orders them anew, so that sizes and
    work do not depend on it."""
    rng, S, kv_max = np.random.default_rng(7), case["S"], case["kv_max"]
    q = np.ones(S, np.int64)
    if case["op"] == "tables" and case["q_max"] > 1:
        q = np.minimum(case["q_max"], 1 + rng.integers(0, max(1, 2 * case["q_total"] // S), S))
        if S > 1:
            q[rng.random(S) < 0.5] = 1   # decodes beside chunks
            q[rng.random(S) < 0.02] = 0  # requests that pause
    elif case["op"] == "q4_rows" and case["q_max"] > 1:
        q = rng.integers((case["q_max"] + 1) // 2, case["q_max"] + 1, S)
        q[0] = case["q_max"]
    elif case["op"] == "window" and case["q_total"] > S:
        q += rng.multinomial(case["q_total"] - S, rng.dirichlet(np.ones(S)))
    q = np.minimum(q, kv_max)
    if case["op"] == "q4_attend":
        return q, rng.integers(case["kv_min"], kv_max + 1, S)
    return q, np.minimum(q + rng.integers(0, kv_max, S), kv_max)


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _ragged(q, seq, ps, rng, spare=3):
    pages = -(-seq // ps)
    cu_q = np.concatenate([[0], np.cumsum(q)])
    cu_p = np.concatenate([[0], np.cumsum(pages)])
    P = int(cu_p[-1]) + spare
    return dict(seq_lens=_ints(seq), cu_q_lens=_ints(cu_q), cu_kv_lens=_ints(cu_p * ps),
                page_indices=_ints(rng.permutation(P)[: int(cu_p[-1])]), P=P, T=int(cu_q[-1]), S=len(q))


def _meta(st):
    return st["seq_lens"], st["cu_q_lens"], st["cu_kv_lens"], st["page_indices"]


def _randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=dtype)


def _freqs(dim, yarn, base=10000.0, factor=40.0, orig=4096, beta_fast=32.0, beta_slow=1.0):
    """Radians per position of each pair, 64 bits; yarn: pairs that turn often keep their frequency, pairs that
    turn rarely are slowed by `factor`, a linear ramp between."""
    f = base ** (-np.arange(0, dim, 2, dtype=np.float64) / dim)
    if not yarn:
        return f, 1.0
    at = lambda turns: dim * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), dim - 1)
    keep = 1.0 - np.clip((np.arange(dim // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, st = case["op"], {"case": dict(case)}
    if op != "rope":
        q, seq = _lens(case)
        order = rng.permutation(len(q))
        q, seq = q[order], seq[order]
    if op == "tables":
        ps = case["ps"]
        old, new = -(-(seq - q) // ps), -(-seq // ps)
        width = -(-case["kv_max"] // ps) + 1
        ids = rng.permutation(int(new.sum()) + 17).astype(np.int32)
        bt = np.full((len(q), width), -1, np.int32)
        live = np.arange(width)[None, :] < old[:, None]
        bt[live] = ids[: int(old.sum())]
        st.update(q_lens=_ints(q), seq_lens=_ints(seq), block_table=_ints(bt), free=_ints(ids[int(old.sum()):]),
                  T=int(q.sum()) + 5, PTW=int(new.sum()) + 9)  # padded: a captured step's sizes stay the same
    elif op == "rope":
        T, H, dt = case["T"], case["H"], {"bf16": torch.bfloat16, "fp32": torch.float32}[case["dtype"]]
        start = rng.integers(0, case["max_pos"] - T // 2)
        pos = np.concatenate([np.arange(start, start + T - T // 2),
                              rng.integers(0, case["max_pos"], T // 2)])  # a prefill's run, then decode tokens
        f, mscale = _freqs(ROPE, case["yarn"])
        st.update(positions=_ints(pos), freqs=torch.from_numpy(f).to(DEV), scale=mscale,
                  proj=_randn(gen, T, H, 128 + ROPE, dtype=dt),        # [no rotation 128 | rotary 64] of a projection
                  k=_randn(gen, T, 1, DK, dtype=dt), q_idx=_randn(gen, T, IDX_HEADS, IDX_DIM, dtype=dt),
                  k_idx=_randn(gen, T, 1, IDX_DIM, dtype=dt), q=_randn(gen, T, H, DK, dtype=dt),
                  k_out=torch.empty(T, 1, DK, device=DEV, dtype=dt),
                  q_idx_out=torch.empty(T, IDX_HEADS, IDX_DIM, device=DEV, dtype=dt),
                  k_idx_out=torch.empty(T, 1, IDX_DIM, device=DEV, dtype=dt))
    elif op == "q4_rows":
        st.update(_ragged(q, seq, case["ps"], rng))
        rows = _randn(gen, st["T"], DK)
        rows[:, :NOPE] *= torch.exp(_randn(gen, st["T"], 1, dtype=torch.float32)).bfloat16()  # rows of unlike size
        seqs = np.repeat(np.arange(case["S"]), q)
        pos = np.concatenate([np.arange(a - b, a) for a, b in zip(seq, q)])
        ent = np.concatenate([[0], np.cumsum(-(-seq // case["ps"]))])[seqs] + pos // case["ps"]
        slots = st["page_indices"].cpu().numpy()[ent].astype(np.int64) * case["ps"] + pos % case["ps"]
        st.update(rows=rows, slots=_ints(slots), out=torch.empty(st["T"], DK, device=DEV, dtype=torch.bfloat16),
                  cache=torch.zeros(st["P"], case["ps"], ROW4, device=DEV, dtype=torch.uint8))
    elif op == "q4_attend":
        S, ps, K = case["S"], case["ps"], case["K"]
        st.update(_ragged(q, seq, ps, rng))
        pool = _pack(_randn(gen, 8192, DK))
        pick = torch.randint(0, 8192, (st["P"] * ps,), generator=gen, device=DEV)
        st["cache"] = pool[pick].view(st["P"], ps, ROW4)
        n = seq if case["unit"] == "token" else -(-seq // ps)
        sel = np.full((S, K), -1, np.int32)
        for s in range(S):
            m = min(K, int(n[s]))
            sel[s, :m] = np.sort(rng.permutation(int(n[s]))[:m])
        if case["empty"]:
            sel[rng.integers(0, S)] = -1  # a row that selects nothing
            sel[:, 0] = -1
        st.update(sel=_ints(sel), q=_randn(gen, S, case["H"], DK), seq_np=seq,
                  o=torch.empty(S, case["H"], NOPE, device=DEV, dtype=torch.bfloat16))
    else:
        st.update(_ragged(q, seq, case["ps"], rng))
        st.update(q=_randn(gen, st["T"], case["H"], DK), kv=_randn(gen, st["P"], case["ps"], DK), seq_np=seq,
                  o=torch.empty(st["T"], case["H"], NOPE, device=DEV, dtype=torch.bfloat16))
    return st


# ------------------------------------------------------------------- passes
def run(st):
    case = st["case"]
    return (_run_own if own else _run_plain)(case["op"], case, st)


def _run_own(op, case, st):
    import deepseek_sparse_attention_score_gb300 as dsa
    if op == "tables":
        t = dsa.dsa_build_page_tables(st["q_lens"], st["seq_lens"], st["block_table"], st["free"], T=st["T"],
                                      PTW=st["PTW"], ps=case["ps"])
        return dict(block_table=st["block_table"], cu_q_lens=t.cu_q_lens, cu_kv_lens=t.cu_kv_lens,
                    page_indices=t.page_indices, token_seq=t.token_seq, positions=t.positions, slots=t.slots,
                    n_taken=t.n_taken)
    if op == "rope":
        R, lay = dsa.RopeTarget, case["layout"]
        dsa.dsa_rope([R(st["proj"][:, :, 128:], st["q"][:, :, NOPE:], layout=lay, scale=st["scale"]),
                      R(st["k"], st["k_out"], rot_off=NOPE, layout=lay, rot_dim=ROPE, scale=st["scale"]),
                      R(st["q_idx"], st["q_idx_out"], rot_dim=ROPE, layout="half"),
                      R(st["k_idx"], st["k_idx_out"], rot_dim=ROPE, layout="half")],
                     st["positions"], st["freqs"], inverse=case["inverse"])
        return st["q"][:, :, NOPE:], st["k_out"], st["q_idx_out"], st["k_idx_out"]
    if op == "q4_rows":
        dsa.dsa_q4_write_back(st["rows"], st["cache"], *_meta(st))
        return dsa.dsa_q4_read_rows(st["cache"], st["slots"], out=st["out"])
    if op == "q4_attend":
        return dsa.dsa_sparse_mla_decode_q4(st["q"], st["cache"], *_meta(st), st["sel"],
                                            unit=1 if case["unit"] == "token" else case["ps"], sm_scale=SM_SCALE,
                                            o=st["o"], want_lse=True)
    return dsa.dsa_window_mla(st["q"], st["kv"], *_meta(st), max_kv=case["kv_max"], sliding_window=case["window"],
                              num_sinks=case["sinks"], sm_scale=SM_SCALE, o=st["o"], want_lse=True)


def _run_plain(op, case, st):
    if op == "tables":
        return _plain_tables(case, st)
    if op == "rope":
        return _plain_rope(case, st)
    if op == "q4_rows":
        flat = st["cache"].view(-1, ROW4)
        flat[st["slots"].long()] = _pack(st["rows"])
        return _unpack(flat[st["slots"].long()]).bfloat16()
    return _plain_attend(op, case, st)


def _excl(x):
    return torch.cumsum(x, 0) - x


def _plain_tables(case, st):
    ps, T, PTW, bt, free = case["ps"], st["T"], st["PTW"], st["block_table"], st["free"]
    q, seq = st["q_lens"].long(), st["seq_lens"].long()
    old, new = (seq - q + ps - 1) // ps, (seq + ps - 1) // ps
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    cu_q, cu_p = torch.cat([zero, torch.cumsum(q, 0)]), torch.cat([zero, torch.cumsum(new, 0)])
    col = torch.arange(bt.shape[1], device=DEV)[None, :]
    at = _excl(new - old)[:, None] + col - old[:, None]
    grow = (col >= old[:, None]) & (col < new[:, None])
    bt.copy_(torch.where(grow, free[at.clamp(0, free.numel() - 1)], bt))
    e = torch.arange(PTW, device=DEV)
    s = torch.searchsorted(cu_p[1:], e, right=True).clamp(max=q.numel() - 1)
    pages = torch.where(e < cu_p[-1], bt[s, (e - cu_p[s]).clamp(0, bt.shape[1] - 1)].long(), -1)
    t = torch.arange(T, device=DEV)
    s = torch.searchsorted(cu_q[1:], t, right=True).clamp(max=q.numel() - 1)
    live = t < cu_q[-1]
    pos = torch.where(live, seq[s] - q[s] + t - cu_q[s], 0)
    slot = bt[s, (pos // ps).clamp(0, bt.shape[1] - 1)].long() * ps + pos % ps
    i32 = lambda x: x.to(torch.int32)
    return dict(block_table=bt, cu_q_lens=i32(cu_q), cu_kv_lens=i32(cu_p * ps), page_indices=i32(pages),
                token_seq=i32(torch.where(live, s, -1)), positions=i32(torch.where(live, pos, -1)),
                slots=i32(torch.where(live, slot, -1)), n_taken=i32((new - old).sum().view(1)))


def _plain_rope(case, st):
    ang = st["positions"].double()[:, None, None] * st["freqs"]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    if case["inverse"]:
        sin = -sin

    def turn(x, out, off, layout, scale):
        out.copy_(x)
        r = x[:, :, off: off + ROPE].float()
        if layout == "half":
            a, b = r[..., : ROPE // 2], r[..., ROPE // 2:]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        out[:, :, off: off + ROPE] = (y * scale).to(out.dtype)
        return out

    lay, sc = case["layout"], st["scale"]
    return (turn(st["proj"][:, :, 128:], st["q"][:, :, NOPE:], 0, lay, sc), turn(st["k"], st["k_out"], NOPE, lay, sc),
            turn(st["q_idx"], st["q_idx_out"], 0, "half", 1.0), turn(st["k_idx"], st["k_idx_out"], 0, "half", 1.0))


def _positions(op, case, st, t0, t1):
    """Key positions [t, n] (-1: none) and requests of tokens t0 .. t1-1."""
    tok = torch.arange(t0, t1, device=DEV)
    seq, cu_q = st["seq_lens"].long(), st["cu_q_lens"].long()
    s = torch.searchsorted(cu_q[1:].contiguous(), tok, right=True)
    pos = (seq[s] - (cu_q[s + 1] - cu_q[s]) + tok - cu_q[s])[:, None]
    if op == "window":
        W, n0 = case["window"], case["sinks"]
        first = torch.arange(n0, device=DEV)[None, :]
        last = pos - W + 1 + torch.arange(W, device=DEV)[None, :]
        j = torch.cat([torch.where(first <= pos - W, first, -1), last.clamp(min=-1)], 1)
    else:
        j = st["sel"][t0:t1].long()
        if case["unit"] == "page":
            j = torch.where(j[:, :, None] >= 0, j[:, :, None] * case["ps"] + torch.arange(case["ps"], device=DEV), -1)
            j = j.flatten(1)
    return torch.where(j <= pos, j, -1), s


def _plain_attend(op, case, st):
    T, H, ps = st["T"], case["H"], case["ps"]
    n = case["window"] + case["sinks"] if op == "window" else case["K"] * (ps if case["unit"] == "page" else 1)
    step = max(1, (1 << 29) // (n * DK))
    base, table = st["cu_kv_lens"].long() // ps, st["page_indices"].long()
    rows = st["kv"].view(-1, DK) if op == "window" else st["cache"].view(-1, ROW4)
    lse = torch.empty(T, H, device=DEV)
    for t0 in range(0, T, step):
        t1 = min(T, t0 + step)
        j, s = _positions(op, case, st, t0, t1)
        ok = j >= 0
        jj = j.clamp(min=0)
        at = (table[base[s][:, None] + jj // ps] * ps + jj % ps).flatten()
        k = (rows[at].float() if op == "window" else _unpack(rows[at])).view(t1 - t0, n, DK)
        z = torch.bmm(st["q"][t0:t1].float(), k.transpose(1, 2)) * SM_SCALE
        z = torch.where(ok[:, None, :], z, -math.inf)
        m = z.amax(-1, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        p = torch.exp(z - m)
        total = p.sum(-1, keepdim=True)
        o = torch.bmm(p, k[:, :, :NOPE]) / torch.where(total > 0, total, torch.ones_like(total))
        st["o"][t0:t1] = o.bfloat16()
        lse[t0:t1] = (m + torch.log(total))[..., 0]
    return st["o"], lse


# --------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "rope":
        T, H, b = case["T"], case["H"], 2 if case["dtype"] == "bf16" else 4
        elems = T * (H * ROPE + DK + (IDX_HEADS + 1) * IDX_DIM)
        return {"bytes": 2 * b * elems + 4 * T + 4 * ROPE, "flops": 3 * T * ROPE * (H + IDX_HEADS + 2)}
    q, seq = _lens(case)
    T, S = int(q.sum()), len(q)
    if op == "tables":
        ps = case["ps"]
        old, new = -(-(seq - q) // ps), -(-seq // ps)
        ints = 4 * S + 2 + int(old.sum()) + int(new.sum()) + 2 * int((new - old).sum()) + 3 * T
        return {"bytes": 4 * ints, "flops": 0}
    if op == "q4_rows":
        return {"bytes": T * (2 * 2 * DK + 2 * ROW4 + 4), "flops": 4 * T * NOPE}
    H = case["H"]
    io = T * H * (2 * (DK + NOPE) + 4)  # queries, outputs and their log-sums
    if op == "q4_attend":
        keys = int(np.minimum(seq, case["K"] * (1 if case["unit"] == "token" else case["ps"])).sum())
        return {"bytes": keys * ROW4 + io + 4 * S * case["K"], "flops": 2 * keys * H * (DK + NOPE)}
    W, n0 = case["window"], case["sinks"]
    pos = np.concatenate([np.arange(b - a, b) for a, b in zip(q, seq)])
    pairs = int((np.minimum(pos + 1, W) + np.minimum(n0, np.maximum(pos - W + 1, 0))).sum())
    rows = int((np.minimum(seq, W + q - 1) + np.minimum(n0, np.maximum(seq - q - W + 1, 0))).sum())
    return {"bytes": rows * 2 * DK + io, "flops": 2 * pairs * H * (DK + NOPE)}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """The operators' definitions in 64 bits."""
    st = prepare(case, seed)
    return {"tables": _exact_tables, "rope": _exact_rope, "q4_rows": _exact_rows}.get(case["op"], _exact_attend)(case, st)


def _exact_tables(case, st):
    ps = case["ps"]
    q, seq = st["q_lens"].cpu().numpy().tolist(), st["seq_lens"].cpu().numpy().tolist()
    bt, free = st["block_table"].cpu().numpy().copy(), st["free"].cpu().numpy()
    cu_q, cu_kv, pages, tok = [0], [0], [], []
    taken = 0
    for s, (n, kv) in enumerate(zip(q, seq)):
        have, need = math.ceil((kv - n) / ps), math.ceil(kv / ps)
        bt[s, have:need] = free[taken: taken + need - have]
        taken += need - have
        cu_q.append(cu_q[-1] + n)
        cu_kv.append(cu_kv[-1] + need * ps)
        pages.append(bt[s, :need])
        for pos in range(kv - n, kv):
            tok.append((s, pos, int(bt[s, pos // ps]) * ps + pos % ps))
    pad = lambda a, n: np.concatenate([a, np.full(n - len(a), -1)]).astype(np.int64)
    tok = np.array(tok, np.int64).reshape(-1, 3)
    return dict(block_table=bt.astype(np.int64), cu_q_lens=np.array(cu_q), cu_kv_lens=np.array(cu_kv),
                page_indices=pad(np.concatenate(pages), st["PTW"]), token_seq=pad(tok[:, 0], st["T"]),
                positions=pad(tok[:, 1], st["T"]), slots=pad(tok[:, 2], st["T"]), n_taken=np.array([taken]))


def _exact_rope(case, st):
    """Each pair is a complex number, turned by exp(i * angle)."""
    ang = st["positions"].double()[:, None] * st["freqs"][None, :]
    w = torch.polar(torch.ones_like(ang), -ang if case["inverse"] else ang)[:, None, :]

    def turn(x, off, layout, scale):
        y = x.double().clone()
        r = y[:, :, off: off + ROPE]
        z = r.reshape(*r.shape[:2], 2, ROPE // 2).transpose(2, 3) if layout == "half" else r.reshape(*r.shape[:2], ROPE // 2, 2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * w) * scale
        y[:, :, off: off + ROPE] = (z.transpose(2, 3) if layout == "half" else z).reshape(*r.shape)
        return y

    lay, sc = case["layout"], st["scale"]
    return (turn(st["proj"][:, :, 128:], 0, lay, sc), turn(st["k"], NOPE, lay, sc), turn(st["q_idx"], 0, "half", 1.0),
            turn(st["k_idx"], 0, "half", 1.0))


def _exact_rows(case, st):
    """The nearest value of the grid, by distance; the scale by a search of the e4m3 values."""
    x = st["rows"].double()
    g = x[:, :NOPE].reshape(-1, GROUP)
    e4m3 = torch.tensor(sorted({m * 2.0 ** -9 for m in range(8)} | {(1 + m / 8) * 2.0 ** e for e in range(-6, 9)
                                                                   for m in range(8)} - {480.0}),
                        dtype=torch.float64, device=DEV)

    def nearest(v, grid):
        hi = torch.searchsorted(grid, v.contiguous()).clamp(1, grid.numel() - 1)
        lo = hi - 1
        dl, dh = v - grid[lo], grid[hi] - v
        return torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)  # ties: the even code

    s = e4m3[nearest(g.abs().amax(1) / 6.0, e4m3)]
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    t = g.abs() / torch.where(s > 0, s, torch.ones_like(s))[:, None]
    v = torch.where(s[:, None] > 0, grid[nearest(t, grid)], torch.zeros_like(t)) * s[:, None]
    return torch.cat([torch.copysign(v, g).reshape(-1, NOPE), x[:, NOPE:]], 1)


def _exact_attend(case, st):
    """Token by token over explicit key lists, keys in 64 bits, softmax about the row's own maximum."""
    window, ps, H = case["op"] == "window", case["ps"], case["H"]
    cu_q, table = st["cu_q_lens"].tolist(), st["page_indices"].long()
    base = (st["cu_kv_lens"] // ps).tolist()
    sel = None if window else st["sel"].cpu().numpy()
    out = torch.zeros(st["T"], H, NOPE, dtype=torch.float64, device=DEV)
    lse = torch.full((st["T"], H), -math.inf, dtype=torch.float64, device=DEV)
    for s in range(st["S"]):
        n = int(st["seq_np"][s])
        need = torch.arange(n, device=DEV)
        rows = table[base[s] + need // ps] * ps + need % ps
        if window:
            kv = st["kv"].view(-1, DK)[rows].double()
        for t in range(cu_q[s], cu_q[s + 1]):
            pos = n - cu_q[s + 1] + t
            if window:
                j = torch.arange(pos + 1, device=DEV)
                lo = max(0, pos - case["window"] + 1)
                k = torch.cat([kv[: min(case["sinks"], lo)], kv[lo: pos + 1]])
            else:
                ids = sel[t][sel[t] >= 0].astype(np.int64)
                if case["unit"] == "page":
                    ids = (ids[:, None] * ps + np.arange(ps)).reshape(-1)
                ids = ids[ids <= pos]
                if not len(ids):
                    continue
                k = _unpack64(st["cache"].view(-1, ROW4)[rows[torch.from_numpy(ids).to(DEV)]])
            z = st["q"][t].double() @ k.T * SM_SCALE
            lse[t] = torch.logsumexp(z, 1)
            out[t] = torch.exp(z - lse[t][:, None]) @ k[:, :NOPE]
    return out, lse


def _unpack64(b):
    """Cache rows read word by word, in 64 bits."""
    w = b[:, : NOPE // 2].contiguous().view(torch.int32).long()
    v = torch.empty(b.shape[0], NOPE, dtype=torch.float64, device=b.device)
    grid = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=b.device)
    for d in range(8):
        nibble = d // 2 + 4 * (d % 2)
        v[:, d::8] = grid[(w >> (4 * nibble)) & 15]
    sc = b[:, NOPE // 2: NOPE // 2 + NOPE // GROUP].long()
    e, m = (sc >> 3) & 15, (sc & 7).double()
    s = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    v *= s.repeat_interleave(GROUP, 1)
    rope = b[:, NOPE // 2 + NOPE // GROUP:].contiguous().view(torch.bfloat16).double()
    return torch.cat([v, rope], 1)
