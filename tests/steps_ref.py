"""Plain 64-bit references of the operators around the attention (page
tables, rotary positions, the 4-bit cache, attention with element-wise error
bounds), for the tests. Python and numpy only, one row at a time."""
import math

import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
# e4m3 values of the codes 0 .. 126
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])
BF16_HALF = 2.0 ** -8  # a rounding to bf16: torch.finfo(torch.bfloat16).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------- tables
def page_tables(q_lens, seq_lens, block_table, free, T, PTW, ps):
    bt = block_table.copy()
    W = bt.shape[1]
    cu_q, cu_kv, pages, toks = [0], [0], [], []
    taken, bad = 0, False
    for s, (q, n) in enumerate(zip(q_lens.tolist(), seq_lens.tolist())):
        if q < 0 or n < q or n > W * ps:
            bad, q, n = True, 0, 0
        had, need = -(-(n - q) // ps), -(-n // ps)
        for j in range(need):
            pg = bt[s, j] if j < had else (free[taken + j - had] if taken + j - had < len(free) else -1)
            if j >= had and len(pages) < PTW:
                bt[s, j] = pg
            pages.append(pg)
        row = pages[len(pages) - need:]
        taken += need - had
        cu_q.append(cu_q[-1] + q)
        cu_kv.append(cu_kv[-1] + need * ps)
        for p in range(n - q, n):
            toks.append((s, p, row[p // ps] * ps + p % ps if row[p // ps] >= 0 else -1))
    bad = bad or len(toks) > T or len(pages) > PTW
    fit = lambda a, n: np.array((list(a) + [-1] * n)[:n], np.int32)
    out = dict(cu_q_lens=np.array(cu_q), cu_kv_lens=np.array(cu_kv), page_indices=fit(pages, PTW),
               token_seq=fit([t[0] for t in toks], T), positions=fit([t[1] for t in toks], T),
               slots=fit([t[2] for t in toks], T), n_taken=np.array([taken]))
    return out, bt, (0x2 if bad else 0) | (0x20 if taken > len(free) else 0)


# --------------------------------------------------------------------- rope
def rope(x, positions, freqs, off, layout, scale, inverse):
    """x fp64 [T, H, D] -> (y, bound factor |a| + |b| per rotated element)."""
    y, mag = x.copy(), np.zeros_like(x)
    n = len(freqs)
    i = np.arange(n)
    ca, cb = (off + 2 * i, off + 2 * i + 1) if layout == "interleaved" else (off + i, off + i + n)
    for t, p in enumerate(positions.tolist()):
        if p < 0:
            continue
        ang = p * freqs * (-1 if inverse else 1)
        a, b = x[t][:, ca], x[t][:, cb]
        y[t][:, ca] = scale * (a * np.cos(ang) - b * np.sin(ang))
        y[t][:, cb] = scale * (b * np.cos(ang) + a * np.sin(ang))
        mag[t][:, ca] = mag[t][:, cb] = abs(scale) * (np.abs(a) + np.abs(b))
    return y, mag


def rope_tol(y, mag, dtype):
    """Rounding of the result, and of the fp32 arithmetic: the angle's
    fraction of a turn (2^-25 turns, 2 pi radians each), sine and cosine, one
    product by the scale and three roundings come to less than 2^-20 of
    |a| + |b|."""
    return np.abs(y) * torch.finfo(dtype).eps / 2 + mag * 2.0 ** -20


# ------------------------------------------------------------- 4-bit cache
def _nearest_even(v, grid):
    hi = min(int(np.searchsorted(grid, v)), len(grid) - 1)
    lo = max(hi - 1, 0)
    dl, dh = v - grid[lo], grid[hi] - v
    return hi if dh < dl or (dh == dl and hi % 2 == 0) else lo


def q4_group(x):
    """16 values -> (codes 0..15, scale code)."""
    if not np.all(np.isfinite(x)):
        return np.zeros(16, np.uint8), 0x7F
    sc = _nearest_even(np.abs(x).max() / 6.0, E4M3)
    s = E4M3[sc]
    codes = [(_nearest_even(abs(v) / s, E2M1) if s > 0 else 0) | (8 if math.copysign(1, v) < 0 else 0) for v in x]
    return np.array(codes, np.uint8), sc


def q4_pack(rows):
    """bf16 tensor [N, 576] -> uint8 [N, 416]."""
    x = f64(rows)
    out = np.zeros((len(x), 416), np.uint8)
    out[:, 288:] = rows[:, 512:].contiguous().cpu().view(torch.uint8).numpy()
    for r in range(len(x)):
        code = np.zeros(512, np.uint8)
        for g in range(32):
            code[16 * g: 16 * g + 16], out[r, 256 + g] = q4_group(x[r, 16 * g: 16 * g + 16])
        for w in range(64):
            word = 0
            for j in range(8):
                word |= int(code[8 * w + j]) << (4 * (j // 2 + 4 * (j % 2)))
            out[r, 4 * w: 4 * w + 4] = np.frombuffer(np.uint32(word).tobytes(), np.uint8)
    return out


def q4_values(b):
    """uint8 [..., 416] -> fp64 [..., 576]."""
    b = np.ascontiguousarray(b)
    w = b[..., :256].copy().view("<u4")
    v = np.zeros(b.shape[:-1] + (512,))
    for j in range(8):
        c = (w >> np.uint32(4 * (j // 2 + 4 * (j % 2)))) & 15
        v[..., j::8] = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    sc = b[..., 256:288].astype(int)
    s = np.where(sc & 127 == 127, np.nan, E4M3[np.minimum(sc & 127, 126)]) * np.where(sc & 128, -1.0, 1.0)
    with np.errstate(invalid="ignore"):
        v = v * np.repeat(s, 16, -1)
    rope_cols = torch.from_numpy(b[..., 288:].copy()).view(torch.bfloat16).double().numpy()
    return np.concatenate([v, rope_cols], -1)


# ---------------------------------------------------------------- attention
def attend(q, keys_of, sm_scale, soft_cap=0.0, Dv=512):
    """q fp64 [T, H, Dk]; ``keys_of(t)`` -> fp64 [n, Dk] visible keys. Returns
    (o, lse, bound of |o|'s error, bound of lse's error).

    The kernel's roundings: P and the output to bf16 (2^-8 each, relative);
    the logits' dot products in fp32 (Dk additions that may truncate, 2^-23 of
    the sum of magnitudes each), the capped logit's tanh (2^-10), exp2 and the
    split merge (2^-18). An error d of a logit moves its weight by e^d - 1 <= 2 d (d <= 1)
    against the others'."""
    T, H, Dk = q.shape
    o, lse = np.zeros((T, H, Dv)), np.full((T, H), -np.inf)
    otol, ltol = np.zeros((T, H, Dv)), np.zeros((T, H))
    for t in range(T):
        k = keys_of(t)
        if not len(k):
            continue
        z = q[t] @ k.T * sm_scale
        d = Dk * 2.0 ** -23 * abs(sm_scale) * (np.abs(q[t]) @ np.abs(k).T).max(1)
        if soft_cap:
            z = soft_cap * np.tanh(z / soft_cap)
            d = d + np.abs(z).max(1) * 2.0 ** -10
        d = d + np.abs(z).max(1) * 2.0 ** -22 + 2.0 ** -18
        m = z.max(1, keepdims=True)
        p = np.exp(z - m)
        l = p.sum(1, keepdims=True)
        o[t] = p @ k[:, :Dv] / l
        lse[t] = (m + np.log(l))[:, 0]
        a = p @ np.abs(k[:, :Dv]) / l
        otol[t] = (BF16_HALF + 4 * d[:, None]) * a + BF16_HALF * np.abs(o[t])
        ltol[t] = 2 * d + 2.0 ** -20 * np.abs(lse[t])
    return o, lse, otol, ltol


def check_attend(o_gpu, lse_gpu, ref, what=""):
    o, lse, otol, ltol = ref
    go, gl = f64(o_gpu), f64(lse_gpu)
    assert np.isfinite(go).all(), f"{what}: {np.count_nonzero(~np.isfinite(go))} outputs are not finite"
    e = np.abs(go - o) - otol
    assert (e <= 0).all(), f"{what}: output past its bound at {np.argwhere(e > 0)[:4].tolist()}, worst {e.max():.3e}"
    none = np.isneginf(lse)
    assert np.array_equal(np.isneginf(gl), none) and (go[none] == 0).all(), f"{what}: rows without keys"
    e = np.abs(gl[~none] - lse[~none]) - ltol[~none]
    assert (e <= 0).all(), f"{what}: lse past its bound, worst {e.max(initial=0):.3e}"


def token_keys(rg, flat, positions_of):
    """keys_of for paged rows ``flat`` fp64 [P * ps, Dk] and the positions
    that token t attends to."""
    seq, pos = rg.token_seq(), rg.token_pos()

    def keys(t):
        j = np.asarray(positions_of(t), np.int64)
        j = j[(j >= 0) & (j <= pos[t])]
        ent = rg.cu_kv_lens[seq[t]] // rg.page_size + j // rg.page_size
        return flat[rg.page_indices[ent].astype(np.int64) * rg.page_size + j % rg.page_size]

    return keys
