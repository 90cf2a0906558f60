"""Plain float64 oracle of the attention-side operators: rotary positions with several axes, the
8-bit paged cache, attention over it.  Written from the formulas; loops over sequences and heads."""
from __future__ import annotations

import numpy as np

SCALE_FLOOR = np.float32(2.0 ** -64)
GROW = np.float32(1.25)


# ------------------------------------------------------------------------------------------- rope
def rope_matrix_angles(dims, freqs, positions) -> np.ndarray:
    """Angles [tokens, pairs] from float32 positions [tokens, axes] and frequencies, in 64 bits."""
    out, at = [], 0
    for a, d in enumerate(dims):
        f = np.asarray(freqs[at:at + d // 2], np.float64)
        out.append(np.asarray(positions, np.float64)[:, a:a + 1] * f[None, :])
        at += d // 2
    return np.concatenate(out, axis=1)


def rope_pairs(dims, layout: str):
    """Entries (first, second) of each pair."""
    n = sum(dims) // 2
    i = np.arange(n)
    return (2 * i, 2 * i + 1) if layout == "pairs" else (i, i + n)


def rope(x: np.ndarray, dims, freqs, positions, layout: str, inverse: bool = False) -> np.ndarray:
    """x [tokens, heads, head_dim] turned; positions [tokens, axes]."""
    t = rope_matrix_angles(dims, freqs, positions)[:, None, :]
    c, s = np.cos(t), np.sin(t) * (-1.0 if inverse else 1.0)
    a, b = rope_pairs(dims, layout)
    y = np.array(x, np.float64)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


# ------------------------------------------------------------------------------------------ cache
def quantise(x: np.ndarray, inv: np.float32) -> np.ndarray:
    """Codes of float32 x: rint(x inv) within +-127, NaN as 0."""
    with np.errstate(invalid="ignore", over="ignore"):
        c = np.clip(np.rint(x.astype(np.float32) * inv), -127, 127)
    return np.where(np.isnan(x), 0, c).astype(np.int8)


def append_block(codes: np.ndarray, scale, held: int, x: np.ndarray):
    """One (block, head): codes int8 [page, d] with `held` tokens, new rows x float32 [n, d] behind them.
    Returns (codes, scale).  Every operation is a single float32 one, as the definition says."""
    f = np.float32
    finite = np.abs(x[np.isfinite(x)])
    most = f(finite.max()) if finite.size else f(0)
    need = max(most * (f(1) / f(127)), SCALE_FLOOR)
    codes = codes.copy()
    if held and need <= f(scale):
        s = f(scale)
    else:
        s = max(need, GROW * f(scale)) if held else need
        if held:
            codes[:held] = quantise(codes[:held].astype(np.float32), f(scale) / s)
    codes[held:held + len(x)] = quantise(x, f(1) / s)
    return codes, s


def kv_append(k_codes, v_codes, k_scales, v_scales, table, start, new_k, new_v) -> None:
    """In place; table [batch][pages], new_k / new_v: a float32 [n, heads, d] for each sequence."""
    pages, heads, page, _ = k_codes.shape
    for b, (nk, nv) in enumerate(zip(new_k, new_v)):
        at, n = int(start[b]), len(nk)
        done = 0
        while done < n:
            p, held = divmod(at + done, page)
            m = min(page - held, n - done)
            pg = int(table[b][p]) if p < len(table[b]) else -1
            if 0 <= pg < pages:
                for h in range(heads):
                    k_codes[pg, h], k_scales[pg, h] = append_block(k_codes[pg, h], k_scales[pg, h], held, nk[done:done + m, h])
                    c, v_scales[pg, h] = append_block(v_codes[pg, h].T, v_scales[pg, h], held, nv[done:done + m, h])
                    v_codes[pg, h] = c.T
            done += m


def kv_tokens(codes, scales, pages_of_seq, n: int, turned: bool) -> np.ndarray:
    """Tokens 0 .. n-1 of a sequence, float64 [n, heads, d]; NaN for a block that is absent."""
    num, heads = codes.shape[:2]
    page, d = (codes.shape[3], codes.shape[2]) if turned else (codes.shape[2], codes.shape[3])
    out = np.full((n, heads, d), np.nan)
    for t0 in range(0, n, page):
        pg = int(pages_of_seq[t0 // page]) if t0 // page < len(pages_of_seq) else -1
        if 0 <= pg < num:
            c = codes[pg].astype(np.float64)
            c = (c.transpose(0, 2, 1) if turned else c) * scales[pg].astype(np.float64)[:, None, None]
            m = min(page, n - t0)
            out[t0:t0 + m] = c[:, :m].transpose(1, 0, 2)
    return out


# -------------------------------------------------------------------------------------- attention
def visible(length: int, n: int, causal_block: int, window: int) -> tuple[np.ndarray, np.ndarray]:
    """(lo, hi) of each of the n queries that end a sequence of `length` tokens."""
    pos = length - n + np.arange(n)
    hi = np.full(n, length)
    if causal_block:
        hi = np.where(pos < 0, 0, np.minimum(length, (pos // causal_block + 1) * causal_block))
    lo = np.maximum(0, hi - window) if window else np.zeros(n, int)
    return lo, hi


def attention(q, k, v, causal_block: int, window: int, scale: float):
    """One sequence: q [n, heads, d] float64, k and v [length, kv_heads, d] (NaN: absent tokens).
    Returns (o, lse, spread): spread[n, heads, 3] holds sum_j P_j |v_j| 's largest entry, the largest
    |score|, and the largest P_j times the largest |v| entry, from which error bounds are made."""
    n, heads, d = q.shape
    length, kv_heads, _ = k.shape
    g = heads // kv_heads
    lo, hi = visible(length, n, causal_block, window)
    j = np.arange(length)
    seen = (j[None] >= lo[:, None]) & (j[None] < hi[:, None]) & ~np.isnan(k[:, 0, 0])[None]
    o, lse, spread = np.zeros(q.shape), np.full((n, heads), -np.inf), np.zeros((n, heads, 3))
    some = seen.any(1)
    for h in range(heads):
        kk, vv = np.nan_to_num(k[:, h // g]), np.nan_to_num(v[:, h // g])
        s = np.where(seen, scale * (q[:, h] @ kk.T), -np.inf)
        top = np.where(some, s.max(1, initial=-np.inf), 0.0)
        p = np.exp(s - top[:, None])
        z = p.sum(1)
        p = p / np.where(some, z, 1.0)[:, None]
        o[:, h] = p @ vv
        lse[some, h] = top[some] + np.log(z[some])
        spread[:, h, 0] = (p @ np.abs(vv)).max(1, initial=0.0)
        mag = np.abs(scale) * (np.abs(q[:, h]) @ np.abs(kk).T)
        spread[:, h, 1] = np.where(seen, mag, 0.0).max(1, initial=0.0)
        spread[:, h, 2] = (p * np.abs(vv).max(1, initial=0.0)[None]).max(1, initial=0.0)
    return o, lse, spread
