"""Softmax-attention operators: plain, slow, fp64 CPU definitions (the oracle).

TEST INFRASTRUCTURE ONLY, as ``oracle.falcon``: no code shared with the CUDA
library.  Norm per head and rotary positions, the append to the paged 8-bit
cache, attention of one token over it, causal attention of packed prompts.
"""

from __future__ import annotations

import numpy as np

# value of every e4m3 code (0x7f and 0xff are NaN)
_c = np.arange(256)
_exp, _man = (_c >> 3) & 15, _c & 7
E4M3 = np.where(_exp == 0, _man / 8.0 * 2.0 ** -6, (1 + _man / 8.0) * 2.0 ** (_exp - 7.0))
E4M3 = np.where(_c & 127 == 127, np.nan, E4M3) * np.where(_c & 128, -1.0, 1.0)


def norm_rope(x, w, eps, positions, table, layout):
    """x [tokens, H, d]; w None or [d] (eps None: no norm); table None or [rows, rot/2, 2]."""
    y = np.array(x, dtype=np.float64)
    if eps is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        if w is not None:
            y = y * w
    if table is None:
        return y
    rows, half, _ = table.shape
    out = y.copy()
    for t, pos in enumerate(positions):
        ok = 0 <= pos < rows
        for i in range(half):
            a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
            c, s = table[pos, i].astype(np.float64) if ok else (np.nan, np.nan)
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
    return out


def e4m3_encode(x):
    """Nearest-even codes of x, saturating at 448; NaN -> 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    vals = E4M3[:127]
    hi = np.searchsorted(vals, np.nan_to_num(a)).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = np.nan_to_num(a) - vals[lo], vals[hi] - np.nan_to_num(a)
    code = np.where(dlo < dhi, lo, np.where(dhi < dlo, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.nan_to_num(a) == vals[hi], hi, code)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def scale_exponent(x):
    """Smallest e in [-126, 127] with max |finite x| <= 448 * 2^e (127 if none)."""
    a = np.abs(x[np.isfinite(x)])
    top = a.max() if a.size else 0.0
    e = -126
    while e < 127 and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(cache, k, v, cu_new, ctx, block_table):
    """cache {k, v [pages, Hkv, page, d] uint8, k_scale, v_scale [pages, Hkv]
    uint8}; k, v the (already normed and rotated) new rows.  A new cache."""
    out = {n: np.array(a) for n, a in cache.items()}
    pages, Hkv, P, _ = out["k"].shape
    for b in range(len(ctx)):
        rows = np.arange(cu_new[b], cu_new[b + 1])
        pos = ctx[b] + np.arange(len(rows))
        for col in sorted(set((pos // P).tolist())):
            if col >= block_table.shape[1] or not 0 <= block_table[b, col] < pages:
                continue
            pg, mine = block_table[b, col], pos // P == col
            slots = pos[mine] % P
            for x, n in ((k, "k"), (v, "v")):
                for h in range(Hkv):
                    new = x[rows[mine], h]
                    e = scale_exponent(new)
                    if slots[0] > 0:
                        old = int(out[n + "_scale"][pg, h]) - 127
                        if old >= e:
                            e = old
                        else:
                            s = slice(0, slots[0])
                            out[n][pg, h, s] = e4m3_encode(E4M3[out[n][pg, h, s]] * 2.0 ** (old - e))
                    out[n + "_scale"][pg, h] = e + 127
                    out[n][pg, h, slots] = e4m3_encode(new * 2.0 ** -e)
    return out


def cached(cache, name, block_table_row, length):
    """Values [T, Hkv, d] of a sequence's first tokens, and which of them exist."""
    pages, Hkv, P, d = cache[name].shape
    out, ok = np.zeros((length, Hkv, d)), np.zeros(length, dtype=bool)
    for t in range(length):
        col = t // P
        if col < len(block_table_row) and 0 <= block_table_row[col] < pages:
            pg = block_table_row[col]
            s = 2.0 ** (cache[name + "_scale"][pg].astype(np.float64) - 127)
            out[t], ok[t] = E4M3[cache[name][pg, :, t % P]] * s[:, None], True
    return out, ok


def attend(q, k, v, seen, scale):
    """q [n, Hq, d], k and v [T, Hkv, d], seen bool [n, T] -> o [n, Hq, d], lse [n, Hq].  Unseen keys are not touched."""
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    o, lse = np.zeros((n, Hq, d)), np.full((n, Hq), -np.inf)
    for i in range(n):
        j = np.flatnonzero(seen[i])
        if not len(j):
            continue
        for h in range(Hq):
            s = scale * (k[j, h // G].astype(np.float64) @ q[i, h].astype(np.float64))
            m = s.max()
            p = np.exp(s - m)
            o[i, h] = p @ v[j, h // G] / p.sum()
            lse[i, h] = m + np.log(p.sum())
    return o, lse


def decode(q, cache, block_table, lens, scale):
    o, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    for b, n in enumerate(lens):
        n = max(0, int(n))
        k, ok = cached(cache, "k", block_table[b], n)
        v, _ = cached(cache, "v", block_table[b], n)
        o[b:b + 1], lse[b:b + 1] = attend(q[b:b + 1], k, v, ok[None], scale)
    return o, lse


def prompt(q, k, v, cu_q, cu_k, scale):
    o, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    for b in range(len(cu_q) - 1):
        i0, i1, j0, j1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        lq, lk = i1 - i0, j1 - j0
        seen = np.arange(lk)[None] <= np.arange(lq)[:, None] + (lk - lq)
        o[i0:i1], lse[i0:i1] = attend(q[i0:i1], k[j0:j1], v[j0:j1], seen, scale)
    return o, lse
