"""CPU definitions of the paged-cache serving operators: TEST INFRASTRUCTURE ONLY.

The page plan of a step, rotary positions, the int8 append, page bounds, page selection
and attention over page lists, written sequentially in numpy from their definitions
(include/sl8.h states them as readings; the pages name the paged int8 cache, not how it is
filled or pruned).  Lengths and tables are Python integers; rotations and attention are
64-bit; what the definitions fix bit for bit (codes, bounds, scores) uses the fp32
operations they name.  Pinned by ``tests/test_oracle_serving.py``.
"""
from __future__ import annotations

import numpy as np


def _quant(x):
    """codes (int8) and fp32 scales of the rows of an fp32 array: s = max|x| / 127, RNE(x / s)."""
    x = np.asarray(x, np.float32)
    s = np.abs(x).max(-1).astype(np.float32) / np.float32(127.0)
    with np.errstate(invalid="ignore", divide="ignore"):
        c = np.rint(x / s[..., None])
    c = np.where((s[..., None] == 0) | np.isinf(s[..., None]), 0, np.clip(c, -127, 127))
    return c.astype(np.int8), s


def paged_assign(ctx, new, release, table, free, count, page, max_tokens):
    """One request after another.  table [B, max_blocks] and free [capacity] are copied.
    Returns a dict with the updated copies."""
    table, free = np.array(table, np.int64), list(np.asarray(free, np.int64))
    B, nb = table.shape
    stack = free[:count]
    ctx = [int(c) for c in ctx]
    for b in range(B):
        if release is not None and release[b]:
            stack += [int(p) for p in table[b, :-(-ctx[b] // page)]]
            ctx[b] = 0
    assert len(stack) <= len(free)
    free[:len(stack)] = stack
    have, asked, start = len(stack), 0, 0
    seqlens, granted, cu = [], [], [0]
    slots, poss = [-1] * max_tokens, [0] * max_tokens
    taken = 0
    for b in range(B):
        n, c = int(new[b]), ctx[b]
        ok = c + n <= nb * page and start + n <= max_tokens
        need = -(-(c + n) // page) - -(-c // page) if ok else 0
        asked += need
        if need and asked > have:
            ok = False
        if ok:
            first = -(-c // page)
            for j in range(need):
                table[b, first + j] = stack[have - 1 - taken]
                taken += 1
        for i in range(n):
            if start + i < max_tokens:
                poss[start + i] = c + i
                if ok:
                    slots[start + i] = int(table[b, (c + i) // page]) * page + (c + i) % page
        start += n
        cu.append(start)
        granted.append(n if ok else 0)
        seqlens.append(c + granted[-1])
    return dict(block_table=table, free_pages=np.array(free), free_count=have - taken, seqlens=np.array(seqlens),
                granted=np.array(granted), cu_new=np.array(cu), slot_map=np.array(slots), token_pos=np.array(poss))


def rope(x, positions, inv_freq, pair_axis=None, adjacent=False):
    """x [T, H, d] rotated, fp64.  positions [axes, T]."""
    y = np.array(x, np.float64)
    half = len(inv_freq)
    for p in range(half):
        a = 0 if pair_axis is None else pair_axis[p]
        t = np.asarray(positions, np.float64)[a] * float(np.float32(inv_freq[p]))
        i, j = (2 * p, 2 * p + 1) if adjacent else (p, half + p)
        u, v = y[:, :, i].copy(), y[:, :, j].copy()
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        y[:, :, i], y[:, :, j] = u * c - v * s, v * c + u * s
    return y


def page_bounds(codes, scales):
    """Bounds of one page and head from its valid rows: codes [n, d] int8, scales [n] fp32.
    Returns (lo, hi) int and S fp32."""
    S = np.float32(scales.max())
    if S == 0 or np.isinf(S):
        z = np.zeros(codes.shape[1], np.int64)
        return z, z.copy(), S
    y = codes.astype(np.float32) * (scales.astype(np.float32) / S)[:, None]
    return np.floor(y.min(0)).astype(np.int64), np.ceil(y.max(0)).astype(np.int64), S


def page_scores(q, lo, hi, S):
    """Scores fp32 of pages (lo, hi [n, d] int, S [n] fp32) for the query heads q [G, d] fp32."""
    c, sq = _quant(q)
    c = c.astype(np.int64)[:, None]
    dots = np.maximum(c * lo[None], c * hi[None]).sum(-1)
    with np.errstate(invalid="ignore"):
        s = dots.astype(np.float32) * S[None].astype(np.float32) * sq[:, None]
    return np.where(np.isnan(s), np.float32(-np.inf), s).max(0)


def select(scores, max_sel, first, last):
    """Kept blocks, ascending: scores [n] of the blocks of one query's range."""
    n = len(scores)
    if n <= max_sel:
        return list(range(n))
    forced = set(range(first)) | set(range(n - last, n))
    rest = sorted((i for i in range(n) if i not in forced), key=lambda i: (-float(scores[i]), i))
    return sorted(forced | set(rest[:max_sel - len(forced)]))


def sparse_attention(q, k_pages, k_scale, v_pages, v_scale, pages, lens):
    """q [R, Hq, d] fp32, pages [R, Hkv, max_sel], lens [R, Hkv]: (out fp64, lse fp64)."""
    R, Hq, d = q.shape
    Hkv, P = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hkv
    out, lse = np.zeros((R, Hq, d)), np.full((R, Hq), -np.inf)
    codes, sq = _quant(q)
    for r in range(R):
        for h in range(Hkv):
            n = int(lens[r, h])
            if n == 0:
                continue
            ids = pages[r, h, :-(-n // P)]
            k = (k_pages[ids, h].astype(np.float64) * k_scale[ids, h].astype(np.float64)[..., None]).reshape(-1, d)[:n]
            v = (v_pages[ids, h].astype(np.float64) * v_scale[ids, h].astype(np.float64)[..., None]).reshape(-1, d)[:n]
            for g in range(G):
                x = k @ codes[r, h * G + g].astype(np.float64) * float(sq[r, h * G + g]) / np.sqrt(d)
                m = x.max()
                e = np.exp(x - m)
                out[r, h * G + g] = e @ v / e.sum()
                lse[r, h * G + g] = m + np.log(e.sum())
    return out, lse
