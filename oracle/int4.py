"""CPU definitions of the paged 4-bit cache's operators: TEST INFRASTRUCTURE ONLY.

The 4-bit rows (groups of 32 channels with a bf16 scale, codes within +-7 held as code + 8, two a
byte), reading them back, and decode attention over their pages, written in numpy from their
definitions (include/sl8.h states them as readings: the pages name 4-bit values, not their layout).
Pinned by ``tests/test_oracle_int4.py``.
"""
from __future__ import annotations

import numpy as np

from .serving import _quant

GROUP = 32


def to_bf16(x):
    """fp32 rounded to bf16 (nearest, ties to even), as fp32; infinities stay."""
    u = np.ascontiguousarray(np.asarray(x, np.float32)).view(np.uint32).astype(np.uint64)
    u = ((u + 0x7fff + ((u >> 16) & 1)) >> 16) << 16
    return u.astype(np.uint32).view(np.float32)


def quant4(x):
    """codes [..., d] in -7 .. 7 and scales [..., d / 32] (bf16 values as fp32) of fp32 rows."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        s = to_bf16(np.fmax.reduce(np.abs(g), -1, initial=np.float32(0)) / np.float32(7))
        c = np.clip(np.rint(g.astype(np.float64) / s[..., None].astype(np.float64)), -7, 7)
    c = np.where((s[..., None] == 0) | np.isinf(s[..., None]) | np.isnan(g), 0, c)
    return c.reshape(x.shape).astype(np.int64), s


def pack(codes):
    n = (np.asarray(codes) + 8).astype(np.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def unpack(packed):
    p = np.asarray(packed)
    return np.stack((p & 15, p >> 4), -1).reshape(*p.shape[:-1], 2 * p.shape[-1]).astype(np.int64) - 8


def values(packed, scales):
    """What packed rows stand for, fp64."""
    with np.errstate(invalid="ignore"):
        return unpack(packed) * np.repeat(np.asarray(scales, np.float64), GROUP, -1)


def gather(pages, table, n):
    """Rows 0 .. n - 1 of a sequence, [Hkv, n, ...], from pages [num_pages, Hkv, page, ...]."""
    page = pages.shape[2]
    ids = np.asarray(table)[:-(-n // page)]
    x = np.moveaxis(pages[ids], 0, 1)  # [Hkv, blocks, page, ...]
    return x.reshape(x.shape[0], x.shape[1] * page, *x.shape[3:])[:, :n]


def visible(L, T, t, mask=None):
    """Tokens that draft query t of T sees: those before the drafts, and drafts by the mask's bits
    (without a mask, up to itself)."""
    return [p for p in range(L) if p < L - T or (p - (L - T) <= t if mask is None else (int(mask) >> (p - (L - T))) & 1)]


def attention(q, kc, ks, vc, vs, tables, lens, masks=None, bounds=False):
    """q [B, T, Hq, d] fp32; packed pages and scales; (out fp64, lse fp64).  bounds: also
    sum_t p_t |v_t| like out, and of each query's tokens the largest sum_c |q_c k_c| / sqrt(d) and the
    largest p_t times a V scale."""
    B, T, Hq, d = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    out, lse = np.zeros(q.shape), np.full(q.shape[:-1], -np.inf)
    size, reach, heavy = np.zeros(q.shape), np.zeros(q.shape[:-1]), np.zeros(q.shape[:-1])
    codes, sq = _quant(q)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        k = values(gather(kc, tables[b], n), gather(ks, tables[b], n))
        v = values(gather(vc, tables[b], n), gather(vs, tables[b], n))
        for t in range(T):
            see = visible(n, T, t, None if masks is None else masks[b][t])
            if not see:
                continue
            for h in range(Hq):
                row = codes[b, t, h].astype(np.float64) * float(sq[b, t, h]) / np.sqrt(d)
                x = k[h // G][see] @ row
                m = x.max()
                e = np.exp(x - m)
                out[b, t, h] = e @ v[h // G][see] / e.sum()
                lse[b, t, h] = m + np.log(e.sum())
                if bounds:
                    size[b, t, h] = e @ np.abs(v[h // G][see]) / e.sum()
                    reach[b, t, h] = (np.abs(k[h // G][see]) @ np.abs(row)).max()
                    heavy[b, t, h] = (e * gather(vs, tables[b], n)[h // G][see].max(-1)).max() / e.sum()
    return (out, lse, size, reach, heavy) if bounds else (out, lse)
