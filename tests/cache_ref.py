"""Plain 64-bit statements of the operators around the attention, for the tests:
rotary positions, the 8-bit cache (its rounding, append and compact), attention
over it, key weights and key selection. numpy and loops; no library code."""
from __future__ import annotations

import math

import numpy as np

INT8, E4M3 = 0, 1
FULL = {INT8: 127.0, E4M3: 448.0}


def nearest(y, fmt):
    """y rounded to the nearest code (as its value), ties to even."""
    y = np.asarray(y, np.float64)
    if fmt == INT8:
        return np.rint(y)
    a = np.abs(y)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = np.exp2(np.maximum(e, -6.0) - 3.0)
    return np.sign(y) * np.minimum(np.rint(a / step) * step, 448.0)


def rope(x, pos, inv_freq, rot, interleaved, mscale=1.0, inverse=False):
    """x [B, N, H, D] float64, pos [B, N]."""
    t = pos[..., None].astype(np.float64) * np.asarray(inv_freq)[None, None]
    c, s = np.cos(t)[:, :, None] * mscale, np.sin(t)[:, :, None] * mscale * (-1 if inverse else 1)
    y = x.copy()
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def append(x, lens, counts, table, codes, ranges, fmt, index=None):
    """codes [pages, H, P, D] (values), ranges [pages, H]; updated copies returned."""
    codes, ranges = codes.copy(), ranges.copy()
    n_pages, H, P, _ = codes.shape
    B, n_src = x.shape[:2]
    for b in range(B):
        cap = table.shape[1] * P
        a = min(max(int(lens[b]), 0), cap)
        for h in range(H):
            for blk in range(a // P, table.shape[1]):
                lo, hi = max(a, blk * P), min(a + int(counts[b]), (blk + 1) * P)
                page = int(table[b, blk])
                if hi <= lo or not 0 <= page < n_pages:
                    continue
                rows = []
                for i in range(lo - a, hi - a):
                    src = i if index is None else int(index[b, h, i])
                    rows.append(x[b, src, h] if 0 <= src < n_src else np.zeros_like(x[b, 0, h]))
                rows = np.array(rows)
                old = ranges[page, h] if lo > blk * P else 0.0
                top = np.abs(rows).max() if not np.isnan(rows).any() else np.nan
                r = top if np.isnan(top) or np.isnan(old) else max(top, old)
                if np.isnan(old):
                    r = old
                s, e = lo - blk * P, hi - blk * P
                if not np.isfinite(r) or r == 0:
                    codes[page, h, :e] = 0
                else:
                    if s:
                        codes[page, h, :s] = nearest(codes[page, h, :s] * old / r, fmt)
                    codes[page, h, s:e] = nearest(rows * FULL[fmt] / r, fmt)
                ranges[page, h] = r
    return codes, ranges


def compact(index, kept, lens, table, new_table, codes, ranges, fmt):
    out, new = codes.copy(), ranges.copy()
    n_pages, H, P, _ = codes.shape
    for b in range(index.shape[0]):
        for h in range(H):
            for blk in range(new_table.shape[1]):
                to, n = int(new_table[b, blk]), min(int(kept[b]) - blk * P, P)
                if n <= 0 or not 0 <= to < n_pages:
                    continue
                src = []
                for i in index[b, h, blk * P: blk * P + n]:
                    page = int(table[b, i // P]) if 0 <= i < lens[b] else -1
                    src.append((page, int(i) % P) if 0 <= page < n_pages else None)
                r2 = max([ranges[s[0], h] for s in src if s] or [0.0])
                for k, s in enumerate(src):
                    out[to, h, k] = 0 if s is None or r2 == 0 else nearest(
                        codes[s[0], h, s[1]] * ranges[s[0], h] / r2, fmt)
                new[to, h] = r2
    return out, new


def values(codes, ranges, table, b, h, n, fmt):
    """The first n cached values of a sequence and head, [n, D]; None where a page is missing."""
    P = codes.shape[2]
    rows, there = [], []
    for j in range(n):
        page = int(table[b, j // P])
        ok = 0 <= page < codes.shape[0]
        there.append(ok)
        rows.append(codes[page, h, j % P] * ranges[page, h] / FULL[fmt] if ok
                    else np.zeros(codes.shape[3]))
    return np.array(rows).reshape(n, codes.shape[3]), np.array(there, bool)


def attention(q, k8, v8, kr, vr, table, lens, scale, fmt):
    """(o, its bound, weights, their bound). The bounds follow the arithmetic:
    fp32 scores off by at most D 2^-23 sum_d |q_d k_d| scale (each of D exact
    products added with an error of at most one last place of the running sum)
    plus 2^-20 of |s| for the scalings; 2^x good to 2^-21; P in fp16 (2^-11 of
    each weight, and nothing below 2^-32 of the largest); o in bf16 (2^-8 of o)."""
    B, nq, Hq, D = q.shape
    H = k8.shape[1]
    G, P = Hq // H, k8.shape[2]
    cap = table.shape[1] * P
    o, bo = np.zeros(q.shape), np.zeros(q.shape)
    w, bw = np.zeros((B, H, cap)), np.zeros((B, H, cap))
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        for h in range(H):
            k, ok = values(k8, kr, table, b, h, n, fmt)
            v, _ = values(v8, vr, table, b, h, n, fmt)
            for i in range(nq):
                m = n - nq + i + 1
                if m <= 0 or not ok[:m].any():
                    continue
                for g in range(G):
                    qq = q[b, i, h * G + g]
                    s = np.where(ok[:m], (k[:m] @ qq) * scale, -np.inf)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    err = (np.abs(k[:m]) @ np.abs(qq)) * scale * D * 2.0 ** -23
                    err = 2 * (err + np.abs(np.where(ok[:m], s, 0)) * 2.0 ** -20).max() + 2.0 ** -20
                    o[b, i, h * G + g] = p @ v[:m]
                    mass = p @ np.abs(v[:m])
                    bo[b, i, h * G + g] = (np.abs(p @ v[:m]) * 2.0 ** -8 * (1 + err)
                                           + mass * (2.0 ** -11 + 2 * err)
                                           + m * 2.0 ** -32 * np.abs(v[:m]).max() + 1e-30)
                    w[b, h, :m] += p
                    bw[b, h, :m] += p * 2 * err + 1e-30
    return o, bo, w, bw


def key_weights(q, k, scale, L, lens):
    """(weights, bound): as for attention, without P's rounding."""
    B, N, Hq, D = q.shape
    H = k.shape[2]
    G = Hq // H
    w, bw = np.zeros((B, H, N)), np.zeros((B, H, N))
    for b in range(B):
        n = min(max(int(lens[b]), 0), N)
        for h in range(Hq):
            kk = k[b, :n, h // G]
            rows = np.arange(max(0, n - L), n)
            s = (q[b, rows, h] @ kk.T) * scale
            mag = (np.abs(q[b, rows, h]) @ np.abs(kk).T) * scale * D * 2.0 ** -23
            seen = np.arange(n)[None] <= rows[:, None]
            err = np.where(seen, mag + np.abs(s) * 2.0 ** -20, 0).max(1, keepdims=True,
                                                                      initial=0)
            s = np.where(seen, s, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True, initial=-1e300))
            p /= p.sum(1, keepdims=True)
            w[b, h // G, :n] += p.sum(0)
            bw[b, h // G, :n] += (p * (4 * err + 2.0 ** -19)).sum(0) + 1e-30
    return w, bw


def select(w, n, keep, sinks, recent):
    """Indices kept of one row of n weights."""
    if n <= keep:
        return list(range(n))

    def rank(j):
        held = j < sinks or j >= n - recent
        x = float(w[j])
        return (not held, math.isnan(x), 0.0 if math.isnan(x) else -x, j)

    return sorted(sorted(range(n), key=rank)[:keep])
