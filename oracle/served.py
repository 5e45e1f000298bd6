"""Plain double-precision reference of what a served layer does around its cache
and a layer between its blocks: attention of one new token of each sequence over
a paged, quantised key/value cache, eviction from that cache by weight, and the
norms around a block with its gate and residual scale, forward and backward.

TEST INFRASTRUCTURE ONLY, as the rest of this package.  Arrays are numpy; values
of a cache are float64 [pages, page, heads, d].
"""
from __future__ import annotations

import numpy as np


def stored(codes, scales, kind):
    """The values of codes [..., d] (int4: uint8 [..., d / 2], the even element in the low half)
    with scales [..., d / group]."""
    if kind == "int4":
        low, high = codes.astype(np.int64) & 15, codes.astype(np.int64) >> 4
        codes = np.stack([(low ^ 8) - 8, (high ^ 8) - 8], -1).reshape(*codes.shape[:-1], -1)
    x = codes.astype(np.float64)
    group = x.shape[-1] // scales.shape[-1]
    return (x.reshape(*x.shape[:-1], -1, group) * scales.astype(np.float64)[..., None]).reshape(x.shape)


def slots_of(table, j, page):
    return table[j // page] * page + j % page


def seen(n, cap, window, slots, total):
    """The positions that count, of a length that may be out of range, on pages that may be."""
    n = min(max(int(n), 0), cap)
    j = np.arange(max(0, n - window) if window else 0, n)
    s = slots(j)
    ok = (s >= 0) & (s < total)
    return j[ok], s[ok]


def attention(q, k, v, table, lengths, scale, window=0, cap=None):
    """q [sequences, hq, d]; k, v [pages, page, hk, d].  Returns out, lse, weights [sequences, hk, positions] and the
    sizes that rounding errors scale with: the largest sum |q k| scale of each query head, and sum p |v| of each output."""
    pages, page, hk, d = k.shape
    seqs, hq = q.shape[:2]
    heads = hq // hk
    cap = table.shape[1] * page if cap is None else min(cap, table.shape[1] * page)
    kf, vf = k.reshape(-1, hk, d), v.reshape(-1, hk, d)
    out, lse = np.zeros(q.shape), np.full((seqs, hq), -np.inf)
    weights, sizes, spread = np.zeros((seqs, hk, cap)), np.zeros((seqs, hq)), np.zeros(q.shape)
    for s in range(seqs):
        def slot(j):
            p = table[s][j // page]
            return np.where((p >= 0) & (p < pages), p * page + j % page, -1)
        j, at = seen(lengths[s], cap, window, slot, pages * page)
        if len(j) == 0:
            continue
        for h in range(hq):
            g = h // heads
            prod = kf[at, g] * q[s, h]
            l = scale * prod.sum(-1)
            m = l.max()
            base = 0.0 if np.isneginf(m) else m
            e = np.exp(l - base)
            total = e.sum()
            lse[s, h] = base + np.log(total) if total != 0 else -np.inf
            p = e / total if total != 0 else e
            out[s, h] = p @ vf[at, g]
            weights[s, g, j] += p
            sizes[s, h] = np.abs(scale * prod).sum(-1).max()
            spread[s, h] = p @ np.abs(vf[at, g])
    return out, lse, weights, sizes, spread


def evict(weights, lengths, keep, first, recent, cap):
    """kept [sequences, heads, keep] (-1 behind the last) and the new lengths."""
    seqs, heads = weights.shape[:2]
    kept = np.full((seqs, heads, keep), -1, dtype=np.int64)
    new = np.zeros(seqs, dtype=np.int64)
    for s in range(seqs):
        n = min(max(int(lengths[s]), 0), cap)
        new[s] = min(n, keep)
        for h in range(heads):
            if n <= keep:
                kept[s, h, :n] = np.arange(n)
                continue
            between = range(first, n - recent)

            def rank(j):
                w = weights[s, h, j]
                return (0, 0.0, j) if np.isnan(w) else (1, -float(w), j)
            best = sorted(between, key=rank)[:keep - first - recent]
            kept[s, h] = sorted([*range(first), *best, *range(n - recent, n)])
    return kept, new


def _spread(gate, rows):
    return np.ones((1, 1)) if gate is None else np.repeat(gate, rows // gate.shape[0], 0)


def block_fwd(x, f, gate, w_post, alpha, eps, post=True):
    """y (not rounded), r1"""
    r1 = 1 / np.sqrt((f * f).mean(-1, keepdims=True) + eps) if post else np.ones((x.shape[0], 1))
    n = f * r1 * (w_post if post and w_post is not None else 1.0)
    return x + alpha * _spread(gate, x.shape[0]) * n, r1[:, 0]


def block_pre(y, w_pre, eps):
    """h, r2 of a stored y"""
    r2 = 1 / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    return y * r2 * (1.0 if w_pre is None else w_pre), r2[:, 0]


def block_bwd(dh, dy, f, y, gate, w_post, w_pre, r1, r2, alpha, post=True):
    """dx, df, dgate (None without a gate), dw_post, dw_pre"""
    rows, cols = f.shape
    g = _spread(gate, rows)
    dx = np.zeros_like(f) if dy is None else dy.copy()
    dw_pre = None
    if dh is not None:
        r2 = r2[:, None]
        big = dh * (1.0 if w_pre is None else w_pre)
        dx += r2 * big - y * r2 ** 3 * ((big * y).sum(-1, keepdims=True) / cols)
        dw_pre = (dh * y * r2).sum(0)
    r1 = r1[:, None] if post else np.ones((rows, 1))
    w = 1.0 if not post or w_post is None else w_post
    dn = alpha * g * dx
    dgate = None if gate is None else (alpha * dx * f * r1 * w).reshape(gate.shape[0], -1, cols).sum(1)
    if not post:
        return dx, dn, dgate, None, dw_pre
    small = dn * w
    df = r1 * small - f * r1 ** 3 * ((small * f).sum(-1, keepdims=True) / cols)
    return dx, df, dgate, (dn * f * r1).sum(0), dw_pre
