"""Plain double-precision reference of the operators on attention heads: RMSNorm
of each head with the rotation by position, its backward, and the quantised
key/value cache.

TEST INFRASTRUCTURE ONLY, as the rest of this package.  Arrays are numpy
float64: rows [tokens, heads, d], positions int64 [axes, tokens].
"""
from __future__ import annotations

import numpy as np

QMAX = {"e4m3": 448.0, "int8": 127.0, "int4": 7.0}


def angles(pos, inv_freq, axis=None):
    """[tokens, pairs] in radians, reduced exactly: the products of 63-bit positions
    with 24-bit frequencies are formed as Python integers over a power of two."""
    from fractions import Fraction
    pos = np.atleast_2d(np.asarray(pos, dtype=np.int64))
    axis = [0] * len(inv_freq) if axis is None else list(axis)
    two_pi = Fraction(31415926535897932384626433832795028841971, 5 * 10 ** 39)
    out = np.empty((pos.shape[1], len(inv_freq)))
    for p, f in enumerate(np.asarray(inv_freq, dtype=np.float32)):
        f = Fraction(float(f))
        for t in range(pos.shape[1]):
            a = int(pos[axis[p], t]) * f
            out[t, p] = float(a - (a / two_pi).__floor__() * two_pi)
    return out


def rotate(x, ang, pairs="half", inverse=False):
    n = ang.shape[1]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None] * (-1.0 if inverse else 1.0)
    y = x.copy()
    a, b = (slice(0, n), slice(n, 2 * n)) if pairs == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    u, v = x[..., a], x[..., b]
    y[..., a] = u * c - v * s
    y[..., b] = v * c + u * s
    return y


def pair_size(x, n, pairs="half"):
    """|u| + |v| of the pair each element belongs to (|x| outside the rotated part):
    the size that rounding errors of a rotated element scale with."""
    z = np.abs(x)
    a, b = (slice(0, n), slice(n, 2 * n)) if pairs == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    u, v = z[..., a].copy(), z[..., b].copy()
    z[..., a] = z[..., b] = u + v
    return z


def norm_rope_fwd(x, w, ang, eps, pairs="half"):
    """y, r"""
    r = 1.0 / np.sqrt((x * x).mean(-1) + eps)
    n = x * r[..., None]
    if w is not None:
        n = n * w
    return rotate(n, ang, pairs), r


def norm_rope_bwd(dy, x, w, ang, eps, pairs="half"):
    """dx, dw"""
    r = 1.0 / np.sqrt((x * x).mean(-1) + eps)[..., None]
    back = rotate(dy, ang, pairs, inverse=True)
    g = back if w is None else back * w
    s = (g * x).sum(-1, keepdims=True)
    return r * g - x * r ** 3 * s / x.shape[-1], (back * x * r).sum((0, 1))


def _round_e4m3(u):
    e = np.floor(np.log2(np.maximum(np.abs(u), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.rint(u / step) * step


def quantise(x, kind, group):
    """(codes as the numbers they are, scales as float32) of x[..., d]; ties to even."""
    parts = x.reshape(*x.shape[:-1], -1, group)
    m = np.abs(parts).max(-1, keepdims=True)
    bad = ~np.isfinite(parts).all(-1, keepdims=True)
    zero = ~bad & (m < 2.0 ** -100)
    div = np.where(bad | zero, 1.0, m)
    with np.errstate(invalid="ignore", over="ignore"):
        u = np.where(bad | zero, 0.0, parts * QMAX[kind] / div)
        scale = np.where(bad, np.nan, np.where(zero, 0.0, m / QMAX[kind])).astype(np.float32)
    codes = _round_e4m3(u) if kind == "e4m3" else np.rint(u)
    return codes.reshape(x.shape), scale[..., 0]
