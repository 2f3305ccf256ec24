"""fp64 oracle of attention with changed scores (cap, bias by distance, prefix) and of
rotary positions, each straight from its definition.

With x = scale <q_i, k_j>: y = cap tanh(x / cap) (cap 0: x), z = y - slope_h |i - j|, and
attention over z; a causal query i sees key j when j <= i or j < prefix."""
from __future__ import annotations

import numpy as np


def changed(x, gq, gk, cap, slope):
    """(z, dz/dx) of scores x (m, n); gq, gk: tokens."""
    x = np.asarray(x, dtype=np.float64)
    th = np.tanh(x / cap) if cap else np.zeros_like(x)
    y = cap * th if cap else x
    return y - slope * np.abs(np.asarray(gq)[:, None] - np.asarray(gk)[None, :]), 1.0 - th * th


def seen(gq, gk, causal, prefix, segq=None, segk=None):
    """Which keys each query sees; prefix: tokens of the sequence that all see (with segments: counted
    from the sequence's first token, which the callers subtract)."""
    gq, gk = np.asarray(gq)[:, None], np.asarray(gk)[None, :]
    see = (gk <= gq) | (gk < prefix) if causal else np.ones((gq.shape[0], gk.shape[1]), dtype=bool)
    if segq is not None:
        see &= np.asarray(segq)[:, None] == np.asarray(segk)[None, :]
    return see


def head(q, k, v, gq, gk, scale, cap=0.0, slope=0.0, causal=False, prefix=0, do=None):
    """One head: dict of out, lse, P and, with do, dq, dk, dv and their parts; rows that see nothing: 0, -inf."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    z, g = changed(scale * (q @ k.T), gq, gk, cap, slope)
    z = np.where(seen(gq, gk, causal, prefix), z, -np.inf)
    m = z.max(1, initial=-np.inf)
    some = np.isfinite(m)
    e = np.exp(z - np.where(some, m, 0.0)[:, None])
    l = e.sum(1)
    P = e / np.where(some, l, 1.0)[:, None]
    r = {"out": P @ v, "lse": np.where(some, m + np.log(np.where(some, l, 1.0)), -np.inf), "P": P, "g": g, "z": z}
    if do is not None:
        do = np.asarray(do, dtype=np.float64)
        D = (do * r["out"]).sum(1)
        dP = do @ v.T
        dx = P * (dP - D[:, None]) * g
        r.update(D=D, dP=dP, dx=dx, dq=scale * (dx @ k), dk=scale * (dx.T @ q), dv=P.T @ do)
    return r


def rotate(x, cos, sin, pos, axes, interleaved, inverse=False):
    """x (rows, heads, d); cos, sin (positions, r / 2); pos (axes, rows); axes: the axis of each pair."""
    x = np.array(x, dtype=np.float64)
    f = np.arange(len(axes))
    row = np.asarray(pos)[np.asarray(axes)].T  # (rows, pairs)
    c, s = np.asarray(cos, np.float64)[row, f][:, None], np.asarray(sin, np.float64)[row, f][:, None]
    if inverse:
        s = -s
    a, b = (2 * f, 2 * f + 1) if interleaved else (f, f + len(axes))
    xa, xb = x[..., a], x[..., b]
    x[..., a], x[..., b] = xa * c - xb * s, xb * c + xa * s
    return x
