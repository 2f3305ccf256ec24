"""fp64 oracle of the paged 4-bit key / value cache: quantisation, rotation,
paging and attention, each straight from its definition."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)])
GROUP = 16


def nearest(x, grid):
    """Index of the number of `grid` (ascending, from 0) nearest to x >= 0; ties to the even index."""
    x = np.minimum(np.asarray(x, dtype=np.float64), grid[-1])
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    down, up = x - grid[lo], grid[hi] - x
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def quantise(x):
    """(codes (..., d / 2) uint8, scales (..., d / 16) uint8) of (..., d) numbers."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    s8 = np.maximum(nearest(np.abs(g).max(-1) / 6.0, E4M3), 1)
    code = nearest(np.abs(g) / E4M3[s8][..., None], E2M1) + 8 * np.signbit(g)
    code = code.reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), s8.astype(np.uint8)


def dequantise(codes, scales):
    codes = np.asarray(codes)
    code = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    return v * np.repeat(E4M3[np.asarray(scales)], GROUP, -1)


def rotate(x, cos, sin, interleaved):
    """x (rows, heads, d); cos, sin (rows, r / 2): pairs of the first r head dims turned."""
    x = np.array(x, dtype=np.float64)
    r = 2 * cos.shape[-1]
    i = np.arange(r // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    c, s = np.asarray(cos, np.float64)[:, None], np.asarray(sin, np.float64)[:, None]
    xa, xb = x[..., a], x[..., b]
    x[..., a], x[..., b] = xa * c - xb * s, xb * c + xa * s
    return x


def attention(q, k, v, scale, n_before):
    """q (n, h, d) over k, v (m, hk, d): row j sees keys [0, n_before[j]).

    Returns out (n, h, d), lse (h, n), and two sizes that error bounds are made
    of: sum p |v| / l (n, h, d) and max_j sum |q k_j| scale (h, n)."""
    n, h, d = q.shape
    m, hk = k.shape[:2]
    out, lse = np.zeros((n, h, d)), np.full((h, n), -np.inf)
    size, dots = np.zeros((n, h, d)), np.zeros((h, n))
    see = np.arange(m)[None] < np.asarray(n_before)[:, None]
    some = see.any(1)
    for i in range(h):
        kk, vv = k[:, i * hk // h], v[:, i * hk // h]
        s = np.where(see, (q[:, i] @ kk.T) * scale, -np.inf)
        mx = np.where(some, s.max(1, initial=-np.inf), 0.0)
        p = np.exp(s - mx[:, None])
        l = p.sum(1)
        safe = np.where(some, l, 1.0)[:, None]
        out[:, i], size[:, i] = p @ vv / safe, p @ np.abs(vv) / safe
        lse[i, some] = mx[some] + np.log(l[some])
        dots[i] = (np.abs(q[:, i]) @ np.abs(kk).T).max(1, initial=0.0) * scale
    return out, lse, size, dots
