"""The polynomials of the cap and of its derivative (csrc/ra_api.cu, score_params): what they are off by, and how they are made.

tanh(u) = u (1 + w P(w)) and 1 - tanh(u)^2 = 1 + w G(w) with w = u^2, each with the least largest error relative to the
function for |u| up to T.  Such coefficients come from Lawson's algorithm (C. L. Lawson, 1961): least squares over a
grid, whose weights are multiplied by the errors again and again."""
import os
import re

import numpy as np
import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ring_attn_gb300", "csrc", "ra_api.cu")


def tanh_over_u(w):
    return np.tanh(np.sqrt(w)) / np.sqrt(w)


def derivative(w):
    return 1 / np.cosh(np.sqrt(w)) ** 2


def grid(T, n):
    """w of Chebyshev points, for in the middle of the interval the errors change least."""
    w = (np.cos(np.linspace(0, np.pi, n)) + 1) / 2 * T * T
    return w[w > 1e-10].astype(np.longdouble)


def errors(f, T, c, n=20001):
    w = grid(T, n)
    return np.abs((1 + w * sum(np.longdouble(x) * w ** i for i, x in enumerate(c))) / f(w) - 1).astype(float)


def lawson(f, T, n_coef, steps=600):
    """(largest error, coefficients) of 1 + w (c_0 + c_1 w + ...) next to f, relatively, for w up to T^2."""
    w = grid(T, 8001)
    size = (w / f(w)).astype(float)
    want = ((f(w) - 1) / w).astype(float)
    x = (w / (T * T)).astype(float)
    weight, best = np.ones_like(x), (np.inf, None)
    for _ in range(steps):
        r = np.sqrt(weight) * size
        c = np.linalg.lstsq(np.stack([x ** i for i in range(n_coef)], 1) * r[:, None], want * r, rcond=None)[0]
        e = np.abs((sum(c[i] * x ** i for i in range(n_coef)) - want) * size)
        if e.max() < best[0]:
            best = (e.max(), [c[i] / T ** (2 * i) for i in range(n_coef)])
        weight = weight * (e / e.max() + 1e-3)
        weight /= weight.sum()
    return best


def coefficients(name):
    text = open(SOURCE).read()
    row = re.search(r"\b%s\[(\d)\] = \{([^}]*)\}" % name, text)
    c = [float(x) for x in row.group(2).split(",")]
    assert len(c) == int(row.group(1))
    return c


@pytest.mark.parametrize("name,f,T,bits", [
    ("p0", tanh_over_u, 0.4, 23.1), ("p1", tanh_over_u, 0.6, 23.5), ("p2", tanh_over_u, 1.0, 24.1),
    ("d0", derivative, 0.4, 14.1), ("d1", derivative, 0.6, 15.4), ("d2", derivative, 1.0, 16.7),
])
def test_errors_and_making(name, f, T, bits):
    c = coefficients(name)
    off = errors(f, T, c).max()
    assert off <= 2.0 ** -(bits - 0.06)  # as the kernels' comment has it, to a decimal
    least, made = lawson(f, T, len(c))
    assert off <= 1.02 * least + 1e-12  # none does much better
    w = T * T
    # the same polynomial: where two are within e of one function they are within 2 e of one another
    x = np.linspace(0, w, 101)
    assert np.abs(sum((a - b) * x ** (i + 1) for i, (a, b) in enumerate(zip(c, made)))).max() <= 2.1 * off
