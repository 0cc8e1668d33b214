"""Plain 64-bit forms of the operators for activations in 8 bits (models:
include/ss_rows8.h, include/ss_rms.h, include/ss_dense.h), from their
definitions, in NumPy.

Inputs are converted to float64 first; nothing is rounded to fewer bits but
what the 8-bit formats round.
"""
from __future__ import annotations

import numpy as np

GROUP = 32
Q = {"int8": 127.0, "e4m3": 448.0}
LEAST = -111     # exponent of the least scale
NAN = 255        # biased exponent of a group that is not finite


def _f(a):
    return np.asarray(a, dtype=np.float64)


def scale_exponents(x, fmt):
    """Biased exponents [n, groups] of the scales of the rows x [n, D]."""
    x = _f(x)
    n, D = x.shape
    G = -(-D // GROUP)
    e = np.zeros((n, G), dtype=np.int64)
    for g in range(G):
        most = np.abs(x[:, g * GROUP:(g + 1) * GROUP]).max(1) if n else np.zeros(0)
        for i, m in enumerate(most):
            if not np.isfinite(m):
                e[i, g] = NAN
                continue
            s = LEAST
            while m > Q[fmt] * 2.0 ** s:
                s += 1
            e[i, g] = s + 127
    return e


def round_to(z, fmt):
    """The nearest value of the format (ties to even) of |z| <= Q."""
    z = _f(z)
    if fmt == "int8":
        return np.rint(z)
    lead = np.maximum(np.frexp(z)[1] - 1, -6)
    step = np.ldexp(1.0, lead - 3)
    return np.rint(z / step) * step


def held(x, fmt):
    """(what the rows read as, q, biased exponents)."""
    x = _f(x)
    e = scale_exponents(x, fmt)
    wide = np.repeat(e, GROUP, axis=1)[:, :x.shape[1]]
    bad = wide == NAN
    s = np.ldexp(1.0, np.where(bad, 127, wide) - 127)
    q = round_to(np.where(bad, 0.0, x) / s, fmt)
    return np.where(bad, np.nan, q * s), q, e


def rms_fwd(h, gamma, eps):
    """(y, rstd) of the rows h (the sum with the residual, rounded as it is kept)."""
    h = _f(h)
    gamma = np.ones(h.shape[1]) if gamma is None else _f(gamma)
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1.0 / np.sqrt((h * h).sum(1) / h.shape[1] + eps)
        return h * rstd[:, None] * gamma, rstd


def rms_bwd(dy, h, gamma, rstd, dsum=None):
    """(dx, dgamma) with rstd as the forward gave it."""
    dy, h = _f(dy), _f(h)
    D = h.shape[1]
    gamma = np.ones(D) if gamma is None else _f(gamma)
    g = h * _f(rstd)[:, None]
    a = dy * gamma
    dx = _f(rstd)[:, None] * (a - g * ((a * g).sum(1, keepdims=True) / D))
    return dx if dsum is None else dx + _f(dsum), (dy * g).sum(0)


def dense_bwd(dy, x):
    """(dW [N, D], db [N], the sums of the summands' magnitudes)."""
    dy, x = _f(dy), _f(x)
    return dy.T @ x, dy.sum(0), np.abs(dy).T @ np.abs(x), np.abs(dy).sum(0)
