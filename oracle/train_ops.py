"""Plain 64-bit forms of the training operators (models: include/ss_embed.h,
include/ss_norm.h, include/ss_clip.h), from their definitions, in NumPy.

Inputs are converted to float64 first; nothing is rounded to fewer bits.
"""
from __future__ import annotations

import numpy as np


def _f(a):
    return np.asarray(a, dtype=np.float64)


def embed_fwd(table, ids, scale):
    table, ids = _f(table), np.asarray(ids, dtype=np.int64)
    out = np.zeros((len(ids), table.shape[1]))
    for i, v in enumerate(ids):
        if 0 <= v < len(table):
            out[i] = scale * table[v]
    return out


def embed_bwd(dout, ids, V, scale):
    """(gradient, sum of the summands' magnitudes, summands of each row)."""
    dout, ids = _f(dout), np.asarray(ids, dtype=np.int64)
    here = (ids >= 0) & (ids < V)
    g = np.zeros((V, dout.shape[1]))
    mag = np.zeros_like(g)
    np.add.at(g, ids[here], scale * dout[here])
    np.add.at(mag, ids[here], np.abs(scale * dout[here]))
    return g, mag, np.bincount(ids[here], minlength=V)


def layer_norm_fwd(x, gamma, beta, eps):
    x = _f(x)
    D = x.shape[1]
    gamma = np.ones(D) if gamma is None else _f(gamma)
    beta = np.zeros(D) if beta is None else _f(beta)
    mean = x.sum(1) / D
    var = ((x - mean[:, None]) ** 2).sum(1) / D
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1.0 / np.sqrt(var + eps)
        y = (x - mean[:, None]) * rstd[:, None] * gamma + beta
    return y, mean, rstd


def layer_norm_bwd(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta) with mean and rstd as the forward gave them."""
    dy, x = _f(dy), _f(x)
    D = x.shape[1]
    gamma = np.ones(D) if gamma is None else _f(gamma)
    h = (x - _f(mean)[:, None]) * _f(rstd)[:, None]
    a = dy * gamma
    ma = a.sum(1, keepdims=True) / D
    mah = (a * h).sum(1, keepdims=True) / D
    return _f(rstd)[:, None] * (a - ma - h * mah), (dy * h).sum(0), dy.sum(0)


def grad_clip(tensors, max_norm, eps):
    """(norm, coefficient, scaled tensors)."""
    ts = [_f(t) for t in tensors]
    with np.errstate(over="ignore", invalid="ignore"):
        norm = np.sqrt(sum(float((t * t).sum()) for t in ts))
    if not np.isfinite(norm):
        return norm, 0.0, ts
    coef = min(1.0, max_norm / (norm + eps)) if norm + eps > 0 else 1.0
    return norm, coef, [coef * t for t in ts]
