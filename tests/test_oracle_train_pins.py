"""Pins of the training operators' 64-bit forms: closed cases by hand, and
every gradient against central differences of its forward."""
import numpy as np
import pytest

import oracle.train_ops as O


def test_lookup_by_hand():
    t = [[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]]
    out = O.embed_fwd(t, [2, -1, 0, 3, 2], 0.5)
    assert out.tolist() == [[2.5, 3.0], [0, 0], [0.5, 1.0], [0, 0], [2.5, 3.0]]
    g, mag, cnt = O.embed_bwd([[1.0], [-2.0], [4.0], [np.nan]], [1, 1, 0, 7], 3, 2.0)
    assert g.tolist() == [[8.0], [-2.0], [0.0]]
    assert mag.tolist() == [[8.0], [6.0], [0.0]] and cnt.tolist() == [1, 2, 0]


def test_lookup_gradient_against_differences():
    r = np.random.default_rng(1)
    t, w = r.normal(size=(5, 3)), r.normal(size=(9, 3))
    ids = r.integers(-1, 6, 9)
    g, _, _ = O.embed_bwd(w, ids, 5, 1.7)
    for k in np.ndindex(5, 3):
        d = np.zeros_like(t)
        d[k] = 1e-5
        num = ((O.embed_fwd(t + d, ids, 1.7) - O.embed_fwd(t - d, ids, 1.7)) * w).sum() / 2e-5
        assert abs(num - g[k]) < 1e-8


def test_norm_by_hand():
    y, mean, rstd = O.layer_norm_fwd([[1.0, 3.0], [5.0, 5.0]], None, None, 0.0)
    assert mean.tolist() == [2.0, 5.0] and rstd[0] == 1.0 and np.isinf(rstd[1])
    assert y[0].tolist() == [-1.0, 1.0]
    y, _, rstd = O.layer_norm_fwd([[5.0, 5.0]], [2.0, 2.0], [1.0, -1.0], 0.25)
    assert rstd[0] == 2.0 and y.tolist() == [[1.0, -1.0]]


@pytest.mark.parametrize("D", [1, 2, 7])
def test_norm_gradient_against_differences(D):
    r = np.random.default_rng(D)
    n, eps = 4, 1e-2
    x, w, g, b = r.normal(size=(n, D)), r.normal(size=(n, D)), r.normal(size=D), r.normal(size=D)
    _, mean, rstd = O.layer_norm_fwd(x, g, b, eps)
    dx, dg, db = O.layer_norm_bwd(w, x, g, mean, rstd)

    def L(x, g, b):
        return (O.layer_norm_fwd(x, g, b, eps)[0] * w).sum()

    h = 1e-5
    for k in np.ndindex(n, D):
        d = np.zeros_like(x)
        d[k] = h
        assert abs((L(x + d, g, b) - L(x - d, g, b)) / (2 * h) - dx[k]) < 1e-7
    for j in range(D):
        d = np.zeros(D)
        d[j] = h
        assert abs((L(x, g + d, b) - L(x, g - d, b)) / (2 * h) - dg[j]) < 1e-8
        assert abs((L(x, g, b + d) - L(x, g, b - d)) / (2 * h) - db[j]) < 1e-8


def test_clip_by_hand():
    norm, coef, out = O.grad_clip([[3.0], [[4.0]], []], 2.5, 0.0)
    assert norm == 5.0 and coef == 0.5 and out[0][0] == 1.5 and out[1][0][0] == 2.0
    assert O.grad_clip([[3.0]], 4.0, 0.0)[1] == 1.0
    assert O.grad_clip([[0.0]], 0.0, 0.0)[1] == 1.0
    assert O.grad_clip([[np.inf]], 4.0, 0.0)[1] == 0.0
