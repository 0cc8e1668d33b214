"""Pins of the 64-bit forms for activations in 8 bits: the formats by listing
their values, the scale's definition, and the gradients by central
differences."""
import numpy as np
import pytest

import oracle.rows8 as O


def e4m3_values():
    """Every finite value of 1 sign, 4 exponent and 3 mantissa bits (bias 7)."""
    v = [m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
         for e in range(16) for m in range(8) if not (e == 15 and m == 7)]
    return np.array(sorted(set(v + [-x for x in v])))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rounding_is_to_the_nearest_value(fmt):
    values = np.arange(-127.0, 128.0) if fmt == "int8" else e4m3_values()
    assert values.max() == O.Q[fmt]
    r = np.random.default_rng(0)
    z = np.concatenate([values, (values[1:] + values[:-1]) / 2, r.uniform(-O.Q[fmt], O.Q[fmt], 3000),
                        r.normal(size=3000) * 0.01])
    got = O.round_to(z, fmt)
    off = np.abs(z[:, None] - values[None, :])
    near = off.min(1)
    assert np.isin(got, values).all()
    assert (np.abs(got - z) <= near * (1 + 1e-12)).all()
    for v, g, o in zip(z, got, off):          # a tie goes to the even one
        tied = values[o == o.min()]
        if len(tied) == 2:
            k = np.flatnonzero(values == g)[0]
            if fmt == "int8":
                assert g % 2 == 0
            else:
                step = abs(tied[1] - tied[0])
                assert (abs(g) / step) % 2 == 0, (v, g, k)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_scale_is_the_least_power_that_fits(fmt):
    r = np.random.default_rng(1)
    x = r.normal(size=(50, 70)) * np.exp(r.uniform(-60, 60, (50, 1)))
    x[3] = 0
    x[4, :32] = O.Q[fmt] * 2.0 ** 5            # on the border
    x[5, :32] = np.nextafter(O.Q[fmt] * 2.0 ** 5, np.inf)
    x[6, 40] = np.nan
    x[7, 69] = -np.inf
    y, q, e = O.held(x, fmt)
    assert e.shape == (50, 3) and e[4, 0] == 132 and e[5, 0] == 133 and (e[3] == 16).all()
    assert e[6, 1] == 255 and e[7, 2] == 255 and np.isnan(y[6, 32:64]).all() and np.isnan(y[7, 64:]).all()
    for g in range(3):
        m = np.abs(x[:, 32 * g:32 * g + 32]).max(1)
        s = np.ldexp(1.0, e[:, g] - 127)
        ok = e[:, g] != 255
        assert (m[ok] <= O.Q[fmt] * s[ok]).all()
        assert (m[ok & (e[:, g] > 16)] > O.Q[fmt] * s[ok & (e[:, g] > 16)] / 2).all()
    fin = np.isfinite(y)
    s = np.ldexp(1.0, np.repeat(e, 32, 1)[:, :70] - 127)
    lim = s / 2 if fmt == "int8" else np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10)
    assert (np.abs(y - x)[fin] <= lim[fin]).all()


def test_rms_gradients_against_differences():
    r = np.random.default_rng(2)
    n, D, eps = 4, 9, 1e-2
    h, w, g, up = r.normal(size=(n, D)), r.normal(size=(n, D)), r.normal(size=D), r.normal(size=(n, D))
    y, rstd = O.rms_fwd(h, g, eps)
    dx, dg = O.rms_bwd(w, h, g, rstd, up)
    loss = lambda h, g: (O.rms_fwd(h, g, eps)[0] * w).sum() + (h * up).sum()  # noqa: E731
    t = 1e-5
    for _ in range(20):
        vh, vg = r.normal(size=(n, D)), r.normal(size=D)
        num = (loss(h + t * vh, g + t * vg) - loss(h - t * vh, g - t * vg)) / (2 * t)
        assert abs(num - ((dx * vh).sum() + (dg * vg).sum())) < 1e-7 * (1 + abs(num))


def test_dense_gradient_against_differences():
    r = np.random.default_rng(3)
    x, dy = r.normal(size=(7, 5)), r.normal(size=(7, 3))
    dw, db, mw, mb = O.dense_bwd(dy, x)
    W, b = r.normal(size=(3, 5)), r.normal(size=3)
    loss = lambda W, b: ((x @ W.T + b) * dy).sum()  # noqa: E731
    vW, vb = r.normal(size=W.shape), r.normal(size=3)
    num = (loss(W + vW, b + vb) - loss(W - vW, b - vb)) / 2      # linear
    assert abs(num - ((dw * vW).sum() + (db * vb).sum())) < 1e-12 * (mw * np.abs(vW)).sum() + 1e-12 * (mb * np.abs(vb)).sum()
