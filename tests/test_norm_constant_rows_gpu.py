"""Layer norm of rows that hold one value, or nearly one: the deviations from
the mean are zero (or a few units of the last place), whatever the width and
however large the value, so that an error of the mean, which 1 / sqrt(eps)
would amplify, shows.

What is expected, u = 2^-24, h = D / 32 + 64 a bound on the additions that any
one summand of a row goes through.  The float32 mean is off by at most
d = (h + 2) u |c|.  While |mean| rstd <= 8 that is all: y is off by d rstd |gamma|
and two roundings, the variance by d^2.  Above (a constant c comes there from
0.036 on, eps^1/2 times 8 and d^2 <= eps or far larger) it is put right: it is a
whole number k <= h + 2 of units of c's last place, so the deviations x - mean
are exact (the two lie within a factor of two) and equal; their sum is exact
while D k < 2^24 (D <= 9000 here), and so is its quotient by D, which takes
them off again: y is beta bit for bit, and mean is c.  The variance is then off
by (h + 3) u d^2 (at most h additions and three roundings of what its two parts
leave of one another), and rstd by half of that over eps and 3 u, relative.
In 16 bits the sums themselves are exact, and the quotient is c."""
import numpy as np
import pytest

import oracle.train_ops as O
from train_ops import U, U32, assert_close, dtype, f64, rows

pytestmark = pytest.mark.gpu
EPS = 1e-5
WIDTHS = [1, 3, 41, 47, 61, 82, 83, 97, 164, 188, 333, 1001, 2044, 4097, 8191, 9000]


@pytest.fixture(scope="module")
def ss():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_differentiable_gb300 as m
    return m


def run(ss, values, D, t, pad, affine=True):
    """(y, mean, rstd, beta in the type of y) of rows that each hold one value."""
    import torch
    x, _ = rows(np.repeat(np.asarray(values)[:, None], D, 1), t, pad)
    y, _ = rows(np.zeros(x.shape), t, pad)
    g = torch.linspace(-3, 3, D, device="cuda") if affine else None
    b = torch.linspace(1, 2, D, device="cuda") if affine else None
    mean, rstd = (torch.empty(len(values), device="cuda") for _ in range(2))
    ss.ss_layer_norm_fwd(x, g, b, EPS, y, mean, rstd)
    b = torch.zeros(D, device="cuda") if b is None else b
    return x, y, mean, rstd, b.to(dtype(t))


# values that the type holds exactly
VALUES = {"f32": [0.0, 1.0, -1e3, 1e4, 1e6, -0.1, 100 / 3, 12345.678, 1e-3, 3e7],
          "f16": [0.0, 1.0, -1e3, 2049.0 - 1, 60000.0, 0.1, 3.3],
          "bf16": [0.0, 1.0, -1e3, 9984.0, 999424.0, 0.1, 3.3]}


@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_constant_rows(ss, D, t, pad):
    import torch
    x, y, mean, rstd, beta = run(ss, VALUES[t], D, t, pad)
    c = f64(x[:, 0])
    far = np.abs(c) > 0.036
    assert torch.equal(y[far], beta.expand_as(y)[far]), float((y - beta)[far].abs().max())
    assert torch.equal(mean[far], x[far, 0].float())
    h = D / 32 + 64
    d = (h + 2) * U32 * np.abs(c)
    want = np.full(len(mean), 1 / np.sqrt(float(np.float32(EPS))))
    b = np.broadcast_to(f64(beta), y.shape)
    tol = 3 * d[:, None] * want[:, None] + (2 * U32 + (U[t] if t != "f32" else 0)) * np.abs(b)
    assert_close(f64(y)[~far], b[~far], tol[~far], "y")
    assert_close(f64(mean)[~far], c[~far], d[~far], "mean")
    tol = (0.5 * np.where(far, (h + 3) * U32, 1) * d ** 2 / EPS + 4 * U32) * want
    small = d < 1e-3                       # where the bound says something of rstd
    assert_close(f64(rstd)[small], want[small], tol[small], "rstd")


@pytest.mark.parametrize("D", [41, 61, 1001, 9000])
def test_constant_rows_have_no_gradient_through_the_norm(ss, D):
    """h = 0 and rstd = eps^-1/2: dx = rstd (a - mean a), dgamma = 0 exactly."""
    import torch
    r = np.random.default_rng(D)
    x = torch.tensor([1e4, -1e6, 1e3], device="cuda")[:, None].repeat(1, D)
    dy = torch.as_tensor(r.normal(size=(3, D)), device="cuda").float()
    ln = ss.LayerNorm(3, D, eps=EPS)
    ln.forward(x)
    dx = ln.backward(dy, x)
    assert (ln.grads["dgamma"] == 0).all()
    r64 = f64(ln.rstd)
    want = O.layer_norm_bwd(f64(dy), f64(x), None, f64(ln.mean), r64)[0]
    a = np.abs(f64(dy))
    tol = r64[:, None] * U32 * (4 * a + (D / 32 + 70) * a.mean(1, keepdims=True))
    assert_close(dx, want, tol, "dx")


@pytest.mark.parametrize("D", [61, 164, 333, 1001, 4097, 9000])
def test_a_small_spread_about_a_large_value(ss, D):
    """Rows c + (-1, 0 or 1 units of c's last place).  As above the deviations
    from the first mean and their sum are exact, at most d + 1 unit and D times
    that; their mean has one rounding, and taking it off another: u (|dev| + d).
    The squares' mean is off by (h + 6) u (d + 1 unit)^2, rstd by half of that
    times rstd^2 and 3 u, relative; y has two roundings more."""
    import torch
    c = np.array([1e3, 5e3, 1e4, 12345.678], dtype=np.float32)
    unit = np.spacing(c)
    r = np.random.default_rng(D)
    v = (c[:, None] + r.integers(-1, 2, (4, D)) * unit[:, None]).astype(np.float32)
    ln = ss.LayerNorm(4, D, eps=EPS)
    y = f64(ln.forward(torch.as_tensor(v, device="cuda")))
    want, _, rstd = O.layer_norm_fwd(v, None, None, float(np.float32(EPS)))
    h = D / 32 + 64
    d = (h + 1) * U32 * c.astype(np.float64)
    rel = 0.5 * (h + 6) * U32 * (d + unit) ** 2 * rstd ** 2 + 3 * U32
    tol = (rel + 3 * U32)[:, None] * np.abs(want) + (rstd * U32 * d)[:, None]
    assert_close(y, want, tol, "y")
