"""Layer norm and its gradient against the 64-bit forms.

Tolerances, u = 2^-24, h = D / 32 + 64 a bound on the additions that any one
summand of a row goes through:
  mean   h u mean|x| + u |mean|
  var    centred on the computed mean: (h + 3) u var + (mean's error)^2
  rstd   half the variance's relative error with eps added, and 3 u
  y      |r gamma| (mean's error) + (4 u + rstd's relative error) |(x - mu) r gamma|
         + 2 u (|y - beta| + |beta|) + the rounding to y's type
  dx     r [4 u |a| + (h + 3) u mean|a| + (h + 8) u |hh| mean|a hh|
         + 4 u (|a| + |mean a| + |hh mean a hh|)] + the rounding
  dgamma (n + 4) u sum|dy hh|, dbeta (n + 1) u sum|dy|, and the rounding."""
import numpy as np
import pytest

import oracle.train_ops as O
from train_ops import TINY, U, U32, assert_close, dtype, f64, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_differentiable_gb300 as m
    return m


def uT(t):
    return U[t] if t != "f32" else 0.0


def fwd_tolerances(x, gamma, beta, eps, t):
    D = x.shape[1]
    h = D / 32 + 64
    y, mean, rstd = O.layer_norm_fwd(x, gamma, beta, eps)
    gamma = np.ones(D) if gamma is None else gamma
    beta = np.zeros(D) if beta is None else beta
    var = ((x - mean[:, None]) ** 2).mean(1)
    em = h * U32 * np.abs(x).mean(1) + U32 * np.abs(mean)
    er = 0.5 * ((h + 3) * U32 + em ** 2 / (var + eps)) + 3 * U32
    core = np.abs((x - mean[:, None]) * rstd[:, None] * gamma)
    ey = np.abs(rstd[:, None] * gamma) * em[:, None] + (4 * U32 + er[:, None]) * core + \
        2 * U32 * (core + np.abs(beta)) + uT(t) * np.abs(y) + TINY[t]
    return (y, mean, rstd), (ey, em, er * rstd)


def param(v, p):
    import torch
    return None if v is None else torch.as_tensor(v, device="cuda").to(dtype(p))


def opt(v):
    return None if v is None else f64(v)


def fwd_case(ss, n, D, t, p, pad, off, eps=1e-5, affine=True, shift=0.5):
    import torch
    r = np.random.default_rng(n * 3 + D)
    x, _ = rows(r.normal(size=(n, D)) * 2 + shift, t, pad, off)
    y, buf = rows(np.zeros((n, D)), t, pad, off, fill=-7.0)
    g = param(1 + 0.3 * r.normal(size=D), p) if affine else None
    b = param(r.normal(size=D), p) if affine else None
    mean, rstd = (torch.empty(n, device="cuda") for _ in range(2))
    ss.ss_layer_norm_fwd(x, g, b, eps, y, mean, rstd)
    want, tol = fwd_tolerances(f64(x), opt(g), opt(b), float(np.float32(eps)), t)
    for got, w, e, what in zip((y, mean, rstd), want, tol, ("y", "mean", "rstd")):
        assert_close(got, w, e, what)
    y0 = y.clone()
    ss.ss_layer_norm_fwd(x, g, b, eps, y, None, None)
    assert torch.equal(y, y0)
    ss.ss_layer_norm_fwd(x, g, b, eps, x, None, None)     # in place
    assert torch.equal(x, y0)
    y.zero_()
    assert ((buf == 0) | (buf == -7.0)).all()


SHAPES = [(1, 1, "f32", "f32", 0, 0), (0, 7, "f32", "f32", 0, 0), (3, 2, "f16", "f32", 0, 0),
          (1000, 3, "f32", "f32", 0, 0), (333, 16, "bf16", "bf16", 0, 0),
          (777, 48, "f32", "f32", 0, 0), (777, 48, "bf16", "f32", 0, 0), (50, 48, "f32", "f32", 1, 0),
          (129, 50, "f32", "f32", 0, 0), (100, 64, "f16", "f16", 8, 0), (100, 64, "f32", "f32", 4, 1),
          (65, 100, "bf16", "f32", 0, 1), (31, 127, "f32", "f32", 0, 0), (70, 128, "bf16", "bf16", 0, 0),
          (37, 1001, "f16", "f16", 0, 0), (40, 1000, "bf16", "f32", 0, 0), (33, 1024, "f32", "f32", 0, 0),
          (19, 2000, "f16", "f32", 0, 0), (17, 4096, "bf16", "f32", 0, 0), (9, 5001, "f32", "f32", 0, 0),
          (7, 8192, "f32", "f32", 0, 0), (5, 16384, "bf16", "bf16", 0, 0), (3, 20001, "f16", "f32", 0, 0),
          (2, 32768, "f32", "f32", 0, 0), (2, 65536, "bf16", "f32", 0, 0), (4, 65535, "f32", "f32", 0, 0)]


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_forward(ss, case):
    fwd_case(ss, *case)


def test_forward_without_weights(ss):
    fwd_case(ss, 40, 96, "f32", "f32", 0, 0, affine=False)
    fwd_case(ss, 40, 8192, "bf16", "f32", 0, 0, affine=False)


@pytest.mark.parametrize("D", [48, 1001, 4096])
def test_large_mean(ss, D):
    """A mean a thousand times the spread: moments would lose the variance."""
    fwd_case(ss, 20, D, "f32", "f32", 0, 0, shift=2000.0)


@pytest.mark.parametrize("D", [1, 48, 1001, 9000])
def test_constant_rows_and_zero_eps(ss, D):
    """A row without variance: rstd = eps^-1/2, y = beta; NaN and infinite
    values stay in their rows."""
    import torch
    x = torch.ones(5, D, device="cuda") * 3
    x[1] = float("nan")
    x[2, 0] = float("inf")
    b = torch.linspace(-1, 1, D, device="cuda")
    ln = ss.LayerNorm(5, D, eps=0.25)
    y = ln.forward(x, None, b)
    for k in (0, 3, 4):
        assert torch.equal(y[k], b) and float(ln.mean[k]) == 3.0 and float(ln.rstd[k]) == 2.0
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).any()
    ln.eps = 0.0
    ln.forward(x, None, None)
    assert torch.isinf(ln.rstd[0])


def bwd_case(ss, n, D, t, p, pad, off, affine=True, inplace=None):
    import torch
    r = np.random.default_rng(n * 5 + D)
    x, _ = rows(r.normal(size=(n, D)) * 2 + 0.5, t, pad, off)
    dy, _ = rows(r.normal(size=(n, D)), t, pad, off)
    dx, buf = rows(np.zeros((n, D)), t, pad, off, fill=-7.0)
    g = param(1 + 0.3 * r.normal(size=D), p) if affine else None
    x64, dy64, g64 = f64(x), f64(dy), opt(g)
    _, mean, rstd = O.layer_norm_fwd(x64, None, None, 1e-5)
    mean, rstd = (torch.as_tensor(v, device="cuda").float() for v in (mean, rstd))
    dg, db = (torch.full((D,), 9.0, dtype=dtype(p), device="cuda") for _ in range(2))
    ws = torch.empty(ss.ss_layer_norm_workspace_bytes(n, D), dtype=torch.uint8, device="cuda").fill_(0xA5)
    m64, r64 = f64(mean), f64(rstd)
    wdx, wdg, wdb = O.layer_norm_bwd(dy64, x64, g64, m64, r64)
    ss.ss_layer_norm_bwd(dy, x, g, mean, rstd, dx, dg, db, ws)
    h = D / 32 + 64
    a = dy64 * (1.0 if g64 is None else g64)
    hh = (x64 - m64[:, None]) * r64[:, None]
    mean_ = lambda v: v.mean(1, keepdims=True) if n else v[:, :1]  # noqa: E731
    ma, mah = mean_(a), mean_(a * hh)
    tol = r64[:, None] * (4 * U32 * np.abs(a) + (h + 3) * U32 * mean_(np.abs(a)) +
                          (h + 8) * U32 * np.abs(hh) * mean_(np.abs(a * hh)) +
                          4 * U32 * (np.abs(a) + np.abs(ma) + np.abs(hh * mah))) + \
        uT(t) * np.abs(wdx) + TINY[t]
    assert_close(dx, wdx, tol, "dx")
    tg = (n + 4) * U32 * np.abs(dy64 * hh).sum(0) + uT(p) * np.abs(wdg) + TINY[p]
    tb = (n + 1) * U32 * np.abs(dy64).sum(0) + uT(p) * np.abs(wdb) + TINY[p]
    assert_close(dg, wdg, tg, "dgamma")
    assert_close(db, wdb, tb, "dbeta")
    first = [v.clone() for v in (dx, dg, db)]
    into = dx if inplace is None else (dy if inplace == "dy" else x)
    ss.ss_layer_norm_bwd(dy, x, g, mean, rstd, into, dg, db, ws)
    for v, w in zip((into, dg, db), first):
        assert torch.equal(v, w)                     # the same bits, in place too
    if inplace is None:
        ss.ss_layer_norm_bwd(dy, x, g, mean, rstd, dx, None, None, None)
        assert torch.equal(dx, first[0])
    dx.zero_()
    assert ((buf == 0) | (buf == -7.0)).all()


@pytest.mark.parametrize("case", SHAPES + [(5000, 48, "f32", "f32", 0, 0), (6001, 7, "bf16", "bf16", 0, 0),
                                           (2000, 1000, "bf16", "bf16", 0, 0), (701, 513, "f32", "f32", 0, 0)],
                         ids=lambda c: "-".join(map(str, c)))
def test_backward(ss, case):
    bwd_case(ss, *case)


@pytest.mark.parametrize("inplace", ["dy", "x"])
@pytest.mark.parametrize("n,D,t", [(300, 48, "f32"), (40, 1001, "f16"), (20, 4096, "bf16"), (3, 40000, "f32")])
def test_backward_in_place(ss, n, D, t, inplace):
    bwd_case(ss, n, D, t, "f32", 0, 0, inplace=inplace)


def test_backward_without_weights(ss):
    bwd_case(ss, 77, 48, "f32", "f32", 0, 0, affine=False)


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [1, 9, 48, 257, 1000, 3001])
def test_tensors_that_start_differently(ss, D, t):
    """Each tensor with its own offset and stride: the same values as from
    tensors that all start on boundaries."""
    import torch
    r = np.random.default_rng(D)
    n = 45
    xv, dv = r.normal(size=(n, D)), r.normal(size=(n, D))
    plain = [rows(v, t)[0] for v in (xv, dv)]
    ln = ss.LayerNorm(n, D, dtype=dtype(t))
    g = torch.as_tensor(1 + 0.3 * r.normal(size=D), device="cuda").float()
    y = ln.forward(plain[0], g)
    dx = ln.backward(plain[1], plain[0], g)
    want = [f64(v) for v in (y, dx, ln.grads["dgamma"], ln.grads["dbeta"])]
    (_, _, _), (ey, _, _) = fwd_tolerances(f64(plain[0]), f64(g), None, 1e-5, t)
    x, _ = rows(xv, t, pad=3, offset=1)
    dy, _ = rows(dv, t, pad=1, offset=2)
    out, buf = rows(np.zeros((n, D)), t, pad=5, offset=3, fill=-7.0)
    ss.ss_layer_norm_fwd(x, g, None, ln.eps, out)
    assert_close(out, want[0], 2 * ey, "y")
    dg, db = torch.empty_like(g), torch.empty_like(g)
    ss.ss_layer_norm_bwd(dy, x, g, ln.mean, ln.rstd, out, dg, db, ln.workspace)
    # two float32 evaluations of sums of at most max(n, D) terms, and two roundings to the type
    h = (D / 32 + 80) * U32
    scale = np.abs(f64(ln.rstd))[:, None] * (np.abs(dv) + np.abs(dv).mean(1, keepdims=True)) * 4 * \
        (1 + np.abs(f64(plain[0])) ** 2)
    assert_close(out, want[1], 2 * h * scale + 2 * uT(t) * np.abs(want[1]) + TINY[t], "dx")
    hh = np.abs((f64(plain[0]) - f64(ln.mean)[:, None]) * f64(ln.rstd)[:, None])
    assert_close(dg, want[2], 2 * (n + 4) * U32 * (np.abs(dv) * hh).sum(0) * 1.01, "dgamma")
    assert_close(db, want[3], 2 * (n + 4) * U32 * np.abs(dv).sum(0) * 1.01, "dbeta")
    out.zero_()
    assert ((buf == 0) | (buf == -7.0)).all()


@pytest.mark.parametrize("D", [5, 48, 1001])
def test_gradient_against_differences(ss, D):
    """The kernel's gradients along a direction against central differences of
    the 64-bit forward; the step's own error is h^2 / 6 of the third
    derivative, taken from a step twice as long."""
    import torch
    r = np.random.default_rng(D)
    n, eps = 6, 1e-2
    x, w = r.normal(size=(n, D)).astype(np.float32), r.normal(size=(n, D)).astype(np.float32)
    g, b = r.normal(size=D).astype(np.float32), r.normal(size=D).astype(np.float32)
    c = lambda v: torch.as_tensor(v, device="cuda")  # noqa: E731
    ln = ss.LayerNorm(n, D, eps=eps)
    ln.forward(c(x), c(g), c(b))
    dx = f64(ln.backward(c(w), c(x), c(g)))
    dg, db = f64(ln.grads["dgamma"]), f64(ln.grads["dbeta"])
    vx, vg, vb = r.normal(size=(n, D)), r.normal(size=D), r.normal(size=D)
    e32 = float(np.float32(eps))

    def slope(s):
        L = [(O.layer_norm_fwd(x + q * vx, g + q * vg, b + q * vb, e32)[0] * w.astype(np.float64)).sum()
             for q in (s, -s)]
        return (L[0] - L[1]) / (2 * s)
    a, a2 = slope(1e-4), slope(2e-4)
    got = (dx * vx).sum() + (dg * vg).sum() + (db * vb).sum()
    scale = (np.abs(dx * vx).sum() + np.abs(dg * vg).sum() + np.abs(db * vb).sum())
    assert abs(got - a) <= abs(a2 - a) + (D / 32 + 100) * U32 * scale + 1e-9


def test_offsets_past_32_bits(ss):
    import torch
    stride = (1 << 30) + 8
    buf = torch.empty(3 * stride + 64, dtype=torch.bfloat16, device="cuda")
    big = torch.as_strided(buf, (4, 64), (stride, 1))
    small = torch.randn(4, 64, device="cuda").bfloat16()
    big.copy_(small)
    a, b = ss.LayerNorm(4, 64, dtype=torch.bfloat16), ss.LayerNorm(4, 64, dtype=torch.bfloat16)
    assert torch.equal(a.forward(small), b.forward(big))
    assert torch.equal(a.backward(small, small), b.backward(big, big))
    ss.ss_layer_norm_fwd(small, None, None, 1e-5, big)
    assert torch.equal(big, a.y)


def test_another_stream_and_a_captured_graph(ss):
    import torch
    x, dy = torch.randn(500, 48, device="cuda"), torch.randn(500, 48, device="cuda")
    ln = ss.LayerNorm(500, 48)
    ln.forward(x)
    want = [v.clone() for v in (ln.y, ln.backward(dy, x), ln.grads["dgamma"], ln.grads["dbeta"])]
    have = (ln.y, ln.dx, ln.grads["dgamma"], ln.grads["dbeta"])
    s = torch.cuda.Stream()
    for v in have:
        v.fill_(3)
    s.wait_stream(torch.cuda.current_stream())
    ln.forward(x, stream=s)
    ln.backward(dy, x, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(have, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ln.forward(x)
        ln.backward(dy, x)
    for _ in range(3):
        for v in have:
            v.fill_(3)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(have, want))


def test_binding_checks(ss):
    import torch
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError, match="gamma"):
        ss.ss_layer_norm_fwd(x, torch.zeros(7, device="cuda"), None, 1e-5, torch.empty_like(x))
    with pytest.raises(ValueError, match="one type"):
        h = x.half()
        ss.ss_layer_norm_fwd(h, torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda").half(),
                             1e-5, torch.empty_like(h))
    with pytest.raises(ValueError, match="mean"):
        ss.ss_layer_norm_fwd(x, None, None, 1e-5, torch.empty_like(x), torch.zeros(3, device="cuda"))
    ln = ss.LayerNorm(4, 8)
    with pytest.raises(ValueError, match="x must be"):
        ln.forward(x[:3])
    with pytest.raises(ValueError, match="x must be torch.float32"):
        ln.forward(x.half())
    with pytest.raises(ValueError, match="gamma must be torch.float32"):
        ln.forward(x, torch.zeros(8, device="cuda").half())
    with pytest.raises(ValueError, match="dy must be"):
        ln.backward(torch.zeros(4, 7, device="cuda"), x)
    with pytest.raises(ValueError, match="mean"):
        ln.backward(x, x, mean=torch.zeros(5, device="cuda"))
    with pytest.raises(ValueError, match="param_dtype"):
        ss.LayerNorm(4, 8, dtype=torch.float16, param_dtype=torch.bfloat16)
