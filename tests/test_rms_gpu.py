"""Root-mean-square norm, its gradient, and the layer norm's gradient from rows
in 8 bits, against the 64-bit forms.

Tolerances, u = 2^-24, h = D / 32 + 64 a bound on the additions that any one
summand of a row goes through:
  sum    none: one rounding (a float32 sum of two 16-bit values is rounded to 16
         bits as the exact one is: 24 >= 2 p + 2 bits)
  rstd   half the mean square's relative error (h + 3) u, and 3 u
  y      rstd's relative error and 3 u, of |y|, and the rounding to y's type
  8 bits as y, and half a step of the format at the scale that y, enlarged by its
         error, has; and where y is wanted in float32 too, exactly what packing it gives
  dx     with g = h r (the centred h for the layer norm): r [4 u |a| + (h + 3) u mean|a| (layer
         norm) + (h + 8) u |g| mean|a g| + 4 u (|a| + |mean a| + |g mean a g|)] + u |dx| with
         dsum, and the rounding
  dgamma (n + 4) u sum|dy g|, dbeta (n + 1) u sum|dy|, and the rounding."""
import numpy as np
import pytest

import oracle.rows8 as O
import oracle.train_ops as T
from rows8_data import FORMATS, Guarded, torch_format
from train_ops import TINY, U, U32, assert_close, dtype, f64, rows

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def ss():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_differentiable_gb300 as m
    return m


def uT(t):
    return U[t] if t != "f32" else 0.0


def param(v, p):
    import torch
    return None if v is None else torch.as_tensor(v, device="cuda").to(dtype(p))


def opt(v):
    return None if v is None else f64(v)


def values(r, n, D):
    x = r.normal(size=(n, D)) * np.exp(r.uniform(-3, 3, (n, 1)))
    if n > 2:
        x[1] = 0.0
    return x


# (n, D, type, weights' type, unused values after a row, values before the first)
SHAPES = [(1, 1, "f32", "f32", 0, 0), (0, 7, "f32", "f32", 0, 0), (3, 2, "f16", "f32", 0, 0),
          (1000, 3, "f32", "f32", 0, 0), (333, 16, "bf16", "bf16", 0, 0), (200, 24, "bf16", "f32", 0, 0),
          (777, 48, "f32", "f32", 0, 0), (777, 48, "bf16", "f32", 0, 0), (50, 48, "f32", "f32", 1, 0),
          (51, 33, "f16", "f16", 0, 0), (129, 50, "f32", "f32", 0, 0), (100, 64, "f16", "f16", 8, 0),
          (100, 64, "f32", "f32", 4, 1), (65, 100, "bf16", "f32", 0, 1), (31, 127, "f32", "f32", 0, 0),
          (70, 128, "bf16", "bf16", 0, 0), (90, 256, "f32", "f32", 0, 0), (60, 511, "bf16", "f32", 0, 0),
          (37, 1001, "f16", "f16", 0, 0), (40, 1000, "bf16", "f32", 0, 0), (33, 1024, "f32", "f32", 0, 0),
          (19, 2000, "f16", "f32", 0, 0), (1, 4096, "bf16", "bf16", 0, 0), (17, 4096, "bf16", "f32", 0, 0),
          (9, 5001, "f32", "f32", 0, 0), (7, 8192, "f32", "f32", 0, 0), (7, 8191, "bf16", "bf16", 1, 0),
          (6, 8193, "f16", "f32", 0, 0), (5, 16384, "bf16", "bf16", 0, 0), (3, 20001, "f16", "f32", 0, 0),
          (2, 65536, "bf16", "f32", 0, 0), (3, 65535, "f32", "f32", 0, 0)]


def half_step(y, s, fmt):
    """Half the distance of the format's values next to y at scales s."""
    if fmt == "int8":
        return s / 2
    return np.maximum(np.abs(y) * 2.0 ** -4, s * 2.0 ** -10)


def scales_of(y, fmt):
    e = np.repeat(O.scale_exponents(y, fmt), 32, axis=1)[:, :y.shape[1]]
    return np.ldexp(1.0, e - 127)


def fwd_case(ss, n, D, t, p, pad, off, residual=True, affine=True, fmts=("e4m3", "int8"), eps=EPS):
    import torch
    r = np.random.default_rng(n * 3 + D)
    x, _ = rows(values(r, n, D), t, pad, off)
    res = rows(values(r, n, D), t, pad, off)[0] if residual else None
    g = param(1 + 0.3 * r.normal(size=D), p) if affine else None
    y, ybuf = rows(np.zeros((n, D)), t, pad, off, fill=-7.0)
    sm, sbuf = rows(np.zeros((n, D)), t, pad, off, fill=-7.0)
    out, kept = Guarded(ss, n, D, fmts[0], 8, 1), Guarded(ss, n, D, fmts[1])
    rstd = torch.empty(n, device="cuda")
    x0 = x.clone()
    ss.ss_rms_norm_fwd(x, res, g, eps, sm if residual else None, y, out.rows, kept.rows, rstd)
    assert torch.equal(x, x0)
    want_sum = f64((x.double() + res.double()).to(x.dtype)) if residual else f64(x)
    if residual:
        assert_close(sm, want_sum, 0.0, "sum")
    h = D / 32 + 64
    want, want_r = O.rms_fwd(want_sum, opt(g), float(np.float32(eps)))
    er = 0.5 * (h + 3) * U32 + 3 * U32
    assert_close(rstd, want_r, er * want_r, "rstd")
    ey = (er + 3 * U32) * np.abs(want)
    assert_close(y, want, ey + uT(t) * np.abs(want) + TINY[t], "y")
    # kept: the rounded sum, so every bit
    kept.check_untouched()
    assert np.array_equal(f64(kept.rows.unpack(torch.empty(n, D, device="cuda"))), O.held(want_sum, fmts[1])[0])
    out.check_untouched()
    got = f64(out.rows.unpack(torch.empty(n, D, device="cuda")))
    if t == "f32":
        assert np.array_equal(got, O.held(f64(y), fmts[0])[0])
    lim = np.abs(want) + ey
    assert_close(got, want, half_step(lim, scales_of(lim, fmts[0]), fmts[0]) + ey, "y in 8 bits")
    # the 8-bit outputs by themselves give the same bits; y without them may sum a row that does not
    # start on a boundary in another order, and then both are as near as they have to be; in place the same bits
    y0, o0 = y.clone(), out.rows.q.float().clone()
    only = Guarded(ss, n, D, fmts[0])
    ss.ss_rms_norm_fwd(x, res, g, eps, sm if residual else None, out=only.rows)
    assert torch.equal(only.rows.q.float(), o0) and torch.equal(only.rows.scales, out.rows.scales)
    ss.ss_rms_norm_fwd(x, res, g, eps, sm if residual else None, y)
    assert_close(y, want, ey + uT(t) * np.abs(want) + TINY[t], "y alone")
    if D * y.element_size() % 32 == 0 and pad % 8 == 0 and off % 8 == 0:
        assert torch.equal(y, y0)
    y0 = y.clone()
    if residual:
        s0 = sm.clone()
        x2, r2 = rows(x0, t, pad, off)[0], rows(res, t, pad, off)[0]
        ss.ss_rms_norm_fwd(x2, r2, g, eps, x2, r2)            # sum over x, y over the residual
        assert torch.equal(x2, s0) and torch.equal(r2, y0)
        x2 = rows(x0, t, pad, off)[0]
        ss.ss_rms_norm_fwd(x2, res, g, eps, sm, x2)
        assert torch.equal(x2, y0) and torch.equal(sm, s0)
    else:
        ss.ss_rms_norm_fwd(x, None, g, eps, None, x)
        assert torch.equal(x, y0)
    for v, b in ((y, ybuf), (sm, sbuf)):
        v.zero_()
        assert ((b == 0) | (b == -7.0)).all()


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_forward(ss, case):
    fwd_case(ss, *case)


@pytest.mark.parametrize("n,D,t", [(40, 48, "f32"), (41, 96, "bf16"), (21, 1001, "f16"), (9, 4096, "bf16"),
                                   (3, 20000, "f32")])
def test_forward_without_residual_or_weights(ss, n, D, t):
    fwd_case(ss, n, D, t, "f32", 0, 0, residual=False, fmts=("int8", "e4m3"))
    fwd_case(ss, n, D, t, "f32", 0, 0, residual=False, affine=False, fmts=("int8", "int8"))
    fwd_case(ss, n, D, t, "f32", 0, 0, affine=False, fmts=("e4m3", "e4m3"))


@pytest.mark.parametrize("D", [1, 48, 1001, 9000])
def test_rows_that_are_not_finite_and_zero_eps(ss, D):
    """They stay in their rows; a row of zeros without eps has no norm."""
    import torch
    x = torch.ones(6, D, device="cuda") * 3
    x[1] = float("nan")
    x[2, 0] = float("inf")
    x[3] = 0
    m = ss.RMSNorm(6, D, eps=0.0)
    y = m.forward(x)
    for k in (0, 4, 5):
        assert torch.allclose(y[k], torch.ones(D, device="cuda"), rtol=1e-6, atol=0)
        assert float(m.rstd[k]) == pytest.approx(1 / 3, rel=1e-6)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 0]) and (y[2, 1:] == 0).all()
    assert torch.isinf(m.rstd[3]) and torch.isnan(y[3]).all()
    m8 = ss.RMSNorm(6, D, eps=0.25, out=torch.float8_e4m3fn, keep=torch.int8)
    o = m8.forward(x)
    got = o.unpack(torch.empty(6, D, device="cuda"))
    assert torch.isnan(got[1]).all() and torch.isnan(got[2, :32]).all() and (got[3] == 0).all()
    assert (got[2, 32:] == 0).all() and torch.isfinite(got[[0, 4, 5]]).all()
    kept = m8.kept.unpack(got)
    assert torch.isnan(kept[2, :32]).all() and (kept[2, 32:] == 3).all() and (kept[0] == 3).all()


def bwd_case(ss, n, D, t, p, pad, off, kind="rms", source="int8", dsum=True, affine=True, inplace=None):
    import torch
    r = np.random.default_rng(n * 5 + D)
    x, _ = rows(values(r, n, D) + (0.5 if kind == "ln" else 0.0), t, pad, off)
    dy, _ = rows(r.normal(size=(n, D)), t, pad, off)
    up = rows(r.normal(size=(n, D)), t, pad, off)[0] if dsum and kind == "rms" else None
    dx, buf = rows(np.zeros((n, D)), t, pad, off, fill=-7.0)
    g = param(1 + 0.3 * r.normal(size=D), p) if affine else None
    if source == "rows":
        src, x64 = x, f64(x)
    else:
        src = Guarded(ss, n, D, source, 8, 3).rows.pack(x)
        x64 = f64(src.unpack(torch.empty(n, D, device="cuda")))
    if kind == "rms":
        mean, rstd = None, O.rms_fwd(f64(x), None, EPS)[1]
    else:
        _, mean, rstd = T.layer_norm_fwd(f64(x), None, None, EPS)
        mean = torch.as_tensor(mean, device="cuda").float()
    rstd = torch.as_tensor(rstd, device="cuda").float()
    r64, dy64, g64 = f64(rstd), f64(dy), opt(g)
    dg, db = (torch.full((D,), 9.0, dtype=dtype(p), device="cuda") for _ in range(2))
    size = ss.ss_rms_norm_workspace_bytes(n, D)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xA5)
    ln = None
    if kind == "ln":
        ln = ss.LayerNorm(n, D, dtype=dtype(t), param_dtype=dtype(p), forward=False)
        wdx, wdg, wdb = T.layer_norm_bwd(dy64, x64, g64, f64(mean), r64)
        hh = (x64 - f64(mean)[:, None]) * r64[:, None]
    else:
        wdx, wdg = O.rms_bwd(dy64, x64, g64, r64, opt(up))
        hh = x64 * r64[:, None]

    def call(into, weights=True):
        if kind == "ln":                       # its own dx; strides of dx by the C ABI below
            ws8 = ln.workspace
            st = ss._L.ss_layer_norm_bwd8(dy.data_ptr(), dy.stride(0) if n > 1 else D + pad, src.c, ss._dtype(dy, "dy"),
                                          n, D, None if g is None else g.data_ptr(), ss.DTYPE_CODES[dtype(p)],
                                          mean.data_ptr(), rstd.data_ptr(), into.data_ptr(),
                                          into.stride(0) if n > 1 else D + pad, dg.data_ptr() if weights else None,
                                          db.data_ptr() if weights else None, ws8.data_ptr(), ws8.nbytes, ss._stream(None))
            ss._check(st, "ss_layer_norm_bwd8")
        else:
            ss.ss_rms_norm_bwd(dy, src, g, rstd, up, into, dg if weights else None, ws)
    call(dx)
    h = D / 32 + 64
    a = dy64 * (1.0 if g64 is None else g64)
    mean_ = lambda v: v.mean(1, keepdims=True) if n else v[:, :1]  # noqa: E731
    ma = mean_(a) if kind == "ln" else 0.0
    mah = mean_(a * hh)
    tol = r64[:, None] * (4 * U32 * np.abs(a) + (h + 3) * U32 * (mean_(np.abs(a)) if kind == "ln" else 0.0) +
                          (h + 8) * U32 * np.abs(hh) * mean_(np.abs(a * hh)) +
                          4 * U32 * (np.abs(a) + np.abs(ma) + np.abs(hh * mah))) + \
        (2 * U32 * (np.abs(wdx) + np.abs(opt(up))) if up is not None else 0.0) + uT(t) * np.abs(wdx) + TINY[t]
    assert_close(dx, wdx, tol, "dx")
    tg = (n + 4) * U32 * np.abs(dy64 * hh).sum(0) + uT(p) * np.abs(wdg) + TINY[p]
    assert_close(dg, wdg, tg, "dgamma")
    first = [dx.clone(), dg.clone()]
    if kind == "ln":
        assert_close(db, wdb, (n + 1) * U32 * np.abs(dy64).sum(0) + uT(p) * np.abs(wdb) + TINY[p], "dbeta")
    into = {None: dx, "dy": dy, "dsum": up, "h": x if source == "rows" else dx}[inplace]
    call(into)
    assert torch.equal(into, first[0]) and torch.equal(dg, first[1])      # the same bits, in place too
    if inplace is None:
        dg.fill_(9.0)
        call(dx, weights=False)
        assert torch.equal(dx, first[0]) and (dg == 9.0).all()
    dx.zero_()
    assert ((buf == 0) | (buf == -7.0)).all()


MORE = [(0, 48, "bf16", "bf16", 0, 0), (5000, 48, "f32", "f32", 0, 0), (4000, 35, "bf16", "f32", 0, 0), (900, 505, "f16", "f16", 0, 1),
        (300, 8185, "bf16", "f32", 0, 0), (250, 4100, "f32", "f32", 4, 0), (40, 8184, "f32", "f32", 8, 0), (6001, 7, "bf16", "bf16", 0, 0), (2000, 1000, "bf16", "bf16", 0, 0),
        (701, 513, "f32", "f32", 0, 0), (1500, 1001, "bf16", "bf16", 0, 0), (3000, 90, "f16", "f32", 3, 1)]


@pytest.mark.parametrize("case", SHAPES + MORE, ids=lambda c: "-".join(map(str, c)))
def test_backward_from_int8(ss, case):
    bwd_case(ss, *case)


@pytest.mark.parametrize("case", SHAPES[::2] + MORE, ids=lambda c: "-".join(map(str, c)))
def test_backward_from_e4m3(ss, case):
    bwd_case(ss, *case, source="e4m3", dsum=False)


@pytest.mark.parametrize("case", SHAPES[1::2] + MORE, ids=lambda c: "-".join(map(str, c)))
def test_backward_from_rows(ss, case):
    bwd_case(ss, *case, source="rows")


@pytest.mark.parametrize("case", SHAPES + MORE, ids=lambda c: "-".join(map(str, c)))
def test_layer_norm_backward_in_8_bits(ss, case):
    bwd_case(ss, *case, kind="ln", source="int8" if case[1] % 2 else "e4m3")


@pytest.mark.parametrize("inplace", ["dy", "dsum", "h"])
@pytest.mark.parametrize("n,D,t", [(300, 48, "f32"), (40, 1001, "f16"), (20, 4096, "bf16"), (3, 40000, "f32")])
def test_backward_in_place(ss, n, D, t, inplace):
    bwd_case(ss, n, D, t, "f32", 0, 0, source="rows", inplace=inplace)
    if inplace != "h":
        bwd_case(ss, n, D, t, "f32", 0, 0, source="int8", inplace=inplace)


def test_backward_without_weights(ss):
    bwd_case(ss, 77, 48, "f32", "f32", 0, 0, affine=False)
    bwd_case(ss, 77, 48, "f32", "f32", 0, 0, affine=False, kind="ln")


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [1, 9, 48, 257, 1000, 3001])
def test_tensors_that_start_differently(ss, D, t):
    """Each tensor with its own offset and stride: the same bits from the forward, which
    sums a row in one order whatever its place."""
    import torch
    r = np.random.default_rng(D)
    n = 45
    xv, rv, dv, uv = (r.normal(size=(n, D)) for _ in range(4))
    x, res, dy, up = (rows(v, t)[0] for v in (xv, rv, dv, uv))
    g = torch.as_tensor(1 + 0.3 * r.normal(size=D), device="cuda").float()
    m = ss.RMSNorm(n, D, dtype=dtype(t), residual=True, keep=torch.int8)
    y = m.forward(x, g, res)
    dx = m.backward(dy, m.sum, g, up)
    x2, r2 = rows(xv, t, 3, 1)[0], rows(rv, t, 1, 2)[0]
    s2, sb = rows(np.zeros((n, D)), t, 5, 3, fill=-7.0)
    y2, yb = rows(np.zeros((n, D)), t, 2, 7, fill=-7.0)
    k2 = ss.Rows8(n, D)
    ss.ss_rms_norm_fwd(x2, r2, g, m.eps, s2, y2, None, k2)
    assert torch.equal(s2, m.sum) and torch.equal(k2.q, m.kept.q) and torch.equal(k2.scales, m.kept.scales)
    e = (D / 32 + 80) * U32
    assert_close(y2, f64(y), 2 * (e + uT(t)) * np.abs(f64(y)) + TINY[t], "y")
    dy2, u2 = rows(dv, t, 7, 1)[0], rows(uv, t, 0, 3)[0]
    dx2, db = rows(np.zeros((n, D)), t, 1, 1, fill=-7.0)
    dg2 = torch.empty_like(g)
    ss.ss_rms_norm_bwd(dy2, s2, g, m.rstd, u2, dx2, dg2, m.workspace)
    hh = np.abs(f64(m.sum) * f64(m.rstd)[:, None])
    a = np.abs(f64(dy) * f64(g))
    scale = np.abs(f64(m.rstd))[:, None] * (a + hh * (a * hh).mean(1, keepdims=True)) + np.abs(f64(up))
    assert_close(dx2, f64(dx), 2 * e * scale + 2 * uT(t) * np.abs(f64(dx)) + TINY[t], "dx")
    assert_close(dg2, f64(m.grads["dgamma"]), 2 * (n + 4) * U32 * (np.abs(f64(dy)) * hh).sum(0), "dgamma")
    for v, b in ((s2, sb), (y2, yb), (dx2, db)):
        v.zero_()
        assert ((b == 0) | (b == -7.0)).all()


@pytest.mark.parametrize("D", [5, 48, 1001])
def test_gradient_against_differences(ss, D):
    """The kernel's gradients along a direction against central differences of
    the 64-bit forward; the step's own error is h^2 / 6 of the third derivative,
    taken from a step twice as long."""
    import torch
    r = np.random.default_rng(D)
    n, eps = 6, 1e-2
    x, q, w, up = (r.normal(size=(n, D)).astype(np.float32) for _ in range(4))
    g = r.normal(size=D).astype(np.float32)
    c = lambda v: torch.as_tensor(v, device="cuda")  # noqa: E731
    m = ss.RMSNorm(n, D, eps=eps, residual=True)
    m.forward(c(x), c(g), c(q))
    h = f64(m.sum)
    dx = f64(m.backward(c(w), None, c(g), c(up)))
    dg = f64(m.grads["dgamma"])
    vx, vg = r.normal(size=(n, D)), r.normal(size=D)
    e32 = float(np.float32(eps))

    def slope(s):
        L = [(O.rms_fwd(h + k * vx, g + k * vg, e32)[0] * w.astype(np.float64)).sum() +
             ((h + k * vx) * up.astype(np.float64)).sum() for k in (s, -s)]
        return (L[0] - L[1]) / (2 * s)
    a, a2 = slope(1e-4), slope(2e-4)
    got = (dx * vx).sum() + (dg * vg).sum()
    scale = np.abs(dx * vx).sum() + np.abs(dg * vg).sum()
    assert abs(got - a) <= abs(a2 - a) + (D / 32 + 100) * U32 * scale + 1e-9


def test_offsets_past_32_bits(ss):
    import torch
    stride = (1 << 30) + 8
    buf = torch.empty(3 * stride + 64, dtype=torch.bfloat16, device="cuda")
    big = torch.as_strided(buf, (4, 64), (stride, 1))
    small = torch.randn(4, 64, device="cuda").bfloat16()
    big.copy_(small)
    a, b = (ss.RMSNorm(4, 64, dtype=torch.bfloat16, keep=torch.int8) for _ in range(2))
    assert torch.equal(a.forward(small), b.forward(big)) and torch.equal(a.kept.q, b.kept.q)
    assert torch.equal(a.backward(small, small), b.backward(big, big))
    ss.ss_rms_norm_fwd(small, None, None, 1e-5, y=big)
    assert torch.equal(big, a.y)


def test_another_stream_and_a_captured_graph(ss):
    import torch
    x, q, dy = (torch.randn(500, 48, device="cuda") for _ in range(3))
    m = ss.RMSNorm(500, 48, residual=True, keep=torch.float8_e4m3fn)
    ln = ss.LayerNorm(500, 48)
    ln.forward(x)

    def step(stream=None):
        m.forward(x, None, q, stream=stream)
        m.backward(dy, dsum=q, stream=stream)
        ln.backward(dy, m.kept, stream=stream)
    step()
    have = (m.y, m.sum, m.dx, m.grads["dgamma"], ln.dx, ln.grads["dgamma"], ln.grads["dbeta"])
    want = [v.clone() for v in have]
    s = torch.cuda.Stream()
    for v in have:
        v.fill_(3)
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(have, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for v in have:
            v.fill_(3)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(have, want))


def test_class_takes_what_the_forward_left(ss):
    import torch
    x, dy = torch.randn(30, 48, device="cuda"), torch.randn(30, 48, device="cuda")
    a = ss.RMSNorm(30, 48, residual=True)
    a.forward(x, None, dy)
    assert torch.equal(a.backward(dy), a.backward(dy, a.sum).clone())
    b = ss.RMSNorm(30, 48, keep=torch.int8, out=torch.int8)
    assert b.forward(x) is b.out and b.y is None
    assert torch.equal(b.backward(dy).clone(), b.backward(dy, b.kept))
    c = ss.RMSNorm(30, 48)
    c.forward(x)
    with pytest.raises(ValueError, match="x must be given"):
        c.backward(dy)
    assert torch.equal(c.backward(dy, x).clone(), c.backward(dy, x, rstd=c.rstd))


def test_binding_checks(ss):
    import torch
    x = torch.zeros(4, 8, device="cuda")
    m = ss.RMSNorm(4, 8, residual=True)
    with pytest.raises(ValueError, match="residual=True"):
        m.forward(x)
    with pytest.raises(ValueError, match="residual=False"):
        ss.RMSNorm(4, 8).forward(x, None, x)
    with pytest.raises(ValueError, match="x must be"):
        m.forward(x[:3], None, x)
    with pytest.raises(ValueError, match="residual must be torch.float32"):
        m.forward(x, None, x.half())
    with pytest.raises(ValueError, match="gamma must be torch.float32"):
        m.forward(x, torch.zeros(8, device="cuda").half(), x)
    with pytest.raises(ValueError, match="x must be 4 rows of 8"):
        m.backward(x, ss.Rows8(4, 9))
    with pytest.raises(ValueError, match="x must be 4 rows of 8"):
        ss.LayerNorm(4, 8).backward(x, ss.Rows8(3, 8))
    with pytest.raises(ValueError, match="dsum must be"):
        m.backward(x, x, dsum=torch.zeros(4, 7, device="cuda"))
    with pytest.raises(ValueError, match="forward=True"):
        ss.RMSNorm(4, 8, forward=False).forward(x)
    with pytest.raises(ValueError, match="rstd"):
        ss.RMSNorm(4, 8, forward=False).backward(x, x)
    with pytest.raises(ValueError, match="backward=True"):
        ss.RMSNorm(4, 8, backward=False).backward(x, x)
    with pytest.raises(ValueError, match="forward's"):
        ss.RMSNorm(4, 8, forward=False, keep=torch.int8)
    with pytest.raises(ValueError, match="format"):
        ss.RMSNorm(4, 8, out=torch.float16)
    with pytest.raises(ValueError, match="param_dtype"):
        ss.RMSNorm(4, 8, dtype=torch.float16, param_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="y must have x's type"):
        ss.ss_rms_norm_fwd(x, None, None, 1e-5, y=x.half())
    with pytest.raises(ValueError, match="out must be a Rows8"):
        ss.ss_rms_norm_fwd(x, None, None, 1e-5, out=x)
    with pytest.raises(ValueError, match="dx must have"):
        ss.ss_rms_norm_bwd(x, x, None, x[:, 0].contiguous(), None, x.half(), None, None)
    with pytest.raises(ValueError, match="one type"):
        h = x.half()
        ss.ss_rms_norm_bwd(h, h, torch.ones(8, device="cuda"), torch.ones(4, device="cuda"), None, h,
                           torch.ones(8, device="cuda").half(), m.workspace)
    for ws in (m.workspace.cpu(), torch.zeros(4096, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            ss.ss_rms_norm_bwd(x, x, None, torch.ones(4, device="cuda"), None, x, torch.ones(8, device="cuda"), ws)
