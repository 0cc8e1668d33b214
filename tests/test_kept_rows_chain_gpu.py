"""The operators for activations in 8 bits together with the code table's, as a
training step uses them: rows looked up, added to a residual stream and normalised
into 8 bits, a dense layer on them, and the way back from what was kept.  Each
link is checked on the inputs it had, with the links' own tolerances (a sum of m
float32 terms is off by at most m u times the terms' magnitude, u = 2^-24; on the
tensor cores by twice that)."""
import os
import sys

import numpy as np
import pytest

import oracle.rows8 as O
import oracle.train_ops as T
from train_ops import U32, assert_close, f64

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ss():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_differentiable_gb300 as m
    return m


class Block:
    """One block of a stack: y = W rms(lookup + stream) + b in float32."""

    def __init__(self, ss, n, V, D, N, seed=0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.table, self.stream, self.gamma = rnd(V, D), rnd(n, D), 1 + 0.1 * rnd(D)
        self.W, self.dy, self.up = rnd(N, D) / D ** 0.5, rnd(n, N) * 0.1, rnd(n, D) * 0.1
        self.ids = torch.randint(-1, V, (n,), generator=g, device="cuda")
        self.lookup = ss.Embedding(n, V, D, scale=2.0)
        self.norm = ss.RMSNorm(n, D, residual=True, out=torch.float8_e4m3fn, keep=torch.int8)
        self.dense = ss.DenseGrad(n, N, D)
        self.values, self.dnorm = torch.empty(n, D, device="cuda"), torch.empty(n, D, device="cuda")
        self.y = torch.empty(n, N, device="cuda")
        self.grads = [self.lookup.grad, self.norm.grads["dgamma"], self.dense.grads["dweight"],
                      self.dense.grads["dbias"]]
        self.clip = ss.GradClip(self.grads)

    def step(self):
        import torch
        out = self.norm.forward(self.lookup.forward(self.table, self.ids), self.gamma, self.stream)
        torch.mm(out.unpack(self.values), self.W.t(), out=self.y)
        self.dense.backward(self.dy, out)
        torch.mm(self.dy, self.W, out=self.dnorm)
        dx = self.norm.backward(self.dnorm, gamma=self.gamma, dsum=self.up)
        self.lookup.backward(dx, self.ids)

    def results(self):
        return [self.norm.sum, self.norm.rstd, self.values, self.norm.dx, *self.grads]


@pytest.mark.parametrize("n,V,D,N", [(700, 40, 48, 48), (333, 50, 100, 7), (512, 64, 256, 130)])
def test_each_link(ss, n, V, D, N):
    import torch
    b = Block(ss, n, V, D, N)
    b.step()
    ids = b.ids.cpu().numpy()
    codes = f64(b.lookup.out)
    want = T.embed_fwd(f64(b.table), ids, 2.0)
    assert np.array_equal(codes, want)                       # a factor of two
    h = (b.lookup.out + b.stream).double().cpu().numpy()     # one float32 sum
    assert np.array_equal(f64(b.norm.sum), h)
    y, rstd = O.rms_fwd(h, f64(b.gamma), float(np.float32(b.norm.eps)))
    e = (D / 64 + 40) * U32
    assert_close(b.norm.rstd, rstd, e * rstd, "rstd")
    held = O.held(h, "int8")[0]
    assert np.array_equal(f64(b.norm.kept.unpack(torch.empty(n, D, device="cuda"))), held)
    lim = np.abs(y) * (1 + 2 * e)
    s = np.ldexp(1.0, np.repeat(O.scale_exponents(lim, "e4m3"), 32, 1)[:, :D] - 127)
    assert_close(b.values, y, np.maximum(lim * 2.0 ** -4, s * 2.0 ** -10) + 2 * e * np.abs(y), "y in 8 bits")
    dw, db, mw, mb = O.dense_bwd(f64(b.dy), f64(b.values))
    assert_close(b.dense.grads["dweight"], dw, 2 * (n + 16) * U32 * mw, "dweight")
    assert_close(b.dense.grads["dbias"], db, 2 * (n + 16) * U32 * mb, "dbias")
    dn, r = f64(b.dnorm), f64(b.norm.rstd)
    dx, dg = O.rms_bwd(dn, held, f64(b.gamma), r, f64(b.up))
    g = np.abs(held * r[:, None])
    a = np.abs(dn * f64(b.gamma))
    tol = (D / 32 + 80) * U32 * (r[:, None] * (a + g * (a * g).mean(1, keepdims=True)) + np.abs(f64(b.up)))
    assert_close(b.norm.dx, dx, tol, "dx")
    assert_close(b.norm.grads["dgamma"], dg, (n + 4) * U32 * (np.abs(dn) * g).sum(0), "dgamma")
    dt, tm, cnt = T.embed_bwd(f64(b.norm.dx), ids, V, 2.0)
    assert_close(b.lookup.grad, dt, (cnt[:, None] + 1) * U32 * tm + 1e-30, "dtable")
    norm, coef, clipped = T.grad_clip([f64(g) for g in b.grads], 0.5, float(np.float32(1e-6)))
    assert_close(b.clip(0.5), np.array([norm, coef]), 40 * U32 * np.array([norm, coef]), "clip")
    for got, want in zip(b.grads, clipped):
        assert_close(got, want, 40 * U32 * np.abs(want) + 1e-40, "clipped")


def test_a_captured_step_and_two_at_once(ss):
    """Two blocks on two streams, and both in one captured graph: nothing of one is in the other."""
    import torch
    a, b = Block(ss, 900, 30, 96, 200, 1), Block(ss, 1100, 70, 48, 48, 2)
    want = []
    for k in (a, b):
        k.step()
        want.append([v.clone() for v in k.results()])
    torch.cuda.synchronize()

    def check():
        torch.cuda.synchronize()
        for k, w in zip((a, b), want):
            assert all(torch.equal(x, y) for x, y in zip(k.results(), w))
            for x in k.results():
                x.fill_(3)
    check()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        torch.cuda.synchronize()
        for k, q in ((a, s), (b, t)):
            with torch.cuda.stream(q):
                k.step()
        check()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        a.step()
        b.step()
    for _ in range(3):
        torch.cuda.synchronize()
        g.replay()
        check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_the_code_table_example_with_kept_rows(ss, fmt):
    """Its gradients are the formula's at what was kept."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import code_table
    scene = code_table.make_scene3d(11)
    m = code_table.CodeTableScene(scene, 40, keep=code_table.FORMATS[fmt])
    m.step(code_table.target_of(scene))
    m.backward(m.loss(m.render(), code_table.target_of(scene)))
    codes = f64(m.lookup.out)
    held = O.held(codes, fmt)[0]
    dy, gamma, mean, r = f64(m.dcoef), f64(m.params["gamma"]), f64(m.norm.mean), f64(m.norm.rstd)
    dx, dg, db = T.layer_norm_bwd(dy, held, gamma, mean, r)
    h, n = np.abs((held - mean[:, None]) * r[:, None]), len(dy)
    a = np.abs(dy * gamma)
    tol = 160 * U32 * r[:, None] * (a + a.mean(1, keepdims=True) * (1 + h) + h * (a * h).mean(1, keepdims=True))
    assert_close(m.norm.dx, dx, tol + 1e-30, "dcodes")
    assert_close(m.norm.grads["dgamma"], dg, (n + 4) * U32 * (np.abs(dy) * h).sum(0) + 1e-30, "dgamma")
    assert_close(m.norm.grads["dbeta"], db, (n + 1) * U32 * np.abs(dy).sum(0) + 1e-30, "dbeta")
