"""The code-table example: its operators together, as a training step uses
them, against the 64-bit forms, and a loss that falls."""
import os
import sys

import numpy as np
import pytest

import oracle.train_ops as O
from train_ops import U32, assert_close, f64

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import code_table
    return code_table


def test_a_step_matches_the_formulas(example):
    """Lookup, norm and their gradients chained on the device; each link is
    checked on the inputs it had, with the links' own tolerances (a sum of m
    float32 terms is off by at most m u times the terms' magnitude)."""
    scene = example.make_scene3d(11)
    m = example.CodeTableScene(scene, 40)
    target = example.target_of(scene)
    m.backward(m.loss(m.render(), target))
    ids = m.ids.cpu().numpy()
    assert (ids == -1).any()
    D = 48
    s = float(np.float32(D ** 0.5))
    codes = f64(m.lookup.out)
    want = O.embed_fwd(f64(m.params["table"]), ids, s)
    assert_close(codes, want, U32 * np.abs(want) + 1e-45, "codes")
    eps = float(np.float32(m.norm.eps))
    y, mean, rstd = O.layer_norm_fwd(codes, f64(m.params["gamma"]), f64(m.params["beta"]), eps)
    sh = f64(m.splats.sh).reshape(D, -1).T
    mag = np.abs(rstd)[:, None] * (np.abs(codes) + np.abs(codes).mean(1, keepdims=True)) * 0.2
    assert_close(sh, y, 80 * U32 * (mag + np.abs(y)) + 1e-7 * np.abs(y), "coefficients")
    dcoef = f64(m.projector.grads["dsh"]).reshape(D, -1).T
    dx, dg, db = O.layer_norm_bwd(dcoef, codes, f64(m.params["gamma"]), f64(m.norm.mean), f64(m.norm.rstd))
    h = np.abs((codes - f64(m.norm.mean)[:, None]) * f64(m.norm.rstd)[:, None])
    n = len(ids)
    assert_close(m.norm.grads["dgamma"], dg, (n + 4) * U32 * (np.abs(dcoef) * h).sum(0) + 1e-30, "dgamma")
    assert_close(m.norm.grads["dbeta"], db, (n + 1) * U32 * np.abs(dcoef).sum(0) + 1e-30, "dbeta")
    got = f64(m.norm.dx)
    a = np.abs(dcoef) * 0.2
    tol = 160 * U32 * f64(m.norm.rstd)[:, None] * (a + a.mean(1, keepdims=True) * (1 + h) + h * (a * h).mean(1, keepdims=True))
    assert_close(got, dx, tol + 1e-30, "dcodes")
    dt, tmag, cnt = O.embed_bwd(got, ids, 40, s)
    assert_close(m.lookup.grad, dt, (cnt[:, None] + 1) * U32 * tmag + 1e-30, "dtable")
    grads = [g.clone() for g in m.grads.values()]
    norm, coef, clipped = O.grad_clip([f64(g) for g in grads], 0.01, float(np.float32(1e-6)))
    assert_close(m.clip(0.01), np.array([norm, coef]), 40 * U32 * np.array([norm, coef]), "clip")
    assert coef < 1
    for g, w in zip(m.grads.values(), clipped):
        assert_close(g, w, 40 * U32 * np.abs(w) + 1e-40, "clipped")


def test_training_lowers_the_loss(example):
    scene = example.make_scene3d(11, n=2000)
    m = example.CodeTableScene(scene, 64)
    target = example.target_of(scene)
    losses = [float(m.step(target)) for _ in range(60)]
    assert np.isfinite(losses).all()
    assert min(losses[-5:]) < 0.8 * losses[0], losses
