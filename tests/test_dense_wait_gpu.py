"""Failure detection in the dense layer's weight gradient, without faulting the GPU: copies that
are never issued make its bounded waits run out; the results read NaN, the call returns,
and the next one is right."""
import time

import pytest

from train_ops import dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_differentiable_gb300 as m
    return m


# of one tile: parts through the copies' ring (stacked and not), and dy by the copy engine itself; one
# range and many; past one tile: bias out of the tiles and from the conversion, several chains of a range
@pytest.mark.parametrize("n,N,D,t,gt", [
    (256, 48, 48, "f32", "f32"), (256, 48, 48, "bf16", "f32"), (250, 128, 128, "f16", "f16"),
    (256, 104, 64, "bf16", "bf16"), (3000, 64, 96, "f32", "f32"), (300, 200, 200, "bf16", "f32"),
    (400, 200, 200, "f32", "f32"), (6000, 1024, 1024, "bf16", "f32"), (20000, 1024, 1000, "bf16", "bf16")])
def test_a_wait_that_runs_out(ss, n, N, D, t, gt):
    import torch
    g = torch.Generator(device="cuda").manual_seed(n)
    dy = torch.randn(n, N, generator=g, device="cuda").to(dtype(t))
    x = ss.Rows8(n, D).pack(torch.randn(n, D, generator=g, device="cuda"))
    m = ss.DenseGrad(n, N, D, dtype=dtype(t), grad_dtype=dtype(gt))
    dw, db = m.grads["dweight"], m.grads["dbias"]
    m.backward(dy, x)
    want = dw.clone(), db.clone()
    dw.fill_(5.0), db.fill_(5.0)
    torch.cuda.synchronize()
    t0 = time.time()
    ss.ss_test_dense_wait_timeout(dy, x, dw, db, m.workspace)
    torch.cuda.synchronize()
    assert time.time() - t0 < 10.0
    assert torch.isnan(dw).all()
    assert torch.isnan(db).all() or (t != "bf16" and N > 128 and torch.equal(db, want[1]))   # converted before
    m.backward(dy, x)
    assert torch.equal(dw, want[0]) and torch.equal(db, want[1])
