"""Rows in 8 bits whose values and scales are the caller's own, written to `q` and `scales`: read
like packed ones, whatever the buffers' memory held before."""
import pytest

from rows8_data import FORMATS, torch_format
from train_ops import dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_differentiable_gb300 as m
    return m


@pytest.mark.parametrize("t,pad", [("f32", 0), ("f32", 1), ("bf16", 0), ("bf16", 8), ("f16", 3)])
@pytest.mark.parametrize("D", [1, 10, 35, 250, 1001, 9001])
@pytest.mark.parametrize("fmt", FORMATS)
def test_every_reader_takes_the_rows_alone(ss, fmt, D, t, pad):
    import torch
    n = 37
    g = torch.Generator(device="cuda").manual_seed(D)
    packed = ss.Rows8(n, D, torch_format(fmt)).pack(torch.randn(n, D, generator=g, device="cuda"))
    size = packed._buf.shape
    dirt = [torch.full(size, 0x7f, dtype=torch.uint8, device="cuda") for _ in range(4)]     # e4m3's NaN
    del dirt
    filled = ss.Rows8(n, D, torch_format(fmt))
    filled.q.copy_(packed.q)
    filled.scales.copy_(packed.scales)
    dy = torch.randn(n, D + pad, generator=g, device="cuda").to(dtype(t))[:, :D]
    dz = torch.randn(n, 24, generator=g, device="cuda").to(dtype(t))
    gamma = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    mean, rstd = 0.1 * torch.randn(n, generator=g, device="cuda"), 0.5 + torch.rand(n, generator=g, device="cuda")
    results = []
    for r in (packed, filled):
        rms, ln = (k(n, D, dtype=dtype(t), forward=False) for k in (ss.RMSNorm, ss.LayerNorm))
        dense = ss.DenseGrad(n, 24, D, dtype=dtype(t))
        results.append([rms.backward(dy, r, gamma, rstd=rstd), rms.grads["dgamma"],
                        ln.backward(dy, r, gamma, mean, rstd), *ln.grads.values(),
                        dense.backward(dz, r), r.unpack(torch.empty(n, D, device="cuda"))])
    for a, b in zip(*results):
        assert torch.isfinite(a).all() and torch.equal(a, b)
