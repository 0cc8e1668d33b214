"""The weight gradient of a dense layer from kept rows whose bytes packing never
writes, and from rows that read as infinities: what the definition, dW = dy^T x with
x as it is held, gives there."""
import numpy as np
import pytest

import oracle.rows8 as O
from rows8_data import FORMATS, torch_format
from train_ops import U, U32, dtype, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_differentiable_gb300 as m
    return m


def gradient(ss, dy, x):
    m = ss.DenseGrad(x.n, dy.shape[1], x.D, dtype=dy.dtype)
    return m.backward(dy, x).cpu()


# weights of one tile (of up to 64 rows, of more), and past one; dy and x on 16-byte boundaries or not
SHAPES = [(40, 64, 0), (40, 64, 1), (100, 72, 0), (40, 120, 0), (200, 64, 0), (200, 64, 1), (200, 200, 0)]


@pytest.mark.parametrize("N,D,pad", SHAPES)
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_the_formats_nan_reads_as_nan(ss, t, N, D, pad):
    """Both NaNs that e4m3 has, in the middle of a group, beside the largest and the least
    values and at the row's end: their columns are NaN, and no other changes."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(N + D)
    n = 150
    dy = (1 + torch.rand(n, N + pad, generator=g, device="cuda")).to(dtype(t))[:, :N]
    x = ss.Rows8(n, D, torch.float8_e4m3fn).pack(torch.randn(n, D, generator=g, device="cuda"))
    x._buf[7, 2], x._buf[7, 4], x._buf[8, 5], x._buf[9, 33] = 0x7e, 0xfe, 0x01, 0x80
    want = gradient(ss, dy, x)
    x._buf[7, 3], x._buf[149, 40], x._buf[0, D - 1] = 0x7f, 0xff, 0x7f
    assert torch.isnan(x.q[7, 3].float()) and torch.isnan(x.q[149, 40].float())
    got = gradient(ss, dy, x)
    bad = [3, 40, D - 1]
    rest = [j for j in range(D) if j not in bad]
    assert torch.isnan(got[:, bad]).all() and torch.isfinite(want).all()
    assert torch.equal(got[:, rest], want[:, rest])
    back = x.unpack(torch.empty(n, D, device="cuda"))
    assert torch.equal(torch.isnan(back).nonzero().cpu(), torch.tensor([[0, D - 1], [7, 3], [149, 40]]))


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale", [16, 1, 0, 150, 254])
def test_every_e4m3_byte_reads_as_its_value(ss, t, scale):
    """One row against dy = 1: the gradient is x, each of the 256 bytes at the ends of the
    scales too (zero where a product is below float32's least normal: sums may lose that)."""
    import torch
    x = ss.Rows8(1, 256, torch.float8_e4m3fn)
    x._buf.copy_(torch.arange(256, dtype=torch.int32).to(torch.uint8)[None])
    x._scales.fill_(scale)
    dy = torch.ones(1, 3, device="cuda").to(dtype(t))
    q = x.q.float().cpu().numpy().astype(np.float64)
    with np.errstate(over="ignore"):
        want = (q * 2.0 ** (scale - 127)).astype(np.float32)[0]
    got = gradient(ss, dy, x).numpy()
    normal = ~(np.abs(want) < 2.0 ** -126)
    for i in range(3):
        assert np.array_equal(got[i][normal], want[normal], equal_nan=True)
        assert (np.abs(got[i][~normal].astype(np.float64) - want[~normal]) < 2.0 ** -126).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("N,D,pad", SHAPES)
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_rows_that_read_as_infinities(ss, t, N, D, pad, fmt):
    """Values at float32's end are rounded past it.  An infinity times dy is one of the product's
    sign, whether dy has 1, 8 or more significant bits, and NaN where dy is 0 or two meet."""
    import torch
    n, big = 90, float(np.finfo(np.float32).max)
    v = torch.ones(n, D, device="cuda")
    v[3, 10], v[3, 33], v[60, 5], v[60, 33] = big, big, -big, -big
    x = ss.Rows8(n, D, torch_format(fmt)).pack(v)
    dy = torch.full((n, N + pad), 0.75, device="cuda").to(dtype(t))[:, :N]
    values = [1.0, -1.0, 1.0 + 2.0 ** -7, -1.25 - 2.0 ** -10, 2.0 ** -14, 1.0 + 2.0 ** -20, 0.0, -0.0, 3.0 + 2.0 ** -15]
    for k, d in enumerate(values):
        dy[3, k] = d
        dy[60, k + 11] = d
    held = f64(x.unpack(torch.empty(n, D, device="cuda")))
    assert held[3, 10] == np.inf and held[3, 33] == np.inf and held[60, 5] == -np.inf and held[60, 33] == -np.inf
    got = gradient(ss, dy, x).double().numpy()
    d64 = f64(dy)
    with np.errstate(invalid="ignore"):
        terms = d64[:, :, None] * held[:, None, :]
        want = terms.sum(0)
    special = ~np.isfinite(want)
    assert special.any() and np.isnan(want).any() and np.array_equal(got[special], want[special], equal_nan=True)
    tol = 2 * (n + 16) * U32 * np.abs(terms).sum(0)[~special] + (U[t] if t != "f32" else 0.0) * np.abs(want[~special])
    assert (np.abs(got[~special] - want[~special]) <= tol).all()
