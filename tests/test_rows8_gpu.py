"""Rows packed into 8 bits and unpacked: every bit as the 64-bit form says (a
division by a power of two is exact, so there is one rounding and no
tolerance)."""
import numpy as np
import pytest

import oracle.rows8 as O
from rows8_data import FORMATS, Guarded, activations, torch_format
from train_ops import dtype, f64, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_differentiable_gb300 as m
    return m


# (n, D, type, unused values after a row, values before the first, bytes after a row of q, of scales)
SHAPES = [(1, 1, "f32", 0, 0, 0, 0), (0, 7, "f32", 0, 0, 0, 0), (3, 2, "f16", 0, 0, 0, 0), (9, 8, "bf16", 0, 0, 0, 0),
          (1000, 3, "f32", 0, 0, 0, 0), (333, 16, "bf16", 0, 0, 8, 1), (777, 48, "f32", 0, 0, 0, 0),
          (777, 48, "bf16", 0, 0, 0, 0), (50, 48, "f32", 1, 0, 0, 0), (51, 31, "f32", 0, 0, 0, 0),
          (52, 33, "f16", 0, 1, 24, 0), (129, 50, "f32", 0, 3, 0, 2), (100, 64, "f16", 8, 0, 0, 0),
          (100, 64, "f32", 4, 1, 0, 0), (65, 100, "bf16", 0, 1, 0, 0), (31, 127, "f32", 0, 0, 0, 0),
          (70, 128, "bf16", 0, 0, 0, 0), (37, 1001, "f16", 0, 0, 0, 0), (33, 1024, "f32", 0, 0, 0, 0),
          (12, 2503, "bf16", 5, 3, 16, 3), (17, 4096, "bf16", 0, 0, 0, 0), (9, 5001, "f32", 0, 0, 0, 0),
          (3, 20001, "f16", 0, 0, 0, 0), (2, 65536, "bf16", 0, 0, 0, 0), (3, 65535, "f32", 0, 0, 0, 0)]


def check_pack(ss, x, g, fmt):
    import torch
    n, D = x.shape
    assert g.rows.pack(x) is g.rows
    want, q, e = O.held(f64(x), fmt)
    assert np.array_equal(g.rows.scales.cpu().numpy(), e)
    assert np.array_equal(g.rows.q.float().cpu().numpy(), q)
    g.check_untouched()
    return want


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_pack_and_unpack(ss, case, fmt):
    import torch
    n, D, t, pad, off, eq, es = case
    r = np.random.default_rng(n * 7 + D)
    x, _ = rows(activations(r, n, D, t), t, pad, off)
    g = Guarded(ss, n, D, fmt, eq, es)
    want = check_pack(ss, x, g, fmt)
    for u in ("f32", "bf16", "f16"):
        out, buf = rows(np.zeros((n, D)), u, pad, off, fill=-7.0)
        assert g.rows.unpack(out) is out
        if u == "f16":
            exp = torch.as_tensor(np.clip(want, -65504.0, 65504.0)).half().double().numpy()
        else:
            exp = want
        assert np.array_equal(f64(out), exp), u
        out.zero_()
        assert ((buf == 0) | (buf == -7.0)).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_not_finite_groups(ss, fmt):
    """An infinity or a NaN takes its group of 32 and nothing else."""
    x, _ = rows(np.random.default_rng(0).normal(size=(6, 100)), "f32")
    x[0, 5], x[1, 40], x[2, 99], x[3, 64] = float("nan"), float("inf"), float("-inf"), -float("nan")
    g = Guarded(ss, 6, 100, fmt)
    check_pack(ss, x, g, fmt)
    out = g.rows.unpack(x.new_empty(6, 100))
    bad = out.isnan().cpu().numpy()
    want = np.zeros((6, 100), bool)
    want[0, :32] = want[1, 32:64] = want[2, 96:] = want[3, 64:96] = True
    assert np.array_equal(bad, want)
    assert (g.rows.scales.cpu().numpy() == 255).sum() == 4


@pytest.mark.parametrize("fmt", FORMATS)
def test_range_ends(ss, fmt):
    """float32's largest values, subnormals, and negative zeros."""
    import torch
    big = float(np.finfo(np.float32).max)
    x = torch.zeros(4, 64, device="cuda")
    x[0] = big
    x[1, :32], x[1, 32:] = -big, big / 2
    x[2] = 1e-45
    x[3] = -0.0
    g = Guarded(ss, 4, 64, fmt)
    want = check_pack(ss, x, g, fmt)
    with np.errstate(over="ignore"):
        want = want.astype(np.float32)
    assert np.array_equal(f64(g.rows.unpack(torch.empty_like(x))), want.astype(np.float64))


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_byte_reads_as_its_value(ss, fmt):
    """Also bytes that packing never writes (-128, scales outside its range)."""
    import torch
    r = ss.Rows8(256, 32, torch_format(fmt))
    e = torch.tensor([127, 100, 150, 16, 1, 0, 200, 254] * 4)
    r._buf.copy_(torch.arange(256).to(torch.uint8)[None, :].expand(256, 256)[:, :32] * 0 +
                 torch.arange(256, dtype=torch.uint8)[:, None])
    r._scales.copy_(e.repeat(8)[:256, None].to(torch.uint8))
    got = f64(r.unpack(torch.empty(256, 32, device="cuda")))
    q = r.q.float().cpu().numpy().astype(np.float64)
    with np.errstate(over="ignore"):
        want = (q * 2.0 ** (e.repeat(8)[:256, None].numpy() - 127.0)).astype(np.float32).astype(np.float64)
    assert np.array_equal(got, want, equal_nan=True)


def test_offsets_past_32_bits(ss):
    import torch
    stride = (1 << 30) + 8
    big = torch.as_strided(torch.empty(3 * stride + 64, dtype=torch.bfloat16, device="cuda"), (4, 64), (stride, 1))
    small = torch.randn(4, 64, device="cuda").bfloat16()
    big.copy_(small)
    a, b = ss.Rows8(4, 64), ss.Rows8(4, 64)
    assert torch.equal(a.pack(small).q, b.pack(big).q) and torch.equal(a.scales, b.scales)
    want = a.unpack(torch.empty_like(small))
    assert torch.equal(b.unpack(big), want)
    far = torch.empty(3 * stride + 64, dtype=torch.uint8, device="cuda")
    c = ss.Rows8(4, 64)
    c._c.q, c._c.q_stride = far.data_ptr(), stride
    assert torch.equal(c.pack(small).unpack(torch.empty_like(small)), want)


def test_another_stream_and_a_captured_graph(ss):
    import torch
    x = torch.randn(500, 48, device="cuda")
    r, out = ss.Rows8(500, 48), torch.empty(500, 48, device="cuda")
    want = r.pack(x).unpack(out).clone()
    s = torch.cuda.Stream()
    out.zero_()
    r._buf.zero_()
    s.wait_stream(torch.cuda.current_stream())
    r.pack(x, stream=s).unpack(out, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.pack(x).unpack(out)
    for k in range(2):
        out.zero_()
        x.mul_(2)
        g.replay()
        assert torch.equal(out, want * 2 ** (k + 1))


def test_binding_checks(ss):
    import torch
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError, match="format"):
        ss.Rows8(4, 8, torch.uint8)
    for n, D in ((-1, 8), (4, 0), (4, 65537)):
        with pytest.raises(ValueError, match="sizes"):
            ss.Rows8(n, D)
    r = ss.Rows8(4, 8)
    with pytest.raises(ValueError, match="x must be"):
        r.pack(x[:3])
    with pytest.raises(ValueError, match="contiguous rows"):
        r.pack(torch.zeros(8, 4, device="cuda").t())
    with pytest.raises(ValueError, match="float32, float16"):
        r.pack(x.double())
    with pytest.raises(ValueError, match="CUDA"):
        r.pack(x.cpu())
    with pytest.raises(ValueError, match="out must be"):
        r.unpack(torch.zeros(4, 9, device="cuda"))
