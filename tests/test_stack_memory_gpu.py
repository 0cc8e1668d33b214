"""A stack of layers whose rows are kept in 8 bits and whose sums go over the stream's rows:
the same bits as from buffers of their own, and the memory that is left."""
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


def rows(n, D, t, pad, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, D + pad, generator=g, device="cuda").to(dtype(t))[:, :D]


@pytest.mark.parametrize("n,D,t,pad", [(1, 1, "f32", 0), (0, 48, "f32", 0), (700, 48, "f32", 0), (301, 48, "f32", 1), (129, 1001, "bf16", 0),
                                       (65, 4096, "bf16", 8), (40, 333, "f16", 3), (5, 9000, "f32", 0)])
@pytest.mark.parametrize("keep", [None, "int8"])
def test_in_place_gives_the_same_bits(ss, n, D, t, pad, keep):
    import torch
    keep = torch.int8 if keep else None
    a = ss.RMSNorm(n, D, dtype=dtype(t), residual=True, keep=keep)
    b = ss.RMSNorm(n, D, dtype=dtype(t), residual=True, keep=keep, inplace=True)
    assert b.sum is None and b.dx is None and a.sum is not None and a.dx is not None
    x, dy = rows(n, D, t, pad, 1), rows(n, D, t, pad, 2)
    gamma = 1 + 0.1 * rows(1, D, "f32", 0, 3)[0]
    # the same strides for both, as a row's sum goes by them
    s1, s2, d1, d2 = (rows(n, D, t, pad, k) for k in (4, 4, 5, 5))
    whole = a.forward(x, gamma, s1)
    y = b.forward(x, gamma, s2)
    assert y is b.y and torch.equal(s2, a.sum)
    m = ss.RMSNorm(n, D, dtype=dtype(t), residual=True, keep=keep)
    ss.ss_rms_norm_fwd(x, rows(n, D, t, pad, 4), gamma, m.eps, s1, m.y, None, m.kept, m.rstd)
    assert torch.equal(s1, s2) and torch.equal(m.rstd, b.rstd) and torch.equal(m.y, y)
    if pad == 0:
        assert torch.equal(whole, y) and torch.equal(a.rstd, b.rstd)
    if keep:
        assert torch.equal(b.kept.q, m.kept.q) and torch.equal(b.kept.scales, m.kept.scales)
        h = None
    else:
        h = s2
        with pytest.raises(ValueError, match="x must be given"):
            b.backward(dy, None, gamma, d2)
    dx = torch.empty_strided(d1.shape, d1.stride(), dtype=d1.dtype, device="cuda")
    ss.ss_rms_norm_bwd(dy, h if h is not None else b.kept, gamma, b.rstd, d1, dx, a.grads["dgamma"], a.workspace)
    got = b.backward(dy, h, gamma, d2)
    assert got is d2 and torch.equal(d2, dx) and torch.equal(b.grads["dgamma"], a.grads["dgamma"])
    dy2 = rows(n, D, t, pad, 2)
    ss.ss_rms_norm_bwd(dy2, h if h is not None else b.kept, gamma, b.rstd, None, dx, None, None)
    assert b.backward(dy2, h, gamma) is dy2 and torch.equal(dy2, dx)


def test_without_a_residual(ss):
    import torch
    a, b = (ss.RMSNorm(30, 48, keep=torch.int8, inplace=k) for k in (False, True))
    x, dy = rows(30, 48, "f32", 0, 1), rows(30, 48, "f32", 0, 2)
    x0 = x.clone()
    assert torch.equal(a.forward(x), b.forward(x)) and torch.equal(x, x0)
    assert torch.equal(a.backward(dy), b.backward(dy))
    with pytest.raises(ValueError, match="backward=True"):
        ss.RMSNorm(4, 8, backward=False, inplace=True).backward(x, x)


def stack(ss, layers, n, D, **kw):
    """(bytes that the layers hold once they have run, their results)."""
    import torch
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    norms = [ss.RMSNorm(n, D, residual=True, **kw) for _ in range(layers)]
    x, stream, dy = rows(n, D, "f32", 0, 1), rows(n, D, "f32", 0, 2), rows(n, D, "f32", 0, 3)
    gamma = torch.ones(D, device="cuda")
    for m in norms:
        m.forward(x, gamma, stream)
        stream = stream if m.sum is None else m.sum
    d = rows(n, D, "f32", 0, 4)
    for m in reversed(norms):
        d = m.backward(dy.clone(), gamma=gamma, dsum=d)
    torch.cuda.synchronize()
    results = [m.rstd.cpu() for m in norms], d.cpu()
    del x, stream, dy, d, gamma, m
    return torch.cuda.memory_allocated() - before, *results


def test_a_stack_holds_its_rows_in_8_bits_alone(ss):
    """Per layer and element one byte and a 32nd kept, as much of the output; without, four of
    the sum, of y and of dx."""
    import torch
    n, D, layers = 20000, 1024, 6
    whole, r0, d0 = stack(ss, layers, n, D)
    wide, r1, d1 = stack(ss, layers, n, D, out=torch.float8_e4m3fn, keep=torch.int8)
    small, r2, d2 = stack(ss, layers, n, D, out=torch.float8_e4m3fn, keep=torch.int8, inplace=True)
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(r0, r1, r2)) and torch.equal(d1, d2)
    size = n * D
    # PyTorch's allocator leaves a rest of less than 1 MB with a large tensor: rows, scales and workspace
    other = layers * (ss.ss_rms_norm_workspace_bytes(n, D) + 4 * n + 4 * D + 5 * (1 << 20))
    assert small <= layers * 2 * (size * 33 // 32) + other
    assert whole >= layers * 12 * size and wide >= whole - layers * 2 * size
    assert whole - small >= layers * (12 * size - 2 * (size * 33 // 32) - 5 * (1 << 20))
    print("\nbytes of a layer and element: %.2f, with 8 bits %.2f, in place %.2f" % (
        whole / layers / size, wide / layers / size, small / layers / size))
