"""The weight gradient of a dense layer from its input in 8 bits, against the
64-bit form.

Every product is exact, and a sum of n of them in float32, each addition
rounded or cut off (a unit of the last place, 2 u = 2^-23), is off by at most
2 (n + 16) u sum|dy x|; 16 for the splits' sums and float32 parts of dy.  The
bias likewise.  Then the rounding to the gradient's type."""
import numpy as np
import pytest

import oracle.rows8 as O
from rows8_data import Guarded, torch_format
from train_ops import TINY, U, U32, assert_close, dtype, f64, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_differentiable_gb300 as m
    return m


def inputs(ss, n, N, D, t, fmt, pad, off, seed=0):
    r = np.random.default_rng(n * 5 + N * 3 + D + seed)
    dy, _ = rows(r.normal(size=(n, N)) * np.exp(r.uniform(-4, 2, (n, 1))), t, pad, off)
    x = r.normal(size=(n, D)) * np.exp(r.uniform(-3, 3, (n, 1)))
    if n > 2:
        x[1] = 0.0
    xr, _ = rows(x, "f32")
    g = Guarded(ss, n, D, fmt, 8 * (pad % 3), pad % 2)
    g.rows.pack(xr)
    return dy, g


def check(dw, db, dy, x64, gt):
    n = len(dy)
    want_w, want_b, mw, mb = O.dense_bwd(f64(dy), x64)
    u = U[gt] if gt != "f32" else 0.0
    assert_close(dw, want_w, 2 * (n + 16) * U32 * mw + u * np.abs(want_w) + TINY[gt], "dweight")
    assert_close(db, want_b, 2 * (n + 16) * U32 * mb + u * np.abs(want_b) + TINY[gt], "dbias")


# (n, N, D, type, gradient's type, format, unused values after a row of dy, values before the first)
SHAPES = [(1, 1, 1, "f32", "f32", "int8", 0, 0), (0, 5, 7, "f32", "f32", "int8", 0, 0),
          (0, 5, 7, "bf16", "bf16", "e4m3", 0, 0), (7, 3, 2, "f16", "f32", "e4m3", 0, 0),
          (64, 8, 32, "bf16", "bf16", "int8", 0, 0), (100, 48, 48, "f32", "f32", "int8", 0, 0),
          (256, 48, 48, "bf16", "f32", "int8", 0, 0), (257, 64, 40, "f16", "f16", "e4m3", 0, 0),
          (333, 3, 48, "f32", "f32", "e4m3", 1, 0), (1000, 16, 100, "bf16", "f32", "e4m3", 0, 1),
          (65, 127, 129, "f32", "f32", "int8", 0, 0), (63, 128, 128, "bf16", "bf16", "int8", 8, 0),
          (500, 130, 260, "f16", "f32", "int8", 3, 3), (129, 256, 512, "bf16", "f32", "e4m3", 0, 0),
          (2049, 200, 33, "f32", "f32", "e4m3", 0, 0), (40, 1001, 333, "bf16", "bf16", "int8", 0, 0),
          (4097, 65, 1, "bf16", "f32", "int8", 0, 0), (3001, 1, 300, "f32", "f32", "e4m3", 0, 0),
          (5000, 59, 48, "f32", "f32", "int8", 0, 0), (20000, 7, 9, "f16", "f32", "int8", 0, 0),
          (700, 384, 640, "f16", "f16", "e4m3", 0, 0), (70, 2503, 31, "bf16", "f32", "int8", 0, 0),
          (256, 48, 48, "f32", "f32", "int8", 0, 0), (255, 16, 30, "f16", "f32", "e4m3", 8, 0),
          (300, 60, 100, "f32", "f32", "int8", 4, 0), (310, 100, 60, "f32", "f32", "e4m3", 8, 8),
          (320, 120, 128, "f16", "f32", "int8", 0, 0), (3, 65536, 1, "bf16", "bf16", "int8", 0, 0),
          (2, 1, 65536, "f32", "f32", "e4m3", 0, 0), (5, 300, 20000, "f16", "f32", "int8", 0, 0)]


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_gradient(ss, case):
    import torch
    n, N, D, t, gt, fmt, pad, off = case
    dy, g = inputs(ss, n, N, D, t, fmt, pad, off)
    x64 = f64(g.rows.unpack(torch.empty(n, D, device="cuda")))
    ws = torch.empty(ss.ss_dense_grad8_workspace_bytes(n, N, D, dtype(t), dtype(gt)), dtype=torch.uint8, device="cuda").fill_(0xFF)
    dw, buf = rows(np.zeros((N, D)), gt, pad, off, fill=-7.0)
    dw.fill_(5.0)
    db = torch.full((N,), 5.0, dtype=dtype(gt), device="cuda")
    ss.ss_dense_grad8(dy, g.rows, dw, db, ws)
    check(dw, db, dy, x64, gt)
    w0, b0 = dw.clone(), db.clone()
    ws.fill_(0xA5)
    dw.fill_(5.0)
    db.fill_(5.0)
    ss.ss_dense_grad8(dy, g.rows, dw, None, ws)         # the same bits, without the bias
    assert torch.equal(dw, w0) and (db == 5.0).all()
    m = ss.DenseGrad(n, N, D, dtype=dtype(t), grad_dtype=dtype(gt))
    assert m.backward(dy, g.rows) is m.grads["dweight"]
    assert torch.equal(m.grads["dweight"], w0) and torch.equal(m.grads["dbias"], b0)
    dw.zero_()
    assert ((buf == 0) | (buf == -7.0)).all()
    g.check_untouched()


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_products_are_exact(ss, t):
    """One row: the gradient is the product of two values, rounded once."""
    import torch
    r = np.random.default_rng(4)
    dy, _ = rows(r.normal(size=(1, 70)) * np.exp(r.uniform(-8, 8, (1, 70))), t)
    for fmt in ("int8", "e4m3"):
        x = ss.Rows8(1, 90, torch_format(fmt)).pack(torch.as_tensor(r.normal(size=(1, 90)) * 7, device="cuda").float())
        m = ss.DenseGrad(1, 70, 90, dtype=dtype(t))
        dw = f64(m.backward(dy, x))
        want = f64(dy).T @ f64(x.unpack(torch.empty(1, 90, device="cuda")))
        # three parts of a float32 dy are added in float32
        assert (np.abs(dw - want) <= (3 * 2 * U32 if t == "f32" else U32) * np.abs(want)).all()
        assert np.array_equal(f64(m.grads["dbias"]), f64(dy)[0])


@pytest.mark.parametrize("N,pad", [(40, 0), (40, 3), (200, 0), (200, 1)])
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_values_that_are_not_finite(ss, t, N, pad):
    """An infinity gives infinities of the product's sign (NaN beside zeros); NaN and
    rows that read as NaN give NaN; nothing else changes."""
    import torch
    n, D = 100, 64
    dy, _ = rows(np.ones((n, N)), t, pad)
    dy[3, 5], dy[4, 6], dy[7, 8] = float("inf"), float("-inf"), float("nan")
    xv = torch.ones(n, D, device="cuda")
    xv[3, 10] = 0.0
    xv[50, 40] = float("inf")
    x = ss.Rows8(n, D).pack(xv)
    m = ss.DenseGrad(n, N, D, dtype=dtype(t))
    dw = m.backward(dy, x).cpu()
    assert torch.isnan(dw[:, 32:]).all()
    assert dw[5, 0] == float("inf") and torch.isnan(dw[5, 10]) and dw[6, 0] == float("-inf")
    assert torch.isnan(dw[8]).all()
    rest = [i for i in range(N) if i not in (5, 6, 8)]
    assert (dw[rest, :10] == n).all() and (dw[rest, 10] == n - 1).all() and (dw[rest, 11:32] == n).all()
    db = m.grads["dbias"].cpu()
    assert db[5] == float("inf") and db[6] == float("-inf") and torch.isnan(db[8]) and (db[rest] == n).all()


@pytest.mark.parametrize("N", [3, 129])
def test_range_ends(ss, N):
    """The largest float32 and bfloat16 gradients, and scales at both ends."""
    import torch
    big = float(np.finfo(np.float32).max)
    x = torch.ones(2, 32, device="cuda")
    x[0] = 2.0 ** -90
    r = ss.Rows8(2, 32, torch.float8_e4m3fn).pack(x)
    dy = torch.zeros(2, N, device="cuda")
    dy[0, 0], dy[0, 1], dy[1, 2] = big, -big, 2.0 ** -100
    m = ss.DenseGrad(2, N, 32)
    want = f64(dy).T @ f64(x)
    assert (np.abs(f64(m.backward(dy, r)) - want) <= 6 * U32 * np.abs(want)).all()


@pytest.mark.parametrize("n,N,D,t,gt", [
    (200000, 48, 48, "f32", "f32"), (60000, 130, 70, "bf16", "f32"), (3000, 1500, 1100, "f16", "f32"),
    (1700000, 16, 24, "f16", "f32"), (300000, 100, 128, "bf16", "f32"), (100000, 60, 128, "f32", "f32"),
    (9000, 2500, 2300, "bf16", "f32"), (300000, 200, 200, "f32", "f32"), (7000, 2000, 2100, "f32", "f32"),
    (18000, 2400, 2500, "bf16", "bf16"), (20000, 1700, 1800, "f16", "f16"),
    (270000, 200, 200, "bf16", "f32"), (270000, 200, 216, "bf16", "bf16"),
    (70000, 250, 48, "f32", "f32"), (70000, 40, 200, "f16", "f32"), (300000, 1000, 1, "f32", "f32"),
    (280000, 3, 1021, "f16", "f16")])
def test_long_sums(ss, n, N, D, t, gt):
    """Sums of many rows keep float32's accuracy, far below the bound that the number of
    rows gives.  The summands' signs are random: no partial sum is past 6 times their root sum of
    squares (by Hoeffding's inequality with probability 2 exp(-18) each), an addition is off by
    at most u of it, and L such errors of random sign add up to at most 6 sqrt(L) u of it (the
    same inequality).  L: no chain of additions is longer than 4096 rows and 512 splits'
    sums (where the result is float32; in 16 bits 16384 rows, a term that its rounding hides)."""
    limit = 6 * 6 * U32 * (4096 + 512) ** 0.5
    u = U[gt] if gt != "f32" else 0.0
    import torch
    r = torch.Generator(device="cuda").manual_seed(n + N)
    rnd = lambda k: torch.randn(n, k, generator=r, device="cuda")  # noqa: E731
    dy = (rnd(N) * (rnd(1) * 2).exp()).to(dtype(t))
    rows8 = ss.Rows8(n, D).pack(rnd(D) * rnd(1).exp())
    x = rows8.unpack(torch.empty(n, D, device="cuda"))
    m = ss.DenseGrad(n, N, D, dtype=dtype(t), grad_dtype=dtype(gt))
    dw = m.backward(dy, rows8).double()
    want = dy.double().t() @ x.double()
    rss = (dy.double().square().t() @ x.double().square()).sqrt()
    past = torch.isinf(dw)          # float16's rounding has infinities from 65520 on
    assert (want[past].abs() >= 65520 - limit * rss[past]).all() and (gt == "f16" or not past.any())
    assert (want[past] * dw[past] > 0).all()
    assert float((((dw - want).abs() - u * want.abs()) / rss)[~past].max()) <= limit * (1 + u)
    wb = dy.double().sum(0)
    off = (m.grads["dbias"].double() - wb).abs() - u * wb.abs()
    assert float((off / dy.double().square().sum(0).sqrt()).max()) <= limit * (1 + u)


@pytest.mark.parametrize("n,N,D,t,gt,pad", [
    (65536, 256, 48, "f32", "f32", 0), (65541, 129, 33, "f32", "f32", 1), (98304, 7, 300, "f16", "f16", 8),
    (131072, 500, 128, "f16", "f32", 3), (98311, 64, 257, "f32", "f32", 1)])
def test_tiles_of_many_rows(ss, n, N, D, t, gt, pad):
    """A weight that takes one tile after another has each tile's own bits, in place, and
    nothing past the results and the workspace is written."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(n)
    dy = torch.randn(n, N + pad, generator=g, device="cuda").to(dtype(t))[:, :N]
    x = torch.randn(n, D, generator=g, device="cuda")
    r = ss.Rows8(n, D).pack(x)
    need = ss.ss_dense_grad8_workspace_bytes(n, N, D, dtype(t), dtype(gt))
    room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    buf = torch.full((N, D + pad), -7.0, dtype=dtype(gt), device="cuda")
    db = torch.full((N + 64,), -7.0, dtype=dtype(gt), device="cuda")
    dw = buf[:, :D]
    ss.ss_dense_grad8(dy, r, dw, db[:N], room[:need])
    assert (room[need:] == 0xA5).all() and (buf[:, D:] == -7.0).all() and (db[N:] == -7.0).all()
    for i in range(0, N, 128):
        for j in range(0, D, 128):
            part = x[:, j:j + 128].contiguous()
            m = ss.DenseGrad(n, min(128, N - i), part.shape[1], dtype=dtype(t), grad_dtype=dtype(gt))
            m.backward(dy[:, i:i + 128], ss.Rows8(n, part.shape[1]).pack(part))
            assert torch.equal(m.grads["dweight"], dw[i:i + 128, j:j + 128])
            # the bias is the first tile's of a row; tiles of other widths may add its
            # rows up in ranges of another length (of whole stages of 64 rows, or of 32)
            assert j > 0 or torch.equal(m.grads["dbias"], db[i:min(i + 128, N)])
    dw.fill_(3.0)
    ss.ss_dense_grad8(dy, r, dw, None, room[:need])
    assert torch.equal(m.grads["dweight"], dw[i:, j:]) and (db[N:] == -7.0).all()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 200])
def test_offsets_past_32_bits(ss, N, t):
    import torch
    stride = (1 << 30) + 8
    buf = torch.empty(3 * stride + N, dtype=dtype(t), device="cuda")
    big = torch.as_strided(buf, (4, N), (stride, 1))
    small = torch.randn(4, N, device="cuda").to(dtype(t))
    big.copy_(small)
    far = torch.empty(3 * (stride + 8) + 64, dtype=torch.uint8, device="cuda")
    x = torch.randn(4, 64, device="cuda")
    a, b = ss.Rows8(4, 64).pack(x), ss.Rows8(4, 64)
    b._c.q, b._c.q_stride = far.data_ptr(), stride
    b.pack(x)
    m, k = (ss.DenseGrad(4, N, 64, dtype=dtype(t)) for _ in range(2))
    want = m.backward(small, a)
    assert torch.equal(want, k.backward(big, a)) and torch.equal(want, k.backward(small, b))
    b._c.q_stride = stride + 8                       # rows on 16-byte boundaries
    assert torch.equal(want, k.backward(big, b.pack(x)))


@pytest.mark.parametrize("N,t", [(48, "f32"), (48, "bf16"), (300, "f16"), (300, "bf16")])
def test_another_stream_and_a_captured_graph(ss, N, t):
    import torch
    dy, x = torch.randn(3000, N, device="cuda").to(dtype(t)), torch.randn(3000, 100, device="cuda")
    r, m = ss.Rows8(3000, 100), ss.DenseGrad(3000, N, 100, dtype=dtype(t))
    m.backward(dy, r.pack(x))
    have = tuple(m.grads.values())
    want = [v.clone() for v in have]
    s = torch.cuda.Stream()
    for v in have:
        v.fill_(3)
    s.wait_stream(torch.cuda.current_stream())
    m.backward(dy, r, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(have, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.backward(dy, r.pack(x))
    for _ in range(3):
        for v in have:
            v.fill_(3)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(have, want))


def test_binding_checks(ss):
    import torch
    dy, r = torch.zeros(4, 3, device="cuda"), ss.Rows8(4, 8)
    m = ss.DenseGrad(4, 3, 8)
    with pytest.raises(ValueError, match="Rows8"):
        m.backward(dy, torch.zeros(4, 8, device="cuda"))
    with pytest.raises(ValueError, match="4 rows of 8"):
        m.backward(dy, ss.Rows8(4, 9))
    with pytest.raises(ValueError, match="dy must be torch.float32"):
        m.backward(dy.half(), r)
    with pytest.raises(ValueError, match="dy must be"):
        m.backward(torch.zeros(4, 4, device="cuda"), r)
    with pytest.raises(ValueError, match="grad_dtype"):
        ss.DenseGrad(4, 3, 8, dtype=torch.float16, grad_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="sizes"):
        ss.DenseGrad(4, 0, 8)
    dw, db = torch.zeros(3, 8, device="cuda"), torch.zeros(3, device="cuda")
    with pytest.raises(ValueError, match="dbias"):
        ss.ss_dense_grad8(dy, r, dw, db.half(), m.workspace)
    with pytest.raises(ValueError, match="dweight"):
        ss.ss_dense_grad8(dy, r, dw.half(), None, m.workspace)
    with pytest.raises(ValueError, match="dweight must be"):
        ss.ss_dense_grad8(dy, r, dw[:2], None, m.workspace)
    with pytest.raises(ValueError, match="Rows8"):
        ss.ss_dense_grad8(dy, None, dw, None, m.workspace)
    for ws in (m.workspace.cpu(), torch.zeros(1 << 16, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            ss.ss_dense_grad8(dy, r, dw, db, ws)
    assert ss.DenseGrad(4, 3, 8, bias=False).grads.keys() == {"dweight"}
