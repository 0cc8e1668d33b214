"""The scaled lookup and its gradient against the 64-bit forms.

Tolerances.  Forward: one float32 product rounded once more to the row type,
|err| <= (u32 + uT) |v| + the type's least subnormal.  Gradient: a float32 sum
of m summands in any order is off by at most (m - 1) u32 sum|x|; with the
product by the scale, and one rounding to the gradient's type:
(m + 1) u32 sum|s x| + uG |v| + subnormal."""
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


def make_ids(n, V, spread, seed):
    r = np.random.default_rng(seed)
    if spread == "uniform":
        return r.integers(0, V, n)
    if spread == "log":
        return np.minimum((np.exp(r.random(n) * np.log(V + 1)) - 1).astype(np.int64), V - 1)
    if spread == "one":
        return np.where(r.random(n) < 0.9, V // 2, r.integers(0, V, n))
    if spread == "same":
        return np.full(n, V - 1)
    if spread == "absent":
        return np.where(r.random(n) < 0.5, r.integers(0, V, n), np.where(r.random(n) < 0.5, -1, V + 3))
    assert spread == "none"
    return np.full(n, -5)


def fwd_case(ss, n, V, D, t, idt, spread, pad, off, scale=1.7):
    import torch
    r = np.random.default_rng(n + D)
    table, _ = rows(r.normal(size=(V, D)), t, pad, off)
    ids = torch.as_tensor(make_ids(n, V, spread, 3), device="cuda").to(getattr(torch, idt))
    out, buf = rows(np.zeros((n, D)), t, pad, off, fill=-7.0)
    ss.ss_embed_fwd(table, ids, scale, out)
    s = float(np.float32(scale))
    want = O.embed_fwd(f64(table), ids.cpu().numpy(), s)
    assert_close(out, want, (U32 + (U[t] if t != "f32" else 0)) * np.abs(want) + TINY[t], "out")
    out.zero_()
    assert ((buf == 0) | (buf == -7.0)).all()        # nothing outside the rows


FWD = [(0, 5, 8, "f32", "int64", "uniform", 0, 0), (1, 1, 1, "f32", "int32", "uniform", 0, 0),
       (1, 7, 48, "bf16", "int64", "uniform", 0, 0), (257, 100, 48, "f32", "int32", "log", 0, 0),
       (300, 33, 3, "f16", "int64", "absent", 0, 0), (100, 9, 1001, "bf16", "int32", "absent", 0, 1),
       (65, 17, 64, "f16", "int64", "uniform", 8, 0), (65, 17, 64, "f32", "int64", "uniform", 3, 0),
       (65, 17, 64, "f32", "int64", "uniform", 4, 1), (33, 11, 8192, "bf16", "int64", "uniform", 0, 0),
       (5, 3, 65536, "f16", "int32", "absent", 0, 0), (9001, 5000, 17, "f32", "int64", "log", 0, 0),
       (40000, 300, 16, "bf16", "int32", "uniform", 0, 0), (9, 4, 12, "f32", "int64", "none", 0, 0),
       (200003, 4099, 48, "f32", "int64", "log", 0, 0)]


@pytest.mark.parametrize("case", FWD, ids=lambda c: "-".join(map(str, c)))
def test_forward(ss, case):
    fwd_case(ss, *case)


def bwd_case(ss, n, V, D, t, gt, idt, spread, pad, off, scale=0.3):
    import torch
    r = np.random.default_rng(n + 7 * D)
    ids = make_ids(n, V, spread, 5)
    x = r.normal(size=(n, D))
    x[(ids < 0) | (ids >= V)] = np.nan               # an absent id's row is not looked at
    if n > 3:
        x[(ids < 0) | (ids >= V), 0] = np.inf
    dout, _ = rows(x, t, pad, off)
    idst = torch.as_tensor(ids, device="cuda").to(getattr(torch, idt))
    g, buf = rows(np.full((V, D), 9.0), gt, pad, off, fill=-7.0)
    ws = torch.empty(ss.ss_embed_workspace_bytes(n, V, D), dtype=torch.uint8, device="cuda").fill_(0xA5)
    ss.ss_embed_bwd(dout, idst, scale, g, ws)
    s = float(np.float32(scale))
    want, mag, cnt = O.embed_bwd(f64(dout), ids, V, s)
    tol = (cnt[:, None] + 1) * U32 * mag + (U[gt] if gt != "f32" else 0) * np.abs(want) + TINY[gt]
    assert_close(g, want, tol, "dtable")
    first = g.clone()
    ss.ss_embed_bwd(dout, idst, scale, g, ws)
    assert torch.equal(first, g)                     # the same bits again, in a used workspace
    g.zero_()
    assert ((buf == 0) | (buf == -7.0)).all()


BWD = [(0, 5, 8, "f32", "f32", "int64", "uniform", 0, 0),
       (1, 1, 1, "f32", "f32", "int32", "uniform", 0, 0),
       (1, 300000, 4, "bf16", "bf16", "int64", "uniform", 0, 0),
       (7, 3, 5, "f16", "f32", "int64", "same", 0, 0),
       (256, 1000, 48, "f32", "f32", "int32", "uniform", 0, 0),
       (511, 16, 48, "f32", "f32", "int64", "absent", 0, 0),
       (500, 20, 48, "bf16", "f32", "int64", "none", 0, 0),
       (4096, 255, 48, "f32", "f32", "int64", "uniform", 0, 0),
       (4097, 256, 48, "bf16", "bf16", "int32", "log", 0, 0),
       (8191, 64000, 40, "bf16", "bf16", "int64", "log", 0, 0),
       (8193, 65536, 24, "f16", "f16", "int64", "one", 0, 0),
       (20000, 70000, 3, "f32", "f32", "int64", "log", 0, 0),
       (30011, 17, 1, "f32", "f32", "int32", "one", 0, 0),
       (9999, 5, 1001, "bf16", "f32", "int64", "log", 0, 1),
       (3000, 70, 1000, "f16", "f32", "int32", "one", 0, 0),
       (700, 40, 8192, "bf16", "bf16", "int64", "same", 0, 0),
       (333, 9, 5000, "f32", "f32", "int64", "absent", 3, 0),
       (1000, 77, 64, "f16", "f16", "int64", "uniform", 8, 0),
       (1000, 77, 64, "f32", "f32", "int64", "uniform", 4, 1),
       (100000, 4096, 16, "f32", "f32", "int64", "same", 0, 0),
       (300000, 4096, 12, "f32", "f32", "int32", "log", 0, 0),
       (120000, 100, 48, "bf16", "f32", "int64", "one", 0, 0),
       (5, 3, 65536, "f32", "f32", "int64", "uniform", 0, 0),
       (256, 5, 8, "f16", "f32", "int32", "absent", 0, 0), (255, 700, 3, "bf16", "bf16", "int64", "one", 2, 1),
       (257, 700, 3, "bf16", "bf16", "int64", "one", 2, 1), (33, 60, 4096, "f32", "f32", "int64", "log", 0, 0),
       (32, 7, 4096, "bf16", "bf16", "int64", "same", 0, 0), (100, 16000, 1, "f32", "f32", "int32", "log", 0, 0),
       (100, 30000, 2, "f16", "f16", "int32", "uniform", 0, 0), (17, 2, 1001, "f16", "f32", "int64", "none", 0, 1)]


@pytest.mark.parametrize("case", BWD, ids=lambda c: "-".join(map(str, c)))
def test_backward(ss, case):
    bwd_case(ss, *case)


# Up to 256 ids: every slice of the columns sorts and clears for itself.
FEW = [(200, 1000, 700, "bf16", "f32", "int64", "log", 0, 0), (256, 100, 8190, "f32", "f32", "int64", "same", 0, 0),
       (150, 4096, 256, "f32", "f32", "int32", "log", 0, 0), (256, 20, 5, "f16", "f16", "int64", "one", 0, 0),
       (60, 300, 1111, "bf16", "f32", "int64", "absent", 3, 1), (256, 1000, 333, "f32", "f32", "int32", "uniform", 1, 1),
       (2, 2048, 24, "f16", "f16", "int64", "same", 8, 0), (128, 30, 65536, "bf16", "bf16", "int64", "log", 0, 0),
       (255, 40, 1002, "f32", "f32", "int64", "none", 2, 0)]


@pytest.mark.parametrize("case", FEW, ids=lambda c: "-".join(map(str, c)))
def test_backward_of_few_ids(ss, case):
    bwd_case(ss, *case)


def test_offsets_past_32_bits(ss):
    """Rows a billion values apart: the last starts past 2^32 bytes and 2^31 values."""
    import torch
    stride = (1 << 30) + 8
    buf = torch.empty(3 * stride + 16, dtype=torch.bfloat16, device="cuda")
    big = torch.as_strided(buf, (4, 16), (stride, 1))
    big.copy_(torch.arange(64, dtype=torch.float32).view(4, 16))
    ids = torch.tensor([3, 0, 3, 9, 2], device="cuda")
    small = torch.empty(5, 16, dtype=torch.bfloat16, device="cuda")
    ss.ss_embed_fwd(big, ids, 1.0, small)
    want = O.embed_fwd(np.arange(64.0).reshape(4, 16), ids.cpu().numpy(), 1.0)
    assert np.array_equal(f64(small), want)
    back = torch.tensor([1, 0, 3, 2], device="cuda")
    ss.ss_embed_fwd(small[:4], back, 1.0, big)
    assert np.array_equal(f64(big), want[:4][[1, 0, 3, 2]])
    ws = torch.empty(ss.ss_embed_workspace_bytes(4, 4, 16), dtype=torch.uint8, device="cuda")
    src = big.clone()
    for d, g in ((big, torch.empty(4, 16, dtype=torch.bfloat16, device="cuda")),
                 (src, big)):
        ss.ss_embed_bwd(d, ids[:4], 1.0, g, ws)
        assert np.array_equal(f64(g), O.embed_bwd(f64(src), ids[:4].cpu().numpy(), 4, 1.0)[0])


def test_infinities_and_nan_stay_in_their_rows(ss):
    import torch
    table = torch.ones(4, 24, device="cuda")
    table[1] = float("inf")
    table[2] = float("nan")
    e = ss.Embedding(4, 4, 24)
    out = e.forward(table, torch.tensor([0, 1, 2, 7], device="cuda"))
    assert (out[0] == 1).all() and torch.isinf(out[1]).all() and torch.isnan(out[2]).all() and (out[3] == 0).all()
    g = e.backward(out, torch.tensor([3, 2, 1, 1], device="cuda"))
    assert (g[0] == 0).all() and torch.isnan(g[1]).all() and torch.isinf(g[2]).all() and (g[3] == 1).all()


def test_another_stream_and_a_captured_graph(ss):
    import torch
    r = np.random.default_rng(0)
    ids = torch.as_tensor(make_ids(6000, 500, "log", 1), device="cuda")
    dout = torch.as_tensor(r.normal(size=(6000, 48)), device="cuda").float()
    e = ss.Embedding(6000, 500, 48)
    want = e.backward(dout, ids).clone()
    e.grad.fill_(5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    e.backward(dout, ids, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(e.grad, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        e.backward(dout, ids)
    dout.mul_(2)                                     # a power of two: every rounding the same
    for _ in range(3):
        e.grad.fill_(5)
        g.replay()
        assert torch.equal(e.grad, 2 * want)


def test_profile_names_the_kernels(ss):
    """Per-kernel timing sees the launches that overlap as well."""
    import torch
    e = ss.Embedding(6000, 50, 16)
    ids = torch.as_tensor(make_ids(6000, 50, "log", 1), device="cuda")
    dout = torch.ones(6000, 16, device="cuda")
    want = e.backward(dout, ids).clone()
    ss.ss_profile_enable(True)
    ss.ss_profile_collect()
    try:
        e.backward(dout, ids)
        names = ss.ss_profile_collect()
    finally:
        ss.ss_profile_enable(False)
    assert {"k_embed_count", "k_embed_move", "k_embed_sum"} <= set(names)
    assert torch.equal(e.grad, want)


def test_gradient_against_differences(ss):
    """The lookup is linear: its slope along a direction, through the kernels."""
    import torch
    r = np.random.default_rng(2)
    n, V, D = 77, 30, 12
    ids = torch.as_tensor(make_ids(n, V, "absent", 4), device="cuda")
    w = torch.as_tensor(r.normal(size=(n, D)), device="cuda").float()
    e = ss.Embedding(n, V, D, scale=1.25)
    g = f64(e.backward(w, ids))
    t = r.normal(size=(V, D))
    d = r.normal(size=(V, D))
    L = [float((f64(e.forward(torch.as_tensor(t + s * d, device="cuda").float(), ids)) * f64(w)).sum())
         for s in (0.5, -0.5)]
    # the two losses are sums of n D products with float32 inputs: each term 3 roundings
    tol = 8 * U32 * (np.abs(f64(w)).sum() * 1.25 * (np.abs(t).max() + np.abs(d).max()))
    assert abs((L[0] - L[1]) - (g * d).sum()) <= tol


def test_binding_checks_shapes(ss):
    import torch
    e = ss.Embedding(4, 3, 8)
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="out"):
        ss.ss_embed_fwd(torch.zeros(3, 8, device="cuda"), ids[:3], 1.0, e.out)
    with pytest.raises(ValueError, match="contiguous rows"):
        ss.ss_embed_fwd(torch.zeros(8, 3, device="cuda").t(), ids, 1.0, e.out)
    with pytest.raises(ValueError, match="dout"):
        e.backward(torch.zeros(3, 8, device="cuda"), ids)
    with pytest.raises(ValueError, match="float32"):
        e.forward(torch.zeros(3, 8, device="cuda").half(), ids)
    with pytest.raises(ValueError, match="table"):
        e.forward(torch.zeros(4, 8, device="cuda"), ids)
    with pytest.raises(ValueError, match="ids"):
        e.forward(torch.zeros(3, 8, device="cuda"), ids[:2])
    with pytest.raises(ss.SSError, match="workspace"):
        ss.ss_embed_bwd(torch.zeros(4, 8, device="cuda"), ids, 1.0, e.grad, e.workspace[:256])
    assert dtype("f32") == e.out.dtype
