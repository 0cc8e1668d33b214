"""The common norm of gradients and their clipping against the 64-bit forms.

Tolerances, u = 2^-24: at most 64 squares (one rounding each) are added in
float32 before float64 takes over, every term positive, so the sum is within
(64 + 2) u and the norm within half of that and a rounding, 34 u relative;
the coefficient adds three roundings, the product one and the type's own."""
import numpy as np
import pytest

import oracle.train_ops as O
from train_ops import TINY, U, U32, assert_close, dtype, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_differentiable_gb300 as m
    return m


def make(sizes, types, seed, offsets=0):
    """Tensors as views of their own buffers, `offsets` values in."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for k, n in enumerate(sizes):
        t = dtype(types[k % len(types)])
        buf = torch.full((n + offsets + 3,), float("nan"), dtype=t, device="cuda")
        v = buf[offsets:offsets + n]
        v.copy_(torch.randn(n, generator=g, device="cuda") * 0.1)
        out.append(v)
    return out


def check(ss, grads, max_norm, inplace, out_offset=0, eps=1e-6):
    import torch
    src = [f64(x) for x in grads]
    outs, bufs = None, []
    if not inplace:
        bufs = [torch.full((x.numel() + out_offset + 5,), -7.0, dtype=x.dtype, device="cuda") for x in grads]
        outs = [b[out_offset:out_offset + x.numel()].view(x.shape) for b, x in zip(bufs, grads)]
    clip = ss.GradClip(grads, outs, eps=eps)
    m32 = float(np.float32(max_norm))
    norm, coef, want = O.grad_clip(src, m32, float(np.float32(eps)))
    assert_close(clip.norm(), np.array([norm, 1.0]), np.array([34 * U32 * norm, 0.0]), "norm")
    res = f64(clip(max_norm))
    assert_close(res, np.array([norm, coef]), np.array([34, 37]) * U32 * np.array([norm, coef]), "result")
    names = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
    for x, w in zip(grads if inplace else outs, want):
        t = names[x.dtype]
        tol = 38 * U32 * np.abs(w) + (U[t] if t != "f32" else 0) * np.abs(w) + TINY[t]
        if res[1] == 1.0:
            tol = 0.0
        assert_close(x, w, tol, "gradient")
    for b, x in zip(bufs, grads):
        assert (b[:out_offset] == -7.0).all() and (b[out_offset + x.numel():] == -7.0).all()
    if not inplace:
        for x, s in zip(grads, src):
            assert np.array_equal(f64(x), s)
        keep = [o.clone() for o in outs]
        assert np.array_equal(f64(clip(max_norm)), res)       # the same bits again
        assert all(torch.equal(a, b) for a, b in zip(keep, outs))


SIZES = {
    "none": [], "empty": [0, 0], "one": [1], "tiny": [1, 2, 3, 0, 5], "line": [17, 4096, 4095, 4097, 1],
    "mid": [768, 768, 1024, 12288, 256], "large": [300000, 1, 1500001, 48, 999983],
    "long": [12000017, 5],
}


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("types", [["f32"], ["f16"], ["bf16"], ["f32", "bf16", "f16"]], ids=lambda t: "+".join(t))
@pytest.mark.parametrize("name", list(SIZES))
def test_sizes_and_types(ss, name, types, inplace):
    check(ss, make(SIZES[name], types, 1), 0.5 if name != "one" else 1e-3, inplace)


@pytest.mark.parametrize("offset,out_offset", [(1, 1), (2, 1), (0, 1), (3, 0), (4, 8), (8, 0), (5, 5)])
def test_alignment(ss, offset, out_offset):
    sizes = [1, 3, 7, 8, 9, 31, 1000, 4099, 70001]
    check(ss, make(sizes, ["f32", "bf16"], 2, offset), 0.5, False, out_offset)


@pytest.mark.parametrize("count", [2, 31, 32, 33, 64, 65, 300, 1000, 1001, 2500])
def test_many_tensors(ss, count):
    r = np.random.default_rng(count)
    sizes = [int(v) for v in np.exp(r.uniform(0, np.log(5000), count))]
    check(ss, make(sizes, ["f32", "bf16"], 3), 1.0, False)
    check(ss, make(sizes, ["f32", "bf16"], 3), 1.0, True)


def test_below_the_bound_nothing_changes(ss):
    check(ss, make([1000, 70001], ["f32", "f16"], 4), 1e6, False)
    check(ss, make([1000, 70001], ["f32", "f16"], 4), 1e6, True)
    check(ss, make([1000, 70001], ["f32"], 4), float("inf"), True)


def test_zero_gradients_and_zero_bound(ss):
    import torch
    z = [torch.zeros(100, device="cuda"), torch.zeros(7, device="cuda").half()]
    check(ss, z, 1.0, False)
    check(ss, make([1000, 33], ["f32"], 5), 0.0, True)
    c = ss.GradClip(z, eps=0.0)
    assert f64(c(0.0)).tolist() == [0.0, 1.0]        # 0 / 0: nothing to scale


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("sizes", [[10, 20], [100000, 3], [3000000, 7]])
def test_a_norm_that_is_not_finite_scales_nothing(ss, bad, sizes):
    import torch
    grads = make(sizes, ["f32"], 6)
    grads[1][2] = bad
    keep = [g.clone() for g in grads]
    same = lambda a, b: torch.equal(a.view(torch.int32), b.view(torch.int32))  # noqa: E731
    c = ss.GradClip(grads)
    r = f64(c(1.0))
    assert not np.isfinite(r[0]) and r[1] == 0.0
    assert np.isnan(r[0]) == np.isnan(bad)
    assert all(same(a, b) for a, b in zip(grads, keep))
    outs = [torch.empty_like(g) for g in grads]
    assert f64(ss.GradClip(grads, outs)(1.0))[1] == 0.0
    assert all(same(a, b) for a, b in zip(outs, keep))
    assert f64(c.norm())[1] == 0.0


def test_sum_past_32_bit_counts(ss):
    """A tensor of 2^32 + 5 values: offsets past 32 bits; all 2^-8, so that
    every sum is a whole number of 2^-16 and the norm is exact."""
    import torch
    n = (1 << 32) + 5
    x = torch.full((n,), 2.0 ** -8, dtype=torch.bfloat16, device="cuda")
    c = ss.GradClip([x])
    norm = np.sqrt(n * 2.0 ** -16)
    assert abs(float(c.norm()[0]) - norm) <= 2 * U32 * norm
    c(256.0 * 0.25)
    assert (x[-5:] == 2.0 ** -10).all() and (x[:5] == 2.0 ** -10).all()
    assert float(x[::4097].float().max()) == float(x[::4097].float().min()) == 2.0 ** -10


def test_another_stream_and_a_captured_graph(ss):
    import torch
    for sizes in ([768, 256], [700001, 33]):
        grads = make(sizes, ["f32", "bf16"], 7)
        outs = [torch.empty_like(g) for g in grads]
        c = ss.GradClip(grads, outs)
        r = c(0.7).clone()
        want = [o.clone() for o in outs]
        s = torch.cuda.Stream()
        for o in outs:
            o.fill_(3)
        s.wait_stream(torch.cuda.current_stream())
        c(0.7, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(c.result, r) and all(torch.equal(a, b) for a, b in zip(outs, want))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c(0.7)
        for _ in range(3):
            for o in outs:
                o.fill_(3)
            g.replay()
            assert torch.equal(c.result, r) and all(torch.equal(a, b) for a, b in zip(outs, want))
