"""Clipping of gradients whose squares leave float32's range, above or below,
while their norm does not, against the 64-bit forms.

Tolerances, u = 2^-24.  A thread adds at most 33 squares in float32 (a rounding
each), of the values or of the values times a power of two, and pairs of float32
from there on, so that the sum is within 34 u and the norm, its root, within
17 u and two roundings (the sum's to one float32, the root's): 19 u.  Values so
far below the others that their squares are lost are below 2^-30 of the norm
here.  The coefficient adds two roundings, 21 u (a normal number here), the
product one and the type's own."""
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


def make(sizes, types, scale, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda", dtype=torch.float64) * scale).to(dtype(types[k % len(types)]))
            for k, n in enumerate(sizes)]


def check(ss, grads, share, eps=0.0):
    import torch
    src = [f64(x) for x in grads]
    norm = O.grad_clip(src, 1.0, 0.0)[0]
    m32 = float(np.float32(share * norm))
    norm, coef, want = O.grad_clip(src, m32, eps)
    outs = [torch.empty_like(x) for x in grads]
    clip = ss.GradClip(grads, outs, eps=eps)
    assert_close(clip.norm(), np.array([norm, 1.0]), np.array([19 * U32 * norm, 0.0]), "norm")
    res = f64(clip(m32))
    assert_close(res, np.array([norm, coef]), np.array([19, 21]) * U32 * np.array([norm, coef]), "result")
    names = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
    for x, w in zip(outs, want):
        t = names[x.dtype]
        assert_close(x, w, (22 * U32 + (U[t] if t != "f32" else 0)) * np.abs(w) + TINY[t], "gradient")
    assert torch.equal(ss.GradClip(grads, outs, eps=eps)(m32), clip.result)


SIZES = {"one": [1], "small": [100, 1, 7], "ragged": [3000, 4097, 5], "large": [300001, 17],
         "many": [33] * 40, "more than a launch": [50] * 1003}


@pytest.mark.parametrize("types", [["f32"], ["bf16"], ["f32", "bf16"]], ids=lambda t: "+".join(t))
@pytest.mark.parametrize("scale", [1e-36, 1e-30, 1e-24, 1e-20, 1e-14, 1e-13, 1e14, 1e16, 1e20, 1e30, 2e33])
@pytest.mark.parametrize("name", list(SIZES))
def test_values_of_one_size(ss, name, scale, types):
    check(ss, make(SIZES[name], types, scale), 0.25)


@pytest.mark.parametrize("sizes", [[50, 20], [400000, 20], [20, 400000], [5] * 700])
def test_a_few_values_of_another_size(ss, sizes):
    """One value far above the others, or all but a few of them 0 or nearly."""
    for low, high in ((1e-2, 1e25), (1e-30, 1e-2), (1e-30, 1e25), (0.0, 1e-25), (0.0, 1e25), (1e-38, 1e-25)):
        g = make(sizes, ["f32"], low)
        g[-1][1] = high
        check(ss, g, 0.5)


def test_all_sizes_of_float32_one_by_one(ss):
    import torch
    for e in range(-148, 127):
        x = torch.tensor([2.0 ** e, 0.0, -(2.0 ** e), 0.0, 2.0 ** e, 2.0 ** e], dtype=torch.float64, device="cuda").float()
        assert f64(ss.GradClip([x]).norm()).tolist() == [2.0 ** (e + 1), 1.0], e
        y = torch.zeros(90001, device="cuda")        # past what one cluster holds
        y[::30000] = x[0]
        c = ss.GradClip([y], [torch.empty_like(y)])
        assert f64(c(float("inf")))[0] == 2.0 ** (e + 1), e


def test_float16_zeros_beside_tiny_values(ss):
    import torch
    g = make([500, 500], ["f32"], 1e-25) + [torch.zeros(300, dtype=torch.float16, device="cuda")]
    check(ss, g, 0.5)
    g = make([100000], ["f32"], 1e-25) + [torch.zeros(90000, dtype=torch.float16, device="cuda")]
    check(ss, g, 0.5)


@pytest.mark.parametrize("n", [40, 100000])
def test_a_norm_past_float32_scales_nothing(ss, n):
    """The norm itself is past 3.4e38; and a value that is not finite among large ones."""
    import torch
    for k, bad in ((n, 0.0), (3, float("inf")), (3, float("nan"))):
        x = torch.zeros(n, device="cuda")
        x[:k] = 3e38
        if bad != 0.0:
            x[n - 1] = bad
        keep = x.clone()
        r = f64(ss.GradClip([x])(1.0))
        assert not np.isfinite(r[0]) and r[1] == 0.0 and np.isnan(r[0]) == np.isnan(bad)
        assert torch.equal(x.view(torch.int32), keep.view(torch.int32))


def test_nothing_but_zeros(ss):
    import torch
    for n in (0, 5, 100000):
        c = ss.GradClip([torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda").bfloat16()], eps=0.0)
        assert f64(c(1.0)).tolist() == [0.0, 1.0] and f64(c.norm()).tolist() == [0.0, 1.0]
