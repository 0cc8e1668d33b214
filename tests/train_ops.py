"""Shared by the training operators' GPU tests: rows with strides and offsets,
and unit roundoffs."""
import numpy as np

U32 = 2.0 ** -24
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}   # half the least subnormal, or that


def dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def rows(values, name, pad=0, offset=0, fill=float("nan")):
    """A device [n, D] view of `values` in type `name` inside a buffer of
    `fill`: rows `pad` values apart, the first `offset` values in."""
    import torch
    v = torch.as_tensor(values)
    n, D = v.shape
    buf = torch.full((offset + n * (D + pad),), fill, dtype=dtype(name), device="cuda")
    view = buf[offset:].view(n, D + pad)[:, :D]
    view.copy_(v)
    return view, buf


def f64(t):
    return t.detach().double().cpu().numpy()


def assert_close(got, want, tol, what=""):
    got = f64(got) if hasattr(got, "detach") else np.asarray(got)
    assert got.shape == want.shape, (got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    bad = np.abs(got - want) > tol
    bad &= ~(got == want) & ~np.isnan(want)
    if bad.any():
        k = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want) / np.maximum(tol, 1e-300), 0)),
                             got.shape)
        raise AssertionError("%s: %d of %d off; at %s got %.9g want %.9g tol %.3g" % (
            what, bad.sum(), bad.size, k, got[k], want[k], np.broadcast_to(tol, got.shape)[k]))
