"""The bounds that the dense layer's weight gradient is held to on the GPU, on a model of its
sums on the CPU: sums as they are formed stay within them, and each mistake that they are
there for does not: parts in one set of sums, a part lost, chains too long."""
import numpy as np
import pytest

import dense_sums as S

torch = pytest.importorskip("torch")


def inputs(kind, n, N=4, D=6):
    g = torch.Generator().manual_seed(n)
    return [v.numpy() for v in kind(n, N, D, g, "cpu", torch.float32)]


@pytest.mark.parametrize("n", [1, 2, 16, 250, 500, 2048, 5632])
def test_coarse_inputs(n):
    dy, hi, x = inputs(S.coarse, n)
    x64 = x.astype(np.float64)
    want, rests = dy.astype(np.float64).T @ x64, (dy.astype(np.float64) - hi).T @ x64
    limit = S.coarse_limit(want, rests, n, joins=-(-n // S.CHAIN) - 1)
    off = lambda **kw: np.abs(S.chained(dy, x64, **kw) - want) / limit  # noqa: E731
    assert off().max() <= 1.0
    assert np.median(off(parts=2)) > 2.0                     # the third part is missed
    if n >= 250:
        assert np.median(off(one_set=True)) > 2.0
    # and with as many joins as there may be
    limit = S.coarse_limit(want, rests, n)
    assert n > 16 or np.median(off(parts=2)) > 1.2


def test_the_parts_add_up():
    dy, hi, _ = inputs(S.coarse, 100)
    p = S.parts_of(dy)
    assert np.array_equal(sum(p), dy.astype(np.float64)) and np.array_equal(p[0], hi.astype(np.float64))
    assert (p[1] > 0).all() and (p[2] > 0).mean() > 0.9


@pytest.mark.parametrize("n", [160, 2048, 5632, 16384, 20000])
def test_graded_inputs(n):
    dy, x = inputs(S.graded, n)
    x64 = x.astype(np.float64)
    want = dy.astype(np.float64).T @ x64
    limit = S.graded_limit(want)
    assert (np.abs(S.chained(dy, x64) - want) <= limit).all()
    if n >= 16384:
        assert (np.abs(S.chained(dy, x64, chain=S.CHAIN16) - want) > limit).all()
        assert (np.abs(S.chained(dy, x64, chain=S.CHAIN16) - want) <= S.graded_limit(want, True)).all()
