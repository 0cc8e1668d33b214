"""The accuracy of the dense layer's weight gradient: sums of one sign, of which every addition
that is cut off takes a little, within bounds that parts of dy in one set of sums, a part left
out, or too long a chain of additions in the tensor cores would break (as
test_dense_sums_model.py shows on a model)."""
import numpy as np
import pytest

import dense_sums as S
from rows8_data import torch_format
from train_ops import U, dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_differentiable_gb300 as m
    return m


def gradient(ss, dy, x, gt="f32", rows=None):
    """dW in float64, twice the same; `rows`: only the first of it."""
    import torch
    m = ss.DenseGrad(x.n, dy.shape[1], x.D, dtype=dy.dtype, grad_dtype=dtype(gt))
    first = m.backward(dy, x).clone()
    m.backward(dy, x)
    assert torch.equal(m.grads["dweight"], first)
    return first[:rows].double()


def generator(n):
    import torch
    return torch.Generator(device="cuda").manual_seed(n)


def worst(got, want, limit):
    return float(((got - want).abs() / limit).max())


# all of dy and x on 16-byte boundaries, so that weights of one tile have the copy engine bring them
SMALL = [(1, 48, 48), (2, 64, 128), (1, 128, 64), (2, 104, 128), (1, 200, 200), (16, 48, 64), (250, 48, 48), (250, 40, 112),
         (250, 120, 128), (250, 128, 48), (500, 200, 200), (500, 1000, 72)]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("t", ["f32", "f16"])
@pytest.mark.parametrize("n,N,D", SMALL)
def test_no_part_is_lost_or_cut_off(ss, n, N, D, t, fmt):
    dy, hi, xv = S.coarse(n, N, D, generator(n + N), "cuda", dtype(t))
    x = ss.Rows8(n, D, torch_format(fmt)).pack(xv)
    want, rests = dy.double().t() @ xv.double(), (dy.double() - hi).t() @ xv.double()
    assert worst(gradient(ss, dy, x), want, S.coarse_limit(want, rests, n, joins=0)) <= 1.0


@pytest.mark.parametrize("t", ["f32", "f16"])
@pytest.mark.parametrize("n,N,D", [(304 * 2048, 16, 24), (304 * 2048, 80, 96), (304 * 2048 + 1, 64, 64), (200001, 48, 48),
                                   (5632, 1024, 1024), (9000, 300, 2000)])
def test_nor_is_one_of_many_rows(ss, n, N, D, t):
    dy, hi, xv = S.coarse(n, N, D, generator(n + N), "cuda", dtype(t))
    x = ss.Rows8(n, D).pack(xv)
    want, rests = dy.double().t() @ xv.double(), (dy.double() - hi).t() @ xv.double()
    assert worst(gradient(ss, dy, x), want, S.coarse_limit(want, rests, n)) <= 1.0


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,N,D", [(304 * 2048 - 1, 48, 40), (304 * 2048, 16, 24), (304 * 2048 + 1, 100, 64), (5000000, 16, 16),
                                   (2047, 2560, 2560), (2048, 2560, 2560), (2049, 2560, 2560), (16384, 2560, 2560),
                                   (30000, 1300, 2600)])
def test_chains_end(ss, n, N, D, t):
    import torch
    dy, xv = S.graded(n, N, D, generator(n + N), "cuda", dtype(t))
    x = ss.Rows8(n, D).pack(xv)
    held = x.unpack(torch.empty(n, D, device="cuda")).double()
    rows = min(N, 192)
    want = dy[:, :rows].double().t() @ held
    got = gradient(ss, dy, x, rows=rows)
    print("\n%s %d x %d x %d: %.2f of the limit, mean %.2e" % (t, n, N, D, worst(got, want, S.graded_limit(want)),
                                                              float(((got - want) / want).mean())))
    assert worst(got, want, S.graded_limit(want)) <= 1.0


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("n,N,D", [(2000, 48, 48), (1000000, 48, 48), (8191, 1024, 1024), (16384, 2560, 2560), (40000, 300, 2000)])
def test_results_of_16_bits(ss, n, N, D, t):
    """They are the sum's rounding, or the next value where the sum is that near a border."""
    import torch
    dy, xv = S.graded(n, N, D, generator(n + N), "cuda", dtype(t))
    x = ss.Rows8(n, D).pack(xv)
    held = x.unpack(torch.empty(n, D, device="cuda")).double()
    rows = min(N, 192)
    want = dy[:, :rows].double().t() @ held
    if t == "f16" and n > 100000:          # past float16's range
        dy = dy * 0.125
        want = want * 0.125
    got = gradient(ss, dy, x, t, rows)
    step = 2.0 ** torch.floor(torch.log2(want)) * (2 * U[t])        # between values next to the sum
    print("\n%s %d x %d x %d: %.2f of the limit" % (t, n, N, D, worst(got, want, step / 2 + S.graded_limit(want, True))))
    assert worst(got, want, step / 2 + S.graded_limit(want, True)) <= 1.0
