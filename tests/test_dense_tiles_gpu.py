"""A weight that takes one tile after another in one workspace (many rows, a row or a column of
tiles): on another stream, in a captured graph, and two at once."""
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


# a column and a row of tiles; rows off 16-byte boundaries
CASES = [(65600, 256, 48, "f32", 0), (98400, 300, 40, "f16", 0), (65541, 48, 200, "f32", 1), (98304, 64, 300, "f16", 3)]


class Layer:
    def __init__(self, ss, n, N, D, t, pad, seed=0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(n + seed)
        self.dy = torch.randn(n, N + pad, generator=g, device="cuda").to(dtype(t))[:, :N]
        self.x = torch.randn(n, D, generator=g, device="cuda")
        self.kept, self.grad = ss.Rows8(n, D), ss.DenseGrad(n, N, D, dtype=dtype(t))

    def step(self, stream=None):
        self.grad.backward(self.dy, self.kept.pack(self.x, stream=stream), stream=stream)

    def results(self):
        return list(self.grad.grads.values())


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_another_stream_and_a_captured_graph(ss, case):
    import torch
    k = Layer(ss, *case)
    k.step()
    want = [v.clone() for v in k.results()]
    whole = k.dy.double().t() @ k.kept.unpack(torch.empty_like(k.x)).double()
    rss = (k.dy.double().square().t() @ k.x.double().square()).sqrt()
    assert float(((want[0].double() - whole).abs() / rss).max()) < 1e-4      # (the accuracy: test_dense_sums_gpu.py)

    def check():
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(k.results(), want))
        for v in k.results():
            v.fill_(3)
        k.kept._buf.fill_(0)
        torch.cuda.synchronize()
    check()
    s = torch.cuda.Stream()
    k.step(s)
    check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        k.step()
    for _ in range(3):
        g.replay()
        check()


def test_two_at_once(ss):
    """Different weights on different streams, and in one graph on two branches of it."""
    import torch
    layers = [Layer(ss, *CASES[0]), Layer(ss, *CASES[3]), Layer(ss, 3000, 300, 500, "bf16", 0)]
    for k in layers:
        k.step()
    want = [[v.clone() for v in k.results()] for k in layers]

    def check():
        torch.cuda.synchronize()
        for k, w in zip(layers, want):
            assert all(torch.equal(a, b) for a, b in zip(k.results(), w))
            for v in k.results():
                v.fill_(3)
        torch.cuda.synchronize()
    check()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(4):
        for k, s in zip(layers, streams):
            k.step(s)
        check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        for k, s in zip(layers, streams):
            s.wait_stream(main)
            k.step(s)
        for s in streams:
            main.wait_stream(s)
    for _ in range(3):
        g.replay()
        check()
