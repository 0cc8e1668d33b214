"""The training operators' binding on the device: buffers of the wrong place,
type or size are refused before the library is called."""
import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_differentiable_gb300 as m
    return m


def test_clip_result_and_workspace(ss):
    import torch
    c = ss.GradClip([torch.ones(10, device="cuda")])
    arr, ws, ok = c._list, c.workspace, c.result
    for bad in (torch.zeros(2), torch.zeros(1, device="cuda"), torch.zeros(2, device="cuda").double(),
                torch.zeros(4, device="cuda")[::2]):
        with pytest.raises(ValueError, match="result"):
            ss.ss_grad_clip(arr, 1, 1.0, 1e-6, bad, ws)
        with pytest.raises(ValueError, match="result"):
            ss.ss_grad_norm(arr, 1, bad, ws)
    for bad in (ws.cpu(), torch.zeros(1 << 16, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            ss.ss_grad_clip(arr, 1, 1.0, 1e-6, ok, bad)
        with pytest.raises(ValueError, match="workspace"):
            ss.ss_grad_norm(arr, 1, ok, bad)
    ss.ss_grad_norm(arr, 1, ok, ws)
    assert float(ok[0]) == pytest.approx(10 ** 0.5, rel=1e-6)
    assert c.result is ok and float(c(1.0)[0]) == float(ok[0])


def test_gradients_workspaces(ss):
    import torch
    e, x = ss.Embedding(4, 3, 8), torch.zeros(4, 8, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    ln = ss.LayerNorm(4, 8)
    g = ln.grads
    for ws in (lambda t: t.cpu(), lambda t: torch.zeros(t.numel(), 2, dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            ss.ss_embed_bwd(x, ids, 1.0, e.grad, ws(e.workspace))
        with pytest.raises(ValueError, match="workspace"):
            ss.ss_layer_norm_bwd(x, x, None, ln.mean, ln.rstd, ln.dx, g["dgamma"], g["dbeta"], ws(ln.workspace))


def test_a_direction_without_buffers(ss):
    import torch
    t, x = torch.zeros(3, 8, device="cuda"), torch.zeros(4, 8, device="cuda")
    ids, stat = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(4, device="cuda")
    with pytest.raises(ValueError, match="forward=True"):
        ss.Embedding(4, 3, 8, forward=False).forward(t, ids)
    with pytest.raises(ValueError, match="backward=True"):
        ss.Embedding(4, 3, 8, backward=False).backward(x, ids)
    with pytest.raises(ValueError, match="forward=True"):
        ss.LayerNorm(4, 8, forward=False).forward(x)
    with pytest.raises(ValueError, match="backward=True"):
        ss.LayerNorm(4, 8, backward=False).backward(x, x)
    ln = ss.LayerNorm(4, 8, forward=False)
    for given in ({}, {"mean": stat}, {"rstd": stat}):
        with pytest.raises(ValueError, match="mean and rstd"):
            ln.backward(x, x, **given)
    assert (ln.backward(x, x, mean=stat, rstd=stat) == 0).all()


def test_the_current_stream_by_its_public_name(ss):
    """What a PyTorch without the handle's own name takes gives the same stream."""
    prog = textwrap.dedent("""
        import torch
        del torch._C._cuda_getCurrentRawStream
        import gaussian_splatting_differentiable_gb300 as ss
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            assert ss._stream(None) == s.cuda_stream
        assert ss._stream(None) == torch.cuda.current_stream().cuda_stream
    """)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", prog], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    import torch
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert ss._stream(None) == s.cuda_stream


def test_clip_refuses_results_that_overlap(ss):
    import torch
    buf = torch.arange(100.0, device="cuda")
    a, b = buf[:40], buf[40:90]
    inner, across = buf[10:20], buf[30:50]
    out = torch.zeros(100, device="cuda")
    for grads, outs in (([a, a], None), ([a, b, inner], None), ([a, across], None), ([buf, b], None),
                        ([a, b], [out[:40], out[39:89]]),          # result on result
                        ([a, b], [b[:40], out[:50]]),              # result on another gradient
                        ([buf[:10], b], [buf[1:11], out[:50]]),    # result shifted against its gradient
                        ([a, a], [out[:40], out[:40]])):
        with pytest.raises(ValueError, match="overlaps"):
            ss.GradClip(grads, outs)
    empty = buf[5:5]
    ss.GradClip([a, b, empty, empty])
    ss.GradClip([], [])
    c = ss.GradClip([a, a, inner], [out[:40], out[40:80], out[80:90]])   # gradients may
    n2 = float((2 * (a ** 2).sum() + (inner ** 2).sum()))
    assert float(c(1e9)[0]) == pytest.approx(n2 ** 0.5, rel=1e-6)
    assert torch.equal(out[:40], a) and torch.equal(out[40:80], a) and torch.equal(out[80:90], inner)
    in_place = ss.GradClip([a, b], [a, b])
    in_place(float("inf"))
