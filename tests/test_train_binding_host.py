"""The training operators' binding refuses what the library would read or
write outside of, or what is not on the device, before it calls the library;
and the package loads whatever the installed PyTorch has of CUDA (no GPU)."""
import os
import subprocess
import sys
import textwrap

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ss():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gb300 as m
    return m


def test_clip_refuses_what_is_not_its_list(ss):
    from gaussian_splatting_differentiable_gb300._lib import SsTensor
    two, res, ws = (SsTensor * 2)(), torch.zeros(2), torch.zeros(4096, dtype=torch.uint8)
    for f in (lambda t, n: ss.ss_grad_clip(t, n, 1.0, 1e-6, res, ws, stream=0),
              lambda t, n: ss.ss_grad_norm(t, n, res, ws, stream=0)):
        with pytest.raises(ValueError, match="3 tensors in a list of 2"):
            f(two, 3)
        with pytest.raises(ValueError, match="SsTensor"):
            f([two[0]], 1)
        with pytest.raises(ValueError, match="SsTensor"):
            f((SsTensor * 1)()[0], 1)


def test_clip_refuses_host_buffers(ss):
    from gaussian_splatting_differentiable_gb300._lib import SsTensor
    one, ws = (SsTensor * 1)(), torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="result"):
        ss.ss_grad_clip(one, 1, 1.0, 1e-6, torch.zeros(2), ws, stream=0)
    with pytest.raises(ValueError, match="result"):
        ss.ss_grad_norm(one, 1, torch.zeros(2), ws, stream=0)


def test_buffers_are_made_on_the_device(ss):
    for make in (lambda: ss.Embedding(4, 3, 8, device="cpu"), lambda: ss.LayerNorm(4, 8, device="cpu"),
                 lambda: ss.GradClip([], device="cpu")):
        with pytest.raises(ValueError, match="CUDA device"):
            make()


def test_import_without_the_cuda_names_of_torch(ss):
    """A PyTorch without CUDA has none of them; streams given as handles still work."""
    prog = textwrap.dedent("""
        import torch
        for name in [n for n in dir(torch._C) if n.startswith("_cuda_getCurrent") or n == "_cuda_getDevice"]:
            delattr(torch._C, name)
        import gaussian_splatting_differentiable_gb300 as ss
        assert ss._stream(7) == 7
        assert ss.ss_embed_workspace_bytes(4, 3, 8) > 0
    """)
    r = subprocess.run([sys.executable, "-c", prog], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
