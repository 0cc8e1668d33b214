"""The training operators' C ABI on the host (no GPU): exports, workspace
sizes, and refusals of bad arguments before anything is enqueued."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = [os.path.join(ROOT, "include", f) for f in ("ss_embed.h", "ss_norm.h", "ss_clip.h")]
OK, BAD, UNSUPPORTED = 0, 1, 5
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from gaussian_splatting_differentiable_gb300 import _lib
    return _lib.load()


def test_every_declared_function_is_exported_and_bound(lib):
    from gaussian_splatting_differentiable_gb300 import _lib
    src = re.sub(r"/\*.*?\*/", "", "".join(open(h).read() for h in HEADERS), flags=re.S)
    names = set(re.findall(r"\b(ss_[a-z0-9_]+)\s*\(", src))
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (ss_\w+)", out))
    assert names == set(_lib.TRAIN_PROTOTYPES)


def test_workspace_sizes(lib):
    w = lib.ss_embed_workspace_bytes
    assert w(0, 1, 1) > 0 and w(1000, 50, 48) >= 1000 * 8
    for n, V, D in [(-1, 1, 1), (1 << 30, 1, 1), (1, 0, 1), (1, 1 << 31, 1), (1, 1, 0),
                    (1, 1, 65537)]:
        assert w(n, V, D) == 0
    w = lib.ss_layer_norm_workspace_bytes
    assert w(0, 1) > 0 and w(10, 48) >= 2 * 48 * 4
    for n, D in [(-1, 1), (1 << 31, 1), (1, 0), (1, 65537)]:
        assert w(n, D) == 0
    w = lib.ss_clip_workspace_bytes
    assert w(0) > 0 and w(65536) > 0 and w(-1) == 0 and w(65537) == 0


def test_lookup_refusals(lib):
    def f(table=0x1000, dt=F32, V=10, D=8, ts=8, ids=0x1000, idb=4, n=4, out=0x1000, os_=8):
        return lib.ss_embed_fwd(table, dt, V, D, ts, ids, idb, n, 1.0, out, os_, None)
    assert f(n=-1) == UNSUPPORTED and f(n=1 << 30) == UNSUPPORTED and f(V=0) == UNSUPPORTED
    assert f(D=0) == UNSUPPORTED and f(D=65537) == UNSUPPORTED
    assert "65536" in lib.ss_last_error().decode()
    assert f(dt=3) == BAD and f(dt=-1) == BAD and f(idb=2) == BAD
    assert f(table=None) == BAD and f(out=None) == BAD and f(ids=None) == BAD
    assert f(table=0x1002) == BAD and f(out=0x1001, dt=BF16) == BAD
    assert f(ids=0x1004, idb=8) == BAD and f(ts=7) == BAD and f(os_=7) == BAD
    assert "stride" in lib.ss_last_error().decode()
    assert f(n=0, table=None, out=None, ids=None) == OK


def test_lookup_gradient_refusals(lib):
    need = lib.ss_embed_workspace_bytes(4, 10, 8)

    def f(dout=0x1000, dt=F32, ds=8, ids=0x1000, idb=8, n=4, V=10, D=8, g=0x1000, gdt=F32, gs=8,
          ws=0x1000, nb=need):
        return lib.ss_embed_bwd(dout, dt, ds, ids, idb, n, V, D, 1.0, g, gdt, gs, ws, nb, None)
    assert f(V=0) == UNSUPPORTED and f(n=-1) == UNSUPPORTED
    assert f(dt=7) == BAD and f(gdt=F16) == BAD and f(dt=F16, gdt=BF16) == BAD
    assert f(dout=None) == BAD and f(g=None) == BAD and f(ids=None) == BAD
    assert f(ds=3) == BAD and f(gs=3) == BAD and f(g=0x1002) == BAD
    assert f(ws=None) == BAD and f(ws=0x1010) == BAD and f(nb=need - 1) == BAD
    assert "workspace" in lib.ss_last_error().decode()


def test_norm_refusals(lib):
    def f(x=0x1000, dt=F32, xs=8, n=4, D=8, g=0x1000, b=0x1000, pdt=F32, eps=1e-5, y=0x1000, ys=8,
          mean=0x1000, rstd=0x1000):
        return lib.ss_layer_norm_fwd(x, dt, xs, n, D, g, b, pdt, eps, y, ys, mean, rstd, None)
    assert f(n=-1) == UNSUPPORTED and f(D=0) == UNSUPPORTED and f(D=65537) == UNSUPPORTED
    assert f(dt=9) == BAD and f(pdt=F16) == BAD and f(dt=F16, pdt=BF16) == BAD
    assert f(eps=-1.0) == BAD and f(eps=float("nan")) == BAD and f(eps=float("inf")) == BAD
    assert f(x=None) == BAD and f(y=None) == BAD and f(x=0x1002) == BAD
    assert f(g=0x1001) == BAD and f(mean=0x1002) == BAD and f(xs=7) == BAD and f(ys=7) == BAD
    assert f(n=0, x=None, y=None) == OK
    need = lib.ss_layer_norm_workspace_bytes(4, 8)

    def h(dy=0x1000, x=0x1000, dt=F32, n=4, D=8, g=0x1000, pdt=F32, mean=0x1000, rstd=0x1000,
          dx=0x1000, dg=0x1000, db=0x1000, ws=0x1000, nb=need, s=8):
        return lib.ss_layer_norm_bwd(dy, s, x, 8, dt, n, D, g, pdt, mean, rstd, dx, 8, dg, db, ws,
                                     nb, None)
    assert h(D=0) == UNSUPPORTED and h(dt=4) == BAD and h(pdt=BF16) == BAD
    assert h(dy=None) == BAD and h(x=None) == BAD and h(dx=None) == BAD and h(mean=None) == BAD
    assert h(rstd=None) == BAD and h(dg=None) == BAD and h(db=None) == BAD and h(s=7) == BAD
    assert h(ws=None) == BAD and h(ws=0x1010) == BAD and h(nb=need - 1) == BAD
    assert "workspace" in lib.ss_last_error().decode()


def test_clip_refusals(lib):
    from gaussian_splatting_differentiable_gb300._lib import SsTensor
    need = lib.ss_clip_workspace_bytes(1)

    def f(t=(0x1000, 0x1000, 5, F32, 0), n=1, m=1.0, eps=1e-6, res=0x1000, ws=0x1000, nb=need,
          arr=True):
        a = (SsTensor * 1)(SsTensor(*t))
        return lib.ss_grad_clip(a if arr else None, n, m, eps, res, ws, nb, None)
    assert f(n=-1) == UNSUPPORTED and f(n=65537) == UNSUPPORTED and f(arr=False) == BAD
    assert f(t=(0x1000, 0x1000, 1 << 40, F32, 0)) == UNSUPPORTED
    assert f(t=(None, 0x1000, 5, F32, 0)) == BAD and f(t=(0x1000, None, 5, F32, 0)) == BAD
    assert f(t=(0x1002, 0x1000, 5, F32, 0)) == BAD and f(t=(0x1000, 0x1001, 5, BF16, 0)) == BAD
    assert f(t=(0x1000, 0x1000, -1, F32, 0)) == BAD and f(t=(0x1000, 0x1000, 5, 3, 0)) == BAD
    assert f(t=(0x1000, 0x1000, 5, F32, 1)) == BAD
    assert f(m=-1.0) == BAD and f(m=float("nan")) == BAD and f(eps=-1.0) == BAD
    assert f(res=None) == BAD and f(ws=None) == BAD and f(ws=0x1010) == BAD
    assert f(nb=need - 1) == BAD
    assert "workspace" in lib.ss_last_error().decode()
    assert lib.ss_grad_norm(None, 1, 0x1000, 0x1000, need, None) == BAD


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    import gaussian_splatting_differentiable_gb300 as ss
    t, ids = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        ss.ss_embed_fwd(t, ids, 1.0, torch.zeros(3, 8), stream=0)
    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        ss.ss_embed_fwd(t.double(), ids, 1.0, torch.zeros(3, 8), stream=0)
    with pytest.raises(ValueError, match="type"):
        ss.ss_embed_fwd(t, ids, 1.0, torch.zeros(3, 8).half(), stream=0)
    with pytest.raises(ValueError, match="ids"):
        ss.ss_embed_fwd(t, ids.float(), 1.0, torch.zeros(3, 8), stream=0)
    with pytest.raises(ValueError, match="type"):
        ss.ss_layer_norm_fwd(t, None, None, 1e-5, t.half(), stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        ss.GradClip([torch.zeros(3)], device="cpu")
    with pytest.raises(ValueError, match="outputs"):
        ss.GradClip([torch.zeros(3)], [], device="cpu")
