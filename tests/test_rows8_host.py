"""The C ABI of the operators for activations in 8 bits on the host (no GPU):
exports, workspace sizes, and refusals of bad arguments before anything is
enqueued."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = [os.path.join(ROOT, "include", f) for f in ("ss_rows8.h", "ss_rms.h", "ss_dense.h")]
OK, BAD, UNSUPPORTED = 0, 1, 5
F32, F16, BF16 = 0, 1, 2
INT8, E4M3 = 0, 1
A = 0x1000          # an aligned address that nothing looks at


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from gaussian_splatting_differentiable_gb300 import _lib
    return _lib.load()


def rows8(q=A, stride=8, scales=0x1003, scale_stride=1, fmt=INT8, reserved=0):
    from gaussian_splatting_differentiable_gb300._lib import SsRows8
    return SsRows8(q, stride, scales, scale_stride, fmt, reserved)


BAD_ROWS8 = [dict(q=None), dict(q=0x1004), dict(scales=None), dict(stride=12), dict(stride=0),
             dict(scale_stride=0), dict(fmt=2), dict(fmt=-1), dict(reserved=1), dict(stride=1 << 32)]


def test_every_declared_function_is_exported_and_bound(lib):
    from gaussian_splatting_differentiable_gb300 import _lib
    src = re.sub(r"/\*.*?\*/", "", "".join(open(h).read() for h in HEADERS), flags=re.S)
    names = set(re.findall(r"\b(ss_[a-z0-9_]+)\s*\(", src))
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (ss_\w+)", out))
    assert names == set(_lib.ROWS8_PROTOTYPES)


def test_struct_has_the_headers_layout():
    from gaussian_splatting_differentiable_gb300._lib import SsRows8
    assert ctypes.sizeof(SsRows8) == 40
    assert [getattr(SsRows8, f).offset for f, _ in SsRows8._fields_] == [0, 8, 16, 24, 32, 36]


def test_workspace_sizes(lib):
    for w in (lib.ss_rms_norm_workspace_bytes, lib.ss_layer_norm_bwd8_workspace_bytes):
        assert w(0, 1) > 0 and w(10, 48) >= 2 * 48 * 4
        for n, D in [(-1, 1), (1 << 31, 1), (1, 0), (1, 65537)]:
            assert w(n, D) == 0
    w = lib.ss_dense_grad8_workspace_bytes
    for t, g in ((F32, F32), (F16, F16), (BF16, F32)):
        assert w(0, 1, 1, t, g) > 0 and w(10, 48, 48, t, g) > 0
        assert w((1 << 31) - 1, 65536, 65536, t, g) > 65536 * 65536 * 4
        for n, N, D in [(-1, 1, 1), (1 << 31, 1, 1), (1, 0, 1), (1, 1, 0), (1, 65537, 1), (1, 1, 65537)]:
            assert w(n, N, D, t, g) == 0
    assert w(1, 1, 1, 3, 0) == 0 and w(1, 1, 1, F32, F16) == 0 and w(1, 1, 1, F16, BF16) == 0


def test_pack_and_unpack_refusals(lib):
    def pack(x=A, dt=F32, xs=8, n=4, D=8, r=None):
        return lib.ss_rows8_pack(x, dt, xs, n, D, rows8() if r is None else r, None)

    def unpack(x=A, dt=F32, xs=8, n=4, D=8, r=None):
        return lib.ss_rows8_unpack(rows8() if r is None else r, n, D, x, dt, xs, None)
    for f in (pack, unpack):
        assert f(n=-1) == UNSUPPORTED and f(n=1 << 31) == UNSUPPORTED and f(D=0) == UNSUPPORTED
        assert f(D=65537) == UNSUPPORTED and "65536" in lib.ss_last_error().decode()
        assert f(dt=3) == BAD and f(dt=-1) == BAD and f(x=None) == BAD and f(x=0x1002) == BAD
        assert f(dt=BF16, x=0x1001) == BAD and f(xs=7) == BAD
        assert f(D=9, xs=9) == BAD and f(D=33, xs=33, r=rows8(stride=40)) == BAD
        assert "scale_stride" in lib.ss_last_error().decode()
        for kw in BAD_ROWS8:
            assert f(r=rows8(**kw)) == BAD, kw
        assert f(n=0, x=None) == OK
    assert lib.ss_rows8_pack(A, F32, 8, 4, 8, None, None) == BAD
    assert lib.ss_rows8_unpack(None, 4, 8, A, F32, 8, None) == BAD


def test_rms_forward_refusals(lib):
    def f(x=A, dt=F32, xs=8, r=None, rs=8, n=4, D=8, g=A, pdt=F32, eps=1e-5, sum=None, ss=8, y=A, ys=8,
          out=None, kept=None, rstd=A):
        return lib.ss_rms_norm_fwd(x, dt, xs, r, rs, n, D, g, pdt, eps, sum, ss, y, ys, out, kept, rstd,
                                   None)
    assert f(n=-1) == UNSUPPORTED and f(D=0) == UNSUPPORTED and f(D=65537) == UNSUPPORTED
    assert f(dt=9) == BAD and f(pdt=F16) == BAD and f(dt=F16, pdt=BF16) == BAD
    assert f(eps=-1.0) == BAD and f(eps=float("nan")) == BAD and f(eps=float("inf")) == BAD
    assert f(x=None) == BAD and f(x=0x1002) == BAD and f(xs=7) == BAD and f(y=0x1001) == BAD
    assert f(ys=7) == BAD and f(g=0x1001) == BAD and f(rstd=0x1002) == BAD
    assert f(r=A) == BAD and f(sum=A) == BAD
    assert "residual" in lib.ss_last_error().decode()
    assert f(r=A, sum=0x2000, rs=7) == BAD and f(r=A, sum=0x2000, ss=7) == BAD and f(r=A, sum=0x2002) == BAD
    assert f(r=A, sum=0x2000, y=0x2000) == BAD and "same rows" in lib.ss_last_error().decode()
    for kw in BAD_ROWS8:
        assert f(out=rows8(**kw)) == BAD and f(kept=rows8(**kw)) == BAD
    assert f(out=rows8(), kept=rows8()) == BAD and "same rows" in lib.ss_last_error().decode()
    assert f(n=0, x=None, y=None) == OK


def test_backward_refusals(lib):
    need = lib.ss_rms_norm_workspace_bytes(4, 8)

    def rms(dy=A, dys=8, h=A, hs=8, k=None, dt=F32, n=4, D=8, g=A, pdt=F32, rstd=A, ds=None, dss=8, dx=A,
            dxs=8, dg=A, ws=A, nb=need):
        return lib.ss_rms_norm_bwd(dy, dys, h, hs, k, dt, n, D, g, pdt, rstd, ds, dss, dx, dxs, dg, ws, nb,
                                   None)

    def ln(dy=A, dys=8, k=rows8(), dt=F32, n=4, D=8, g=A, pdt=F32, mean=A, rstd=A, dx=A, dxs=8, dg=A, db=A,
           ws=A, nb=need):
        return lib.ss_layer_norm_bwd8(dy, dys, k, dt, n, D, g, pdt, mean, rstd, dx, dxs, dg, db, ws, nb,
                                      None)
    for f in (rms, ln):
        assert f(n=-1) == UNSUPPORTED and f(D=0) == UNSUPPORTED and f(D=65537) == UNSUPPORTED
        assert f(dt=4) == BAD and f(pdt=BF16) == BAD and f(dy=None) == BAD and f(dys=7) == BAD
        assert f(dx=None) == BAD and f(dxs=7) == BAD and f(rstd=None) == BAD and f(rstd=0x1002) == BAD
        assert f(dg=0x1001) == BAD and f(g=0x1001) == BAD and f(dy=0x1002) == BAD
        assert f(ws=None) == BAD and f(ws=0x1010) == BAD and f(nb=need - 1) == BAD
        assert "workspace" in lib.ss_last_error().decode()
    assert rms(h=None) == BAD and rms(k=rows8()) == BAD and "not both" in lib.ss_last_error().decode()
    assert rms(hs=7) == BAD and rms(h=0x1002) == BAD and rms(ds=A, dss=7) == BAD and rms(ds=0x1002) == BAD
    assert ln(k=None) == BAD and ln(mean=None) == BAD and ln(mean=0x1002) == BAD
    assert ln(dg=None) == BAD and ln(db=None) == BAD and ln(db=0x1001) == BAD
    for kw in BAD_ROWS8:
        assert rms(h=None, k=rows8(**kw)) == BAD and ln(k=rows8(**kw)) == BAD


def test_dense_refusals(lib):
    need = lib.ss_dense_grad8_workspace_bytes(4, 3, 8, F32, F32)

    def f(dy=A, dt=F32, dys=3, x=rows8(), n=4, N=3, D=8, dw=A, dws=8, db=A, gdt=F32, ws=A, nb=need):
        return lib.ss_dense_grad8(dy, dt, dys, x, n, N, D, dw, dws, db, gdt, ws, nb, None)
    assert f(n=-1) == UNSUPPORTED and f(N=0) == UNSUPPORTED and f(D=65537) == UNSUPPORTED
    assert f(N=65537) == UNSUPPORTED and f(dt=3) == BAD and f(gdt=F16) == BAD and f(dt=F16, gdt=BF16) == BAD
    assert f(dy=None) == BAD and f(dy=0x1002) == BAD and f(dys=2) == BAD and f(x=None) == BAD
    assert f(dw=None) == BAD and f(dw=0x1002) == BAD and f(dws=7) == BAD and f(db=0x1001) == BAD
    for kw in BAD_ROWS8:
        assert f(x=rows8(**kw)) == BAD
    assert f(ws=None) == BAD and f(ws=0x1010) == BAD and f(nb=need - 1) == BAD
    assert "workspace" in lib.ss_last_error().decode()


def test_binding_refusals(lib):
    torch = pytest.importorskip("torch")
    import gaussian_splatting_differentiable_gb300 as ss
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        ss.Rows8(4, 8, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        ss.RMSNorm(4, 8, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        ss.DenseGrad(4, 3, 8, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        ss.ss_rms_norm_fwd(x, None, None, 1e-5, y=x, stream=0)
    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        ss.ss_rms_norm_bwd(x.double(), x, None, x[:, 0], None, x, None, None, stream=0)
