"""Tile-based differentiable rasterization of projected 2D Gaussian splats on GB300.

The compute path is libss.so (hand-written CUDA for sm_103a behind the C ABI
of include/ss.h, include/ss_project.h and include/ss_ssim.h, and of the training
operators' include/ss_embed.h, include/ss_norm.h and include/ss_clip.h).  This
module is its thin Python binding: each ss_* function
here has the C function's name and arguments and only marshals torch tensors
(device memory) and streams into pointers.  PyTorch provides memory and
streams; every step of the path runs in the library's kernels.  There is no
fallback: importing this package without the built library raises
ImportError.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _lib
from ._lib import (SS_ACCUM_WEIGHT, SS_BF16, SS_DISTORTION, SS_ERR_CAPACITY,  # noqa: F401
                   SS_ERR_DEVICE, SS_ERR_TIMEOUT, SS_F16, SS_F32, SS_MEDIAN_DEPTH, SS_OK, SS_RECORDS_CLEARED, SS_WEIGHT_STATS,
                   STATUS_NAMES, SsGrads, SsSplats)

_L = _lib.load()
TILE = 16


class SSError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = _L.ss_last_error().decode(errors="replace")
        super().__init__("%s: %s: %s" % (where, STATUS_NAMES.get(status, status), msg))
        self.status = status


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# The current stream's handle without a Stream object around it: 0.2 us of host
# time against 2.9 us, a third of a small call.  These names are PyTorch's own;
# one that lacks them (built without CUDA, say) takes the public way.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
if _current_stream is None or _current_device is None:
    def _current_device():
        return None

    def _current_stream(device):
        return torch.cuda.current_stream(device).cuda_stream


def _stream(stream):
    if stream is None:
        return _current_stream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(st: int, where: str):
    if st != SS_OK:
        raise SSError(st, where)


def _f32_host3(bg):
    if bg is None:
        return None
    return (ctypes.c_float * 3)(*[float(x) for x in bg])


@dataclasses.dataclass
class Splats:
    """Device SoA splats (float32, contiguous): mean2d [n,2], conic [n,3],
    opacity [n], rgb [n,3], depth [n]."""
    mean2d: torch.Tensor
    conic: torch.Tensor
    opacity: torch.Tensor
    rgb: torch.Tensor
    depth: torch.Tensor

    @property
    def n(self) -> int:
        return int(self.opacity.shape[0])

    def c(self) -> SsSplats:
        for k in ("mean2d", "conic", "opacity", "rgb", "depth"):
            t = getattr(self, k)
            if t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda:
                raise ValueError("Splats.%s must be a contiguous float32 CUDA tensor" % k)
        return SsSplats(_ptr(self.mean2d), _ptr(self.conic), _ptr(self.opacity), _ptr(self.rgb),
                        _ptr(self.depth), self.n)

    @staticmethod
    def from_numpy(scene, device="cuda") -> "Splats":
        f = lambda a: torch.from_numpy(a).to(device=device, dtype=torch.float32).contiguous()  # noqa
        return Splats(f(scene.mean2d), f(scene.conic), f(scene.opacity), f(scene.rgb),
                      f(scene.depth))


# ------------------------------------------------------------------ C ABI

def ss_abi_version() -> int:
    return int(_L.ss_abi_version())


def ss_constants() -> dict:
    buf = (ctypes.c_float * 4)()
    _L.ss_constants(buf)
    return {"alpha_min": buf[0], "alpha_max": buf[1], "T_eps": buf[2], "tile": int(buf[3])}


def ss_last_error() -> str:
    return _L.ss_last_error().decode(errors="replace")


def ss_workspace_bytes(n_splats: int, n_pairs: int, W: int, H: int) -> int:
    return int(_L.ss_workspace_bytes(n_splats, n_pairs, W, H))


COUNTER_WORDS = 4   # ss_bin_tiles' uint64 counters: pairs, culled, depth-bit range


def _counters(counters):
    """The counters tensor's pointer, after checking that it holds the four
    64-bit words the library writes (a plain pointer crosses the C ABI)."""
    if isinstance(counters, torch.Tensor) and counters.numel() * counters.element_size() < 8 * COUNTER_WORDS:
        raise ValueError("counters must hold %d 64-bit words (got %d bytes)"
                         % (COUNTER_WORDS, counters.numel() * counters.element_size()))
    return _ptr(counters)


def ss_record_bytes(n_splats: int) -> int:
    return int(_L.ss_record_bytes(n_splats))


def ss_bin_tiles(splats: Splats, W: int, H: int, keys, vals, capacity: int, counters, records,
                 stream=None) -> None:
    s = splats.c()
    _check(_L.ss_bin_tiles(ctypes.byref(s), W, H, _ptr(keys), _ptr(vals), capacity,
                           _counters(counters), _ptr(records), _stream(stream)), "ss_bin_tiles")


def ss_pair_count(counters, capacity: int, stream=None):
    """(status, pairs needed, culled); status is SS_OK or SS_ERR_CAPACITY."""
    pairs, culled = ctypes.c_int64(0), ctypes.c_int64(0)
    st = _L.ss_pair_count(_counters(counters), capacity, ctypes.byref(pairs), ctypes.byref(culled),
                          _stream(stream))
    if st not in (SS_OK, SS_ERR_CAPACITY):
        raise SSError(st, "ss_pair_count")
    return st, pairs.value, culled.value


def ss_sort_pairs(keys, vals, n_pairs: int, W: int, H: int, tile_offsets, workspace,
                  stream=None) -> None:
    _check(_L.ss_sort_pairs(_ptr(keys), _ptr(vals), n_pairs, W, H, _ptr(tile_offsets),
                            _ptr(workspace), workspace.numel() * workspace.element_size(),
                            _stream(stream)), "ss_sort_pairs")


def ss_sort_pairs_dev(keys, vals, counters, capacity: int, W: int, H: int, tile_offsets,
                      workspace, stream=None) -> None:
    _check(_L.ss_sort_pairs_dev(_ptr(keys), _ptr(vals), _counters(counters), capacity, W, H,
                                _ptr(tile_offsets), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream)),
           "ss_sort_pairs_dev")


def ss_sort_status(workspace, stream=None) -> int:
    return int(_L.ss_sort_status(_ptr(workspace), _stream(stream)))


def ss_raster_fwd(splats: Splats, vals, tile_offsets, W: int, H: int, bg, flags: int, image,
                  T_final, last_contrib, median_depth=None, stream=None) -> None:
    """The forward from the splats themselves (no records, no blend masks)."""
    s = splats.c()
    _check(_L.ss_raster_fwd(ctypes.byref(s), _ptr(vals), _ptr(tile_offsets), W, H,
                            _f32_host3(bg), flags, _ptr(image), _ptr(T_final), _ptr(last_contrib),
                            _ptr(median_depth), _stream(stream)), "ss_raster_fwd")


def ss_raster_fwd_records(records, n_splats: int, vals, tile_offsets, n_pairs: int, W: int,
                          H: int, bg, flags: int, image, T_final, last_contrib, median_depth,
                          blend_masks, max_weight=None, blend_count=None, distortion=None,
                          dist_totals=None, stream=None, bwd_workspace=None) -> None:
    """bwd_workspace: the workspace of the following ss_raster_bwd_records,
    whose gradient records the forward then clears (pass SS_RECORDS_CLEARED
    to that call; nothing may write the workspace in between)."""
    nbytes = 0 if bwd_workspace is None else bwd_workspace.numel() * bwd_workspace.element_size()
    _check(_L.ss_raster_fwd_records(_ptr(records), n_splats, _ptr(vals), _ptr(tile_offsets),
                                    n_pairs, W, H, _f32_host3(bg), flags, _ptr(image),
                                    _ptr(T_final), _ptr(last_contrib), _ptr(median_depth),
                                    _ptr(blend_masks), _ptr(max_weight), _ptr(blend_count),
                                    _ptr(distortion), _ptr(dist_totals), _ptr(bwd_workspace),
                                    nbytes, _stream(stream)), "ss_raster_fwd_records")


def _grads_struct(grads: dict) -> SsGrads:
    return SsGrads(_ptr(grads["dmean2d"]), _ptr(grads["dconic"]), _ptr(grads["dopacity"]),
                   _ptr(grads["drgb"]), _ptr(grads.get("ddepth")))


def ss_raster_bwd(splats: Splats, vals, tile_offsets, W: int, H: int, bg, flags: int, T_final,
                  last_contrib, dL_dimage, grads: dict, accum_weight, workspace,
                  stream=None) -> None:
    """The backward from the splats themselves: records and blend decisions
    rebuilt in the workspace (ss_workspace_bytes(n, pairs, W, H) bytes)."""
    s = splats.c()
    g = _grads_struct(grads)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_L.ss_raster_bwd(ctypes.byref(s), _ptr(vals), _ptr(tile_offsets), W, H,
                            _f32_host3(bg), flags, _ptr(T_final), _ptr(last_contrib),
                            _ptr(dL_dimage), ctypes.byref(g), _ptr(accum_weight),
                            _ptr(workspace), nbytes, _stream(stream)), "ss_raster_bwd")


def ss_raster_bwd_records(records, n_splats: int, vals, tile_offsets, n_pairs: int, W: int,
                          H: int, bg, flags: int, T_final, last_contrib, blend_masks, dL_dimage,
                          grads: dict, accum_weight, workspace, stream=None, dist_totals=None,
                          dL_ddist=None) -> None:
    """blend_masks may be None: the decisions are then re-evaluated into the
    workspace."""
    g = _grads_struct(grads)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_L.ss_raster_bwd_records(_ptr(records), n_splats, _ptr(vals), _ptr(tile_offsets),
                                    n_pairs, W, H, _f32_host3(bg), flags, _ptr(T_final),
                                    _ptr(last_contrib), _ptr(blend_masks), _ptr(dL_dimage),
                                    _ptr(dist_totals), _ptr(dL_ddist), ctypes.byref(g),
                                    _ptr(accum_weight), _ptr(workspace), nbytes,
                                    _stream(stream)), "ss_raster_bwd_records")


def ss_raster_bwd_noalloc(records, n_splats: int, vals, tile_offsets, n_pairs: int, W: int,
                          H: int, bg, flags: int, T_final, last_contrib, blend_masks, dL_dimage,
                          grads: dict, accum_weight, stream=None) -> None:
    """ss_raster_bwd_records for callers that cannot allocate: no workspace argument;
    the weight scratch is a fixed array inside the library (at most 2,097,152
    splats; concurrent calls race on it)."""
    g = _grads_struct(grads)
    _check(_L.ss_raster_bwd_noalloc(_ptr(records), n_splats, _ptr(vals), _ptr(tile_offsets),
                                    n_pairs, W, H, _f32_host3(bg), flags, _ptr(T_final),
                                    _ptr(last_contrib), _ptr(blend_masks), _ptr(dL_dimage),
                                    ctypes.byref(g), _ptr(accum_weight),
                                    _stream(stream)), "ss_raster_bwd_noalloc")


def ss_profile_enable(on: bool) -> None:
    _L.ss_profile_enable(1 if on else 0)


def ss_profile_collect() -> dict:
    """{kernel name: (launches, total_ms, min_ms, max_ms)} since the last collect."""
    buf = ctypes.create_string_buffer(1 << 20)   # one line per kernel name
    _L.ss_profile_collect(buf, len(buf))
    out = {}
    for line in buf.value.decode().splitlines():
        name, cnt, tot, mn, mx = line.split()
        out[name] = (int(cnt), float(tot), float(mn), float(mx))
    return out


def ss_debug_bounds_enabled() -> bool:
    return bool(_L.ss_debug_bounds_enabled())


def ss_debug_status(stream=None) -> int:
    """SS_OK, or SS_ERR_DEVICE if a device-side bounds check failed since the
    last call (only the SS_DEBUG_BOUNDS build checks; see ss_last_error())."""
    return int(_L.ss_debug_status(_stream(stream)))


def ss_probe_red_f32(buf, rounds: int, stream=None) -> None:
    _check(_L.ss_probe_red_f32(_ptr(buf), buf.numel(), rounds, _stream(stream)),
           "ss_probe_red_f32")


def ss_test_sort_wait_timeout(workspace, stream=None) -> None:
    _check(_L.ss_test_sort_wait_timeout(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                        _stream(stream)), "ss_test_sort_wait_timeout")


# ------------------------------------------------------------------ projection (ss_project.h)

@dataclasses.dataclass
class Splats3D:
    """Device 3D splats (float32, contiguous): mean3 [n,3], scale [n,3],
    quat [n,4] (w, x, y, z), sh [K,3,n] coefficient-major, K = (degree+1)^2."""
    mean3: torch.Tensor
    scale: torch.Tensor
    quat: torch.Tensor
    sh: torch.Tensor
    sh_degree: int

    @property
    def n(self) -> int:
        return int(self.mean3.shape[0])

    def c(self) -> _lib.SsSplats3d:
        for k in ("mean3", "scale", "quat", "sh"):
            t = getattr(self, k)
            if t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda:
                raise ValueError("Splats3D.%s must be a contiguous float32 CUDA tensor" % k)
        return _lib.SsSplats3d(_ptr(self.mean3), _ptr(self.scale), _ptr(self.quat),
                               _ptr(self.sh), self.n, self.sh_degree)

    @staticmethod
    def from_numpy(scene, device="cuda") -> "Splats3D":
        f = lambda a: torch.from_numpy(a).to(device=device, dtype=torch.float32).contiguous()  # noqa
        return Splats3D(f(scene.mean3), f(scene.scale), f(scene.quat), f(scene.sh),
                        scene.sh_degree)


def camera(R, t, fx: float, fy: float, cx: float, cy: float, near: float,
           blur: float) -> _lib.SsCamera:
    """The host ss_camera struct (R row-major world-to-camera rotation)."""
    c = _lib.SsCamera()
    for k, v in enumerate([float(x) for row in R for x in row]):
        c.R[k] = v
    for k in range(3):
        c.t[k] = float(t[k])
    c.fx, c.fy, c.cx, c.cy, c.near_z, c.blur = fx, fy, cx, cy, near, blur
    return c


def ss_project_fwd(splats: Splats3D, cam: _lib.SsCamera, mean2d, conic, depth, rgb,
                   stream=None) -> None:
    s = splats.c()
    _check(_L.ss_project_fwd(ctypes.byref(s), ctypes.byref(cam), _ptr(mean2d), _ptr(conic),
                             _ptr(depth), _ptr(rgb), _stream(stream)), "ss_project_fwd")


def ss_project_bwd(splats: Splats3D, cam: _lib.SsCamera, dmean2d, dconic, drgb, grads: dict,
                   stream=None) -> None:
    """grads: dict of device tensors dmean3, dscale, dquat, dsh (overwritten)."""
    s = splats.c()
    g = _lib.SsGrads3d(*[_ptr(grads[k]) for k in ("dmean3", "dscale", "dquat", "dsh")])
    _check(_L.ss_project_bwd(ctypes.byref(s), ctypes.byref(cam), _ptr(dmean2d), _ptr(dconic),
                             _ptr(drgb), ctypes.byref(g), _stream(stream)), "ss_project_bwd")


class Projector:
    """Output and gradient buffers of the projection for n splats; the 2D
    outputs plus a caller's opacity form the rasterizer's Splats."""

    def __init__(self, n: int, sh_degree: int, device="cuda"):
        d = torch.device(device)
        f = lambda *s: torch.empty(*s, dtype=torch.float32, device=d)  # noqa: E731
        K = (sh_degree + 1) ** 2
        self.n, self.sh_degree = n, sh_degree
        self.mean2d, self.conic, self.depth, self.rgb = f(n, 2), f(n, 3), f(n), f(n, 3)
        self.grads = {"dmean3": f(n, 3), "dscale": f(n, 3), "dquat": f(n, 4), "dsh": f(K, 3, n)}

    def forward(self, splats: Splats3D, cam, stream=None) -> None:
        ss_project_fwd(splats, cam, self.mean2d, self.conic, self.depth, self.rgb, stream)

    def backward(self, splats: Splats3D, cam, dmean2d, dconic, drgb, stream=None) -> None:
        ss_project_bwd(splats, cam, dmean2d, dconic, drgb, self.grads, stream)

    def splats2d(self, opacity) -> Splats:
        return Splats(self.mean2d, self.conic, opacity, self.rgb, self.depth)


# ------------------------------------------------------------------ L1 + SSIM loss (ss_ssim.h)

def ss_ssim_workspace_bytes(C: int, H: int, W: int) -> int:
    return int(_L.ss_ssim_workspace_bytes(C, H, W))


def ss_ssim_loss(img, target, lam: float, loss, dL_dimg, workspace, stream=None) -> None:
    """img, target, dL_dimg: [C,H,W] float32 device tensors; loss: float32[3]
    device tensor (loss, mean SSIM, mean |x - y|)."""
    C, H, W = img.shape
    _check(_L.ss_ssim_loss(_ptr(img), _ptr(target), C, H, W, float(lam), _ptr(loss),
                           _ptr(dL_dimg), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream)),
           "ss_ssim_loss")


class SsimLoss:
    """Buffers of ss_ssim_loss for one image size."""

    def __init__(self, C: int, H: int, W: int, lam: float = 0.2, device="cuda"):
        d = torch.device(device)
        self.lam = lam
        self.loss = torch.zeros(3, dtype=torch.float32, device=d)
        self.grad = torch.empty(C, H, W, dtype=torch.float32, device=d)
        nb = max(ss_ssim_workspace_bytes(C, H, W), 16)
        self.workspace = torch.empty((nb + 15) // 16, 2, dtype=torch.float64, device=d)

    def __call__(self, img, target, stream=None) -> torch.Tensor:
        ss_ssim_loss(img, target, self.lam, self.loss, self.grad, self.workspace, stream)
        return self.grad


# ------------------------------------------------------------------ training operators

DTYPE_CODES = {torch.float32: SS_F32, torch.float16: SS_F16, torch.bfloat16: SS_BF16}


def _code(dtype, name: str) -> int:
    code = DTYPE_CODES.get(dtype)
    if code is None:
        raise ValueError("%s must be float32, float16 or bfloat16 (got %s)" % (name, dtype))
    return code


def _dtype(t, name: str) -> int:
    return _code(t.dtype, name)


def _rows(t, name: str, D: int, n=None):
    """(pointer, row stride) of a [n, D] device tensor with contiguous rows."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != D or (n is not None and shape[0] != n):
        raise ValueError("%s must be [%s, %d] (got %s)" % (name, "n" if n is None else n, D,
                                                           tuple(shape)))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    rs, cs = t.stride()
    if cs != 1 and D > 1:
        raise ValueError("%s must have contiguous rows (column stride %d)" % (name, cs))
    if rs < D:
        if shape[0] > 1:
            raise ValueError("%s has overlapping rows (row stride %d < %d)" % (name, rs, D))
        rs = D               # no second row: any stride will do
    return t.data_ptr(), rs


def _vector(t, name: str, size: int, dtype=None) -> int:
    if t.shape != (size,) or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA vector of %d (got %s)"
                         % (name, size, tuple(t.shape)))
    if dtype is not None and t.dtype is not dtype:
        raise ValueError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    return t.data_ptr()


def _ids(ids, n=None):
    """(pointer, bytes of an id)."""
    size = 8 if ids.dtype is torch.int64 else 4
    if size == 4 and ids.dtype is not torch.int32:
        raise ValueError("ids must be int32 or int64 (got %s)" % ids.dtype)
    shape = ids.shape
    if len(shape) != 1 or (n is not None and shape[0] != n) or not ids.is_cuda or \
            not ids.is_contiguous():
        raise ValueError("ids must be a contiguous CUDA vector%s (got %s)"
                         % ("" if n is None else " of %d" % n, tuple(shape)))
    return ids.data_ptr(), size


def _workspace(nbytes: int, device):
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _device(device):
    """The device of an object's own buffers: the kernels take their pointers as they are."""
    d = torch.device(device)
    if d.type != "cuda":
        raise ValueError("device must be a CUDA device (got %s)" % d)
    return d


def _scratch(workspace):
    """(pointer, bytes) of a caller's workspace."""
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr(), workspace.nbytes


# ---- scaled lookup (ss_embed.h)

def ss_embed_workspace_bytes(n: int, V: int, D: int) -> int:
    return int(_L.ss_embed_workspace_bytes(n, V, D))


def ss_embed_fwd(table, ids, scale: float, out, stream=None) -> None:
    """out[i] = scale * table[ids[i]]; zeros where ids[i] is outside [0, V).
    table: [V, D], out: [n, D] of the same type; ids: int32 or int64 [n]."""
    V, D = table.shape
    code = _dtype(table, "table")
    if out.dtype != table.dtype:
        raise ValueError("out must have the table's type")
    idp, idb = _ids(ids)
    n = ids.shape[0]
    tp, ts = _rows(table, "table", D)
    op, os_ = _rows(out, "out", D, n)
    st = _L.ss_embed_fwd(tp, code, V, D, ts, idp, idb, n, scale, op, os_, _stream(stream))
    if st:
        _check(st, "ss_embed_fwd")


def ss_embed_bwd(dout, ids, scale: float, dtable, workspace, stream=None) -> None:
    """dtable[v] = scale * the sum of the rows of dout whose id is v; every row
    of dtable [V, D] (dout's type or float32) is overwritten."""
    V, D = dtable.shape
    code, gcode = _dtype(dout, "dout"), _dtype(dtable, "dtable")
    idp, idb = _ids(ids)
    n = ids.shape[0]
    dp, ds = _rows(dout, "dout", D, n)
    gp, gs = _rows(dtable, "dtable", D)
    wp, wb = _scratch(workspace)
    st = _L.ss_embed_bwd(dp, code, ds, idp, idb, n, V, D, scale, gp, gcode, gs, wp, wb,
                         _stream(stream))
    if st:
        _check(st, "ss_embed_bwd")


class Embedding:
    """Buffers of the scaled lookup and its gradient for n ids into a table
    of V rows of D values: `out` [n, D] and `grad` [V, D].  They belong to
    one stream at a time: calls on different streams are the caller's to order.
    (The methods check what they are given; their own buffers they made.)"""

    def __init__(self, n: int, V: int, D: int, scale: float = 1.0, dtype=torch.float32,
                 grad_dtype=None, device="cuda", forward: bool = True, backward: bool = True):
        d = _device(device)
        self.n, self.V, self.D, self.scale = n, V, D, float(scale)
        self.dtype, self._code = dtype, _code(dtype, "dtype")
        self._out = torch.empty(n, D, dtype=dtype, device=d) if forward else None
        self._grad = self._workspace = None
        if backward:
            nb = ss_embed_workspace_bytes(n, V, D)
            if nb == 0:
                raise ValueError("sizes out of range")
            self._grad = torch.empty(V, D, dtype=grad_dtype or dtype, device=d)
            self._grad_code = _code(self._grad.dtype, "grad_dtype")
            self._workspace = _workspace(nb, d)

    out = property(lambda self: self._out)
    grad = property(lambda self: self._grad)
    workspace = property(lambda self: self._workspace)

    def _input(self, t, name: str, rows: int):
        if t.dtype is not self.dtype:
            raise ValueError("%s must be %s (got %s)" % (name, self.dtype, t.dtype))
        return _rows(t, name, self.D, rows)

    def forward(self, table, ids, stream=None) -> torch.Tensor:
        tp, ts = self._input(table, "table", self.V)
        idp, idb = _ids(ids, self.n)
        out = self._out
        if out is None:
            raise ValueError("this Embedding was made without forward=True")
        st = _L.ss_embed_fwd(tp, self._code, self.V, self.D, ts, idp, idb, self.n, self.scale,
                             out.data_ptr(), self.D, _stream(stream))
        if st:
            _check(st, "ss_embed_fwd")
        return out

    def backward(self, dout, ids, stream=None) -> torch.Tensor:
        dp, ds = self._input(dout, "dout", self.n)
        idp, idb = _ids(ids, self.n)
        grad, ws = self._grad, self._workspace
        if grad is None:
            raise ValueError("this Embedding was made without backward=True")
        st = _L.ss_embed_bwd(dp, self._code, ds, idp, idb, self.n, self.V, self.D, self.scale,
                             grad.data_ptr(), self._grad_code, self.D, ws.data_ptr(), ws.nbytes,
                             _stream(stream))
        if st:
            _check(st, "ss_embed_bwd")
        return grad


# ---- layer norm (ss_norm.h)

def ss_layer_norm_workspace_bytes(n: int, D: int) -> int:
    return int(_L.ss_layer_norm_workspace_bytes(n, D))


def _param(t, name: str, D: int, code: int, dtype) -> tuple:
    """(pointer, type code) of a parameter vector of the rows' type or float32."""
    p = _vector(t, name, D)
    if t.dtype != dtype and t.dtype != torch.float32:
        raise ValueError("%s must be float32 or the rows' type (got %s)" % (name, t.dtype))
    return p, (code if t.dtype == dtype else SS_F32)


def ss_layer_norm_fwd(x, gamma, beta, eps: float, y, mean=None, rstd=None, stream=None) -> None:
    """y = (x - mean) * rstd * gamma + beta over the rows of x [n, D]; gamma
    and beta [D] (one type, the rows' or float32) or None; mean, rstd:
    float32 [n] or None."""
    n, D = x.shape
    code = _dtype(x, "x")
    if y.dtype != x.dtype:
        raise ValueError("y must have x's type")
    xp, xs = _rows(x, "x", D)
    yp, ys = _rows(y, "y", D, n)
    gp, gc = (None, None) if gamma is None else _param(gamma, "gamma", D, code, x.dtype)
    bp, bc = (None, None) if beta is None else _param(beta, "beta", D, code, x.dtype)
    if gc is not None and bc is not None and gc != bc:
        raise ValueError("gamma and beta must have one type")
    pc = gc if gc is not None else (bc if bc is not None else SS_F32)
    mp = None if mean is None else _vector(mean, "mean", n, torch.float32)
    rp = None if rstd is None else _vector(rstd, "rstd", n, torch.float32)
    st = _L.ss_layer_norm_fwd(xp, code, xs, n, D, gp, bp, pc, eps, yp, ys, mp, rp,
                              _stream(stream))
    if st:
        _check(st, "ss_layer_norm_fwd")


def ss_layer_norm_bwd(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, workspace,
                      stream=None) -> None:
    """dx [n, D], and dgamma, dbeta [D] (both or neither) from dy, the
    forward's x, gamma, mean and rstd; dx may be dy or x."""
    n, D = x.shape
    code = _dtype(x, "x")
    if dy.dtype != x.dtype or dx.dtype != x.dtype:
        raise ValueError("dy and dx must have x's type")
    dyp, dys = _rows(dy, "dy", D, n)
    xp, xs = _rows(x, "x", D)
    dxp, dxs = _rows(dx, "dx", D, n)
    gp, pc = (None, None) if gamma is None else _param(gamma, "gamma", D, code, x.dtype)
    dgp = dbp = None
    for t, name in ((dgamma, "dgamma"), (dbeta, "dbeta")):
        if t is None:
            continue
        p, c = _param(t, name, D, code, x.dtype)
        if pc is not None and c != pc:
            raise ValueError("gamma, dgamma and dbeta must have one type")
        pc = c
        if name == "dgamma":
            dgp = p
        else:
            dbp = p
    mp = _vector(mean, "mean", n, torch.float32)
    rp = _vector(rstd, "rstd", n, torch.float32)
    wp, wb = (None, 0) if workspace is None else _scratch(workspace)
    st = _L.ss_layer_norm_bwd(dyp, dys, xp, xs, code, n, D, gp, SS_F32 if pc is None else pc, mp,
                              rp, dxp, dxs, dgp, dbp, wp, wb, _stream(stream))
    if st:
        _check(st, "ss_layer_norm_bwd")


class LayerNorm:
    """Buffers of the layer norm of n rows of D values: `y`, `mean`, `rstd`
    of the forward, `dx` and `grads` (dgamma, dbeta) of the backward.  They
    belong to one stream at a time, as Embedding's do.  param_dtype is that of
    gamma, beta and their gradients."""

    def __init__(self, n: int, D: int, eps: float = 1e-5, dtype=torch.float32,
                 param_dtype=torch.float32, device="cuda", forward: bool = True,
                 backward: bool = True):
        d = _device(device)
        self.n, self.D, self.eps = n, D, float(eps)
        self.dtype, self._code = dtype, _code(dtype, "dtype")
        self.param_dtype, self._param_code = param_dtype, _code(param_dtype, "param_dtype")
        if param_dtype != dtype and param_dtype != torch.float32:
            raise ValueError("param_dtype must be float32 or the rows' type")
        self._y = self._mean = self._rstd = self._dx = self._workspace = self.grads = None
        if forward:
            self._y = torch.empty(n, D, dtype=dtype, device=d)
            self._mean = torch.empty(n, dtype=torch.float32, device=d)
            self._rstd = torch.empty(n, dtype=torch.float32, device=d)
        if backward:
            nb = ss_layer_norm_workspace_bytes(n, D)
            if nb == 0:
                raise ValueError("sizes out of range")
            self._dx = torch.empty(n, D, dtype=dtype, device=d)
            self._dgamma, self._dbeta = (torch.empty(D, dtype=param_dtype, device=d)
                                         for _ in range(2))
            self.grads = {"dgamma": self._dgamma, "dbeta": self._dbeta}
            self._workspace = _workspace(nb, d)

    y = property(lambda self: self._y)
    mean = property(lambda self: self._mean)
    rstd = property(lambda self: self._rstd)
    dx = property(lambda self: self._dx)
    workspace = property(lambda self: self._workspace)

    def _input(self, t, name: str):
        if t.dtype is not self.dtype:
            raise ValueError("%s must be %s (got %s)" % (name, self.dtype, t.dtype))
        return _rows(t, name, self.D, self.n)

    def forward(self, x, gamma=None, beta=None, stream=None) -> torch.Tensor:
        xp, xs = self._input(x, "x")
        D, p = self.D, self.param_dtype
        gp = None if gamma is None else _vector(gamma, "gamma", D, p)
        bp = None if beta is None else _vector(beta, "beta", D, p)
        y = self._y
        if y is None:
            raise ValueError("this LayerNorm was made without forward=True")
        st = _L.ss_layer_norm_fwd(xp, self._code, xs, self.n, D, gp, bp, self._param_code,
                                  self.eps, y.data_ptr(), D, self._mean.data_ptr(),
                                  self._rstd.data_ptr(), _stream(stream))
        if st:
            _check(st, "ss_layer_norm_fwd")
        return y

    def backward(self, dy, x, gamma=None, mean=None, rstd=None, stream=None) -> torch.Tensor:
        """mean, rstd: the forward's, this object's own if not given."""
        dyp, dys = self._input(dy, "dy")
        xp, xs = self._input(x, "x")
        n, D = self.n, self.D
        gp = None if gamma is None else _vector(gamma, "gamma", D, self.param_dtype)
        dx, ws = self._dx, self._workspace
        if dx is None:
            raise ValueError("this LayerNorm was made without backward=True")
        if self._mean is None and (mean is None or rstd is None):
            raise ValueError("mean and rstd must be given to a LayerNorm made without forward=True")
        mp = self._mean.data_ptr() if mean is None else _vector(mean, "mean", n, torch.float32)
        rp = self._rstd.data_ptr() if rstd is None else _vector(rstd, "rstd", n, torch.float32)
        st = _L.ss_layer_norm_bwd(dyp, dys, xp, xs, self._code, n, D, gp, self._param_code, mp, rp,
                                  dx.data_ptr(), D, self._dgamma.data_ptr(),
                                  self._dbeta.data_ptr(), ws.data_ptr(), ws.nbytes,
                                  _stream(stream))
        if st:
            _check(st, "ss_layer_norm_bwd")
        return dx


# ---- gradient norm and clipping (ss_clip.h)

def ss_clip_workspace_bytes(n_tensors: int) -> int:
    return int(_L.ss_clip_workspace_bytes(n_tensors))


def _tensor_list(grads, outs):
    """The host array of ss_tensor for `grads`, results into `outs` (None: in place)."""
    if outs is not None and len(outs) != len(grads):
        raise ValueError("%d outputs for %d gradients" % (len(outs), len(grads)))
    arr = (_lib.SsTensor * max(len(grads), 1))()
    for k, g in enumerate(grads):
        o = g if outs is None else outs[k]
        code = _dtype(g, "gradient %d" % k)
        if not g.is_cuda or not g.is_contiguous():
            raise ValueError("gradient %d must be a contiguous CUDA tensor" % k)
        if o is not g and (o.dtype != g.dtype or o.shape != g.shape or not o.is_cuda or
                           not o.is_contiguous()):
            raise ValueError("output %d must be a contiguous CUDA tensor like its gradient" % k)
        arr[k] = _lib.SsTensor(g.data_ptr(), o.data_ptr(), g.numel(), code, 0)
    _no_overlaps([(a.inp, a.out, g.nbytes) for a, g in zip(arr, grads) if a.numel])
    return arr


def _no_overlaps(spans):
    """Refuses results that share memory with one another or with a gradient
    other than their own: a gradient listed twice in place would be scaled twice,
    by whichever threads come first."""
    pieces = []
    for i, o, nbytes in spans:
        pieces.append((o, o + nbytes, True))
        if i != o:
            pieces.append((i, i + nbytes, False))
    read_to = written_to = 0
    for start, end, written in sorted(pieces):
        if start < written_to or (written and start < read_to):
            raise ValueError("a result overlaps another result or a gradient (a tensor listed twice?)")
        if written:
            written_to = max(written_to, end)
        else:
            read_to = max(read_to, end)


def _clip_args(tensors, n: int, result, workspace):
    """Pointers and sizes, after checking that the list holds n tensors and the
    result two values (plain pointers cross the C ABI)."""
    if not isinstance(tensors, ctypes.Array) or tensors._type_ is not _lib.SsTensor:
        raise ValueError("tensors must be a ctypes array of SsTensor")
    if n > len(tensors):
        raise ValueError("%d tensors in a list of %d" % (n, len(tensors)))
    if result.dtype != torch.float32 or result.numel() < 2 or not result.is_cuda or \
            not result.is_contiguous():
        raise ValueError("result must be a contiguous float32 CUDA tensor of 2")
    return (result.data_ptr(), *_scratch(workspace))


def ss_grad_clip(tensors, n: int, max_norm: float, eps: float, result, workspace,
                 stream=None) -> None:
    """tensors: the ctypes array of SsTensor (see GradClip); result: float32[2]
    device tensor, (norm, coefficient)."""
    rp, wp, wb = _clip_args(tensors, n, result, workspace)
    st = _L.ss_grad_clip(tensors, n, max_norm, eps, rp, wp, wb, _stream(stream))
    if st:
        _check(st, "ss_grad_clip")


def ss_grad_norm(tensors, n: int, result, workspace, stream=None) -> None:
    rp, wp, wb = _clip_args(tensors, n, result, workspace)
    st = _L.ss_grad_norm(tensors, n, rp, wp, wb, _stream(stream))
    if st:
        _check(st, "ss_grad_norm")


class GradClip:
    """The gradients of a step, clipped together: clip(max_norm) scales them
    in place, or into `outs`, by min(1, max_norm / (norm + eps)) and returns
    `result`, the device float32[2] (norm, coefficient); the coefficient is 0
    and nothing is scaled where the norm is not finite.  The lists are read
    once, here: their tensors must stay where they are, and gradients that are
    new tensors each step need a new object each step.  No result may share
    memory with another, or with a gradient other than its own."""

    def __init__(self, grads, outs=None, eps: float = 1e-6, device="cuda"):
        self.grads, self.outs = list(grads), None if outs is None else list(outs)
        self.eps = float(eps)
        self._n = len(self.grads)
        nb = ss_clip_workspace_bytes(self._n)
        if nb == 0:
            raise ValueError("too many tensors")
        self._list = _tensor_list(self.grads, self.outs)
        d = _device(device)
        self._result = torch.zeros(2, dtype=torch.float32, device=d)
        self._workspace = _workspace(nb, d)

    n = property(lambda self: self._n)
    result = property(lambda self: self._result)
    workspace = property(lambda self: self._workspace)

    def __call__(self, max_norm: float, stream=None) -> torch.Tensor:
        result, ws = self._result, self._workspace
        st = _L.ss_grad_clip(self._list, self._n, max_norm, self.eps, result.data_ptr(),
                             ws.data_ptr(), ws.nbytes, _stream(stream))
        if st:
            _check(st, "ss_grad_clip")
        return result

    def norm(self, stream=None) -> torch.Tensor:
        """result = (norm, 1 if it is finite else 0); scales nothing."""
        result, ws = self._result, self._workspace
        st = _L.ss_grad_norm(self._list, self._n, result.data_ptr(), ws.data_ptr(), ws.nbytes,
                             _stream(stream))
        if st:
            _check(st, "ss_grad_norm")
        return result


# ------------------------------------------------------------------ whole path

class Rasterizer:
    """Buffers for one image size and splat count, reused across calls, and
    the call sequence bin -> pair count -> sort -> forward / backward.

    Pair buffers grow (once) when the binning reports more pairs than their
    capacity; nothing else is allocated after construction."""

    def __init__(self, W: int, H: int, n_splats: int, pair_capacity: int, flags: int = 0,
                 bg=None, device="cuda"):
        self.W, self.H, self.n, self.flags = W, H, n_splats, flags
        self.bg = None if bg is None else [float(x) for x in bg]
        self.device = torch.device(device)
        self.tiles = ((W + TILE - 1) // TILE) * ((H + TILE - 1) // TILE)
        d = self.device
        self.counters = torch.zeros(COUNTER_WORDS, dtype=torch.int64, device=d)
        self.records = torch.empty(max(ss_record_bytes(n_splats), 16), dtype=torch.uint8, device=d)
        self.tile_offsets = torch.zeros(self.tiles + 1, dtype=torch.int32, device=d)
        self._alloc_pairs(max(int(pair_capacity), 1))
        self.image = torch.empty(3, H, W, dtype=torch.float32, device=d)
        self.T_final = torch.empty(H, W, dtype=torch.float32, device=d)
        self.last_contrib = torch.empty(H, W, dtype=torch.int32, device=d)
        self.median_depth = (torch.empty(H, W, dtype=torch.float32, device=d)
                             if flags & SS_MEDIAN_DEPTH else None)
        self.grads = {"dmean2d": torch.empty(n_splats, 2, dtype=torch.float32, device=d),
                      "dconic": torch.empty(n_splats, 3, dtype=torch.float32, device=d),
                      "dopacity": torch.empty(n_splats, dtype=torch.float32, device=d),
                      "drgb": torch.empty(n_splats, 3, dtype=torch.float32, device=d)}
        self.accum_weight = (torch.empty(n_splats, dtype=torch.float32, device=d)
                             if flags & SS_ACCUM_WEIGHT else None)
        stats = flags & SS_WEIGHT_STATS
        self.max_weight = torch.empty(n_splats, dtype=torch.float32, device=d) if stats else None
        self.blend_count = torch.empty(n_splats, dtype=torch.int32, device=d) if stats else None
        dist = flags & SS_DISTORTION
        self.distortion = torch.empty(H, W, dtype=torch.float32, device=d) if dist else None
        self.dist_totals = torch.empty(H, W, 4, dtype=torch.float32, device=d) if dist else None
        if dist:
            self.grads["ddepth"] = torch.empty(n_splats, dtype=torch.float32, device=d)
        self.n_pairs = 0
        self.culled = 0
        self._records_cleared = False   # the forward cleared the backward's records since the last sort

    def _alloc_pairs(self, cap: int):
        d = self.device
        self.capacity = cap
        self.keys = torch.empty(cap, dtype=torch.int64, device=d)
        self.vals = torch.empty(cap, dtype=torch.int32, device=d)
        self.blend_masks = torch.empty(8 * cap, dtype=torch.int32, device=d)
        ws = ss_workspace_bytes(self.n, cap, self.W, self.H)
        if ws == 0:
            raise ValueError("sizes out of range")
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=d)

    def bin_and_sort(self, splats: Splats, stream=None) -> int:
        """Tile lists of `splats`; returns the number of pairs (one host sync)."""
        ss_bin_tiles(splats, self.W, self.H, self.keys, self.vals, self.capacity, self.counters,
                     self.records, stream)
        st, pairs, culled = ss_pair_count(self.counters, self.capacity, stream)
        if st == SS_ERR_CAPACITY:
            self._alloc_pairs(int(pairs * 1.25) + 1024)
            ss_bin_tiles(splats, self.W, self.H, self.keys, self.vals, self.capacity,
                         self.counters, self.records, stream)
            st, pairs, culled = ss_pair_count(self.counters, self.capacity, stream)
            _check(st, "ss_pair_count")
        self.n_pairs, self.culled = pairs, culled
        ss_sort_pairs(self.keys, self.vals, pairs, self.W, self.H, self.tile_offsets,
                      self.workspace, stream)
        self._records_cleared = False   # the sort wrote the workspace
        return pairs

    def forward(self, splats: Splats = None, stream=None) -> None:
        """Composite; uses the records written by the last bin_and_sort.  Also
        clears the backward's gradient records in the workspace, so that the
        next backward() skips that pass; bin_and_sort() resets that, but a
        sort called directly on this workspace between forward() and
        backward() must be followed by forward() again."""
        ss_raster_fwd_records(self.records, self.n, self.vals, self.tile_offsets, self.n_pairs,
                              self.W, self.H, self.bg, self.flags, self.image, self.T_final,
                              self.last_contrib, self.median_depth, self.blend_masks,
                              self.max_weight, self.blend_count, self.distortion,
                              self.dist_totals, stream, bwd_workspace=self.workspace)
        self._records_cleared = True

    def backward(self, splats, dL_dimage: torch.Tensor, stream=None, dL_ddist=None) -> None:
        """Gradients; uses the records written by the last bin_and_sort.
        dL_ddist: [H, W] upstream gradient of the distortion (SS_DISTORTION)."""
        flags = self.flags | (SS_RECORDS_CLEARED if self._records_cleared else 0)
        ss_raster_bwd_records(self.records, self.n, self.vals, self.tile_offsets, self.n_pairs,
                              self.W, self.H, self.bg, flags, self.T_final, self.last_contrib,
                              self.blend_masks, dL_dimage, self.grads, self.accum_weight,
                              self.workspace, stream, self.dist_totals, dL_ddist)
        self._records_cleared = False   # the backward's sums are in them now

    def step(self, splats: Splats, dL_dimage: torch.Tensor, stream=None, dL_ddist=None) -> int:
        """One pass of the whole path: bin, sort, forward, backward."""
        n = self.bin_and_sort(splats, stream)
        self.forward(splats, stream)
        self.backward(splats, dL_dimage, stream, dL_ddist)
        return n

    def step_async(self, splats: Splats, dL_dimage: torch.Tensor, stream=None,
                   dL_ddist=None) -> None:
        """bin -> sort -> forward -> backward with the pair count kept on the
        device: no host synchronisation, so the step can be captured in a
        CUDA graph.  The pair buffers must already be large enough (size them
        with one step() first); check() reports an overflow afterwards."""
        ss_bin_tiles(splats, self.W, self.H, self.keys, self.vals, self.capacity, self.counters,
                     self.records, stream)
        ss_sort_pairs_dev(self.keys, self.vals, self.counters, self.capacity, self.W, self.H,
                          self.tile_offsets, self.workspace, stream)
        ss_raster_fwd_records(self.records, self.n, self.vals, self.tile_offsets, self.capacity,
                              self.W, self.H, self.bg, self.flags, self.image, self.T_final,
                              self.last_contrib, self.median_depth, self.blend_masks,
                              self.max_weight, self.blend_count, self.distortion,
                              self.dist_totals, stream, bwd_workspace=self.workspace)
        ss_raster_bwd_records(self.records, self.n, self.vals, self.tile_offsets, self.capacity,
                              self.W, self.H, self.bg, self.flags | SS_RECORDS_CLEARED,
                              self.T_final, self.last_contrib, self.blend_masks, dL_dimage,
                              self.grads, self.accum_weight, self.workspace, stream,
                              self.dist_totals, dL_ddist)

    def check(self, stream=None) -> None:
        """Raise if the last sort reported a device-side problem (capacity
        overflow, look-back timeout, out-of-range key)."""
        _check(ss_sort_status(self.workspace, stream), "sort status")

    def capture(self, splats: Splats, dL_dimage: torch.Tensor,
                dL_ddist=None) -> "torch.cuda.CUDAGraph":
        """A CUDA graph of step_async on these buffers (replay with .replay())."""
        self.step_async(splats, dL_dimage, dL_ddist=dL_ddist)   # first calls set attributes
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.step_async(splats, dL_dimage, dL_ddist=dL_ddist)
        return g


class StepPipeline:
    """The whole step (bin, sort, forward, backward) fed from and returned to
    pinned host memory, double-buffered across steps on one GPU.

    Two buffer sets, each a Rasterizer with its own captured CUDA graph and
    device input buffers, and three streams: step k's host-to-device input
    copy runs on one copy stream while step k-1 computes, step k's results
    (image, gradients, accumulated weight) come back on a second copy stream
    while step k+1 computes, and events order each buffer set's copy in,
    compute and copy out.  Every step still copies all of its inputs in and
    all of its results out; the copies overlap the other set's compute.

    The pair buffers must be sized first (the constructor runs one
    synchronous step on the given inputs); check() after run() reports a
    capacity overflow or another device-side problem of the last steps."""

    KEYS = ("mean2d", "conic", "opacity", "rgb", "depth")

    def __init__(self, W: int, H: int, n_splats: int, flags: int, host_splats: dict, host_dL,
                 bg=None, device="cuda", capacity=None):
        d = torch.device(device)
        self.device = d
        cap = capacity if capacity is not None else max(64, 3 * n_splats)
        self.r, self.dev_in, self.dev_dL, self.graphs = [], [], [], []
        for b in range(2):
            r = Rasterizer(W, H, n_splats, cap, flags, bg=bg, device=d)
            sp = Splats(**{k: torch.empty(host_splats[k].shape, dtype=torch.float32, device=d)
                           for k in self.KEYS})
            dL = torch.empty(host_dL.shape, dtype=torch.float32, device=d)
            for k in self.KEYS:
                getattr(sp, k).copy_(host_splats[k])
            dL.copy_(host_dL)
            r.step(sp, dL)                 # sizes the pair buffers (one host read)
            self.r.append(r)
            self.dev_in.append(sp)
            self.dev_dL.append(dL)
        for b in range(2):
            self.graphs.append(self.r[b].capture(self.dev_in[b], self.dev_dL[b]))
        torch.cuda.synchronize()
        self.h2d = torch.cuda.Stream(device=d)
        self.comp = torch.cuda.Stream(device=d)
        self.d2h = torch.cuda.Stream(device=d)
        ev = lambda: [torch.cuda.Event(), torch.cuda.Event()]  # noqa: E731
        self.in_ready, self.computed, self.out_read, self.in_free = ev(), ev(), ev(), ev()
        self.started = [False, False]

    def outputs(self, b: int) -> list:
        r = self.r[b]
        out = [r.image] + [r.grads[k] for k in ("dmean2d", "dconic", "dopacity", "drgb")]
        if r.accum_weight is not None:
            out.append(r.accum_weight)
        return out

    def host_output_buffers(self, pin=True) -> list:
        return [torch.empty(o.shape, dtype=o.dtype, pin_memory=pin) for o in self.outputs(0)]

    def submit(self, k: int, host_splats: dict, host_dL, host_out: list) -> None:
        """Enqueue step k: copy in, compute, copy out (all asynchronous)."""
        b = k & 1
        with torch.cuda.stream(self.h2d):
            if self.started[b]:
                self.h2d.wait_event(self.in_free[b])        # step k-2 has read its inputs
            for key in self.KEYS:
                getattr(self.dev_in[b], key).copy_(host_splats[key], non_blocking=True)
            self.dev_dL[b].copy_(host_dL, non_blocking=True)
            self.in_ready[b].record(self.h2d)
        with torch.cuda.stream(self.comp):
            self.comp.wait_event(self.in_ready[b])
            if self.started[b]:
                self.comp.wait_event(self.out_read[b])      # step k-2's results are out
            self.graphs[b].replay()
            self.computed[b].record(self.comp)
            self.in_free[b].record(self.comp)
        with torch.cuda.stream(self.d2h):
            self.d2h.wait_event(self.computed[b])
            for h, o in zip(host_out, self.outputs(b)):
                h.copy_(o, non_blocking=True)
            self.out_read[b].record(self.d2h)
        self.started[b] = True

    def run(self, steps: int, host_splats: dict, host_dL, host_outs: list) -> None:
        """Enqueue `steps` steps (host_outs: two lists of host output buffers,
        used alternately) and wait for all of them."""
        for k in range(steps):
            self.submit(k, host_splats, host_dL, host_outs[k & 1])
        self.d2h.synchronize()

    def check(self) -> None:
        torch.cuda.synchronize()
        for r in self.r:
            r.check()
