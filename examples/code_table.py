"""Train a splat scene whose colours come from a learned code table.

    python examples/code_table.py [--splats N] [--codes V] [--steps K] [--keep int8|e4m3]

Every splat names a row of a table of V codes of 48 values.  A step looks the
rows up and scales them, normalises each (layer norm with learned weights),
takes the result as the splat's degree-3 colour coefficients, projects and
rasterizes the splats, compares the image with a target (L1 + SSIM), sends the
gradients all the way back (rasterizer, projection, layer norm, table), clips
the gradients of everything that is learned by their common norm, and moves
against them.  With --keep, what the norm's backward pass needs of its input is
kept in 8 bits from the forward on, as layers in between would have it; the lookup's
rows are a buffer of its own and stay, so this one norm saves no memory by it.  The target is
the same scene with colours of its own; all data is synthetic.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import gaussian_splatting_differentiable_gb300 as ss  # noqa: E402
from synth.scene3d import make_scene3d  # noqa: E402

COEFFICIENTS = 16     # of degree 3, for each of 3 colours
FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
RATES = {"table": 2.0, "gamma": 0.5, "beta": 0.5, "opacity": 0.2, "mean3": 1e-4, "scale": 1e-4,
         "quat": 1e-3}


class CodeTableScene:
    """A scene's parameters, the buffers of every step, and the step itself."""

    def __init__(self, scene, codes: int, max_norm: float = 0.03, seed: int = 0, device="cuda",
                 keep=None):
        d = torch.device(device)
        g = torch.Generator(device=d).manual_seed(seed)
        n, D = scene.n, 3 * COEFFICIENTS
        c = scene.cam
        self.cam = ss.camera(c.R, c.t, c.fx, c.fy, c.cx, c.cy, c.near, c.blur)
        self.splats = ss.Splats3D.from_numpy(scene, d)
        self.params = {
            "table": torch.randn(codes, D, generator=g, device=d) / D ** 0.5,
            "gamma": torch.full((D,), 0.2, device=d),
            "beta": torch.zeros(D, device=d),
            "opacity": torch.from_numpy(scene.opacity).to(d),
            "mean3": self.splats.mean3, "scale": self.splats.scale, "quat": self.splats.quat,
        }
        # one splat in 64 has no code: its coefficients are the layer norm's offsets
        ids = torch.randint(0, codes, (n,), generator=g, device=d)
        self.ids = torch.where(torch.arange(n, device=d) % 64 == 63, -1, ids)
        self.lookup = ss.Embedding(n, codes, D, scale=D ** 0.5, device=d)
        self.norm = ss.LayerNorm(n, D, device=d)
        self.kept = None if keep is None else ss.Rows8(n, D, keep, device=d)
        self.projector = ss.Projector(n, 3, d)
        self.raster = ss.Rasterizer(scene.W, scene.H, n, 8 * n, device=d)
        self.loss = ss.SsimLoss(3, scene.H, scene.W, device=d)
        self.dcoef = torch.empty(n, D, device=d)
        self.grads = {"table": self.lookup.grad, "gamma": self.norm.grads["dgamma"],
                      "beta": self.norm.grads["dbeta"], "opacity": self.raster.grads["dopacity"],
                      "mean3": self.projector.grads["dmean3"], "scale": self.projector.grads["dscale"],
                      "quat": self.projector.grads["dquat"]}
        self.clip = ss.GradClip(list(self.grads.values()), device=d)
        self.max_norm = max_norm

    def render(self) -> torch.Tensor:
        codes = self.lookup.forward(self.params["table"], self.ids)
        coef = self.norm.forward(codes, self.params["gamma"], self.params["beta"])
        if self.kept is not None:
            self.kept.pack(codes)
        self.splats.sh.view(coef.shape[1], -1).copy_(coef.t())     # [16, 3, n]
        self.projector.forward(self.splats, self.cam)
        self.flat = self.projector.splats2d(self.params["opacity"])
        self.raster.bin_and_sort(self.flat)
        self.raster.forward(self.flat)
        return self.raster.image

    def backward(self, dimage: torch.Tensor) -> None:
        self.raster.backward(self.flat, dimage)
        r = self.raster.grads
        self.projector.backward(self.splats, self.cam, r["dmean2d"], r["dconic"], r["drgb"])
        self.dcoef.copy_(self.projector.grads["dsh"].view(self.dcoef.shape[1], -1).t())
        codes = self.lookup.out if self.kept is None else self.kept
        dcodes = self.norm.backward(self.dcoef, codes, self.params["gamma"])
        self.lookup.backward(dcodes, self.ids)

    def step(self, target: torch.Tensor) -> torch.Tensor:
        """One training step; the loss stays on the device."""
        self.backward(self.loss(self.render(), target))
        self.clip(self.max_norm)                                   # in place
        for k, p in self.params.items():
            p.add_(self.grads[k], alpha=-RATES[k])
        self.params["opacity"].clamp_(0.01, 0.99)
        self.params["scale"].clamp_(min=1e-4)
        return self.loss.loss[0].clone()


def target_of(scene, device="cuda") -> torch.Tensor:
    """The scene's image with its own colour coefficients."""
    c = scene.cam
    sp = ss.Splats3D.from_numpy(scene, device)
    pr = ss.Projector(scene.n, scene.sh_degree, device)
    pr.forward(sp, ss.camera(c.R, c.t, c.fx, c.fy, c.cx, c.cy, c.near, c.blur))
    r = ss.Rasterizer(scene.W, scene.H, scene.n, 8 * scene.n, device=device)
    flat = pr.splats2d(torch.from_numpy(scene.opacity).to(device))
    r.bin_and_sort(flat)
    r.forward(flat)
    return r.image.clone()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--splats", type=int, default=5207)
    ap.add_argument("--codes", type=int, default=256)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--keep", choices=sorted(FORMATS))
    a = ap.parse_args()
    scene = make_scene3d(11, n=a.splats, W=256, H=256)
    target = target_of(scene)
    model = CodeTableScene(scene, a.codes, keep=FORMATS.get(a.keep))
    losses = [model.step(target) for _ in range(a.steps)]
    for k in sorted({0, a.steps // 4, a.steps // 2, a.steps - 1}):
        print("step %4d: loss %.5f" % (k, float(losses[k])))
    print("last step's gradient norm %.4g, scaled by %.4g" % tuple(model.clip.result.tolist()))


if __name__ == "__main__":
    main()
