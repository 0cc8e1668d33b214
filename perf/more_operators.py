"""Cases of the operators that keep a training step's activations in 8 bits:
rows packed and unpacked, the root-mean-square norm with the residual's
addition and an output in 8 bits, the gradients of both norms from rows kept
in 8 bits, and the weight gradient of a dense layer from its input kept in 8
bits.

Between a scene's code table and its colours, every norm and every dense
layer keeps its input for the backward pass: 384 MB for 2,000,000 splats of
48 values in float32, 100 MB in 8 bits.  A group of 32 columns of a row has a
scale, the least power of two s with amax <= Q s (Q = 127 for int8, 448 for
e4m3, and s at least 2^-111); an element is held as x / s rounded.  The sizes
are the renderer's own scenes (256, 76,363 and 2,000,000 splats; 48 = 16 x 3
degree-3 colour coefficients) and generic ones.

`own` false computes the plain forms (elementary torch operations in 32
bits); `own` true calls the package.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
EPS = 1e-5           # both norms: added to the mean of squares
GROUP = 32           # columns that share a scale
LEAST = -111         # the least scale's exponent


def listed():
    return [
        # every splat's 48 values kept for the backward pass and read back
        {"name": "pack 2M x 48 f32 int8", "op": "pack", "n": 2000000, "D": 48, "dtype": "f32",
         "format": "int8", "pad": 0},
        # a few rows of an odd width: latency, and no vector alignment
        {"name": "pack 37 x 1001 f16 e4m3", "op": "pack", "n": 37, "D": 1001, "dtype": "f16",
         "format": "e4m3", "pad": 0},
        # every splat's values in a residual stack, in training
        {"name": "rms 2M x 48 f32", "op": "rms", "n": 2000000, "D": 48, "dtype": "f32",
         "pdtype": "f32", "residual": True, "out": "rows", "keep": "", "pad": 0},
        # a batch of 8K tokens, normalised straight into the 8 bits that the next product reads
        {"name": "rms 8191 x 4096 bf16 to e4m3", "op": "rms", "n": 8191, "D": 4096, "dtype": "bf16",
         "pdtype": "f32", "residual": True, "out": "e4m3", "keep": "", "pad": 0},
        # one token of a decoder: latency
        {"name": "rms 1 x 4096 bf16 to e4m3", "op": "rms", "n": 1, "D": 4096, "dtype": "bf16",
         "pdtype": "bf16", "residual": True, "out": "e4m3", "keep": "", "pad": 0},
        # the backward of the 2M splats' norm from what was kept
        {"name": "rms grad 2M x 48 f32 int8", "op": "rms_grad", "n": 2000000, "D": 48,
         "dtype": "f32", "pdtype": "f32", "format": "int8", "residual": True, "pad": 0},
        # wide rows in 16 bits with 32-bit weights, the residual's gradient joined
        {"name": "rms grad 8191 x 4096 bf16 e4m3", "op": "rms_grad", "n": 8191, "D": 4096,
         "dtype": "bf16", "pdtype": "f32", "format": "e4m3", "residual": True, "pad": 0},
        # the 76,363-splat scene's layer norm, backward from what was kept
        {"name": "norm grad 76363 x 48 f32 int8", "op": "norm_grad", "n": 76363, "D": 48,
         "dtype": "f32", "pdtype": "f32", "format": "int8", "pad": 0},
        # rows of an odd width: no two rows start alike
        {"name": "norm grad 16384 x 1001 bf16 int8", "op": "norm_grad", "n": 16384, "D": 1001,
         "dtype": "bf16", "pdtype": "bf16", "format": "int8", "pad": 0},
        # a dense layer over every splat: many rows, a small weight
        {"name": "dense grad 2M x 48 x 48 f32", "op": "dense_grad", "n": 2000000, "N": 48, "D": 48,
         "dtype": "f32", "gdtype": "f32", "format": "int8", "pad": 0},
        # a dense layer of 4096 over 8K tokens: a matrix product's work
        {"name": "dense grad 8191 x 4096 x 4096", "op": "dense_grad", "n": 8191, "N": 4096,
         "D": 4096, "dtype": "bf16", "gdtype": "bf16", "format": "e4m3", "pad": 0},
        # the smallest scene's dense layer: latency
        {"name": "dense grad 256 x 48 x 48 bf16", "op": "dense_grad", "n": 256, "N": 48, "D": 48,
         "dtype": "bf16", "gdtype": "f32", "format": "int8", "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """The ranges behind the listed cases: one row to two million, widths 1 to
    8192 (dense layers: 1 to 4096 on both sides)."""
    op = rng.choice(["pack", "rms", "rms", "rms_grad", "norm_grad", "dense_grad", "dense_grad"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    pad = rng.choice([0, 0, 0, 1, 8])                          # unused values after each row
    case = {"op": op, "dtype": dtype, "format": rng.choice(["int8", "e4m3"]), "pad": pad}
    if op == "dense_grad":
        D, N = _log_int(rng, 1, 4096), _log_int(rng, 1, 4096)
        most = min(2000000, 60000000 // (N + D), 110000000000 // (N * D))
        case.update({"n": _log_int(rng, 1, most), "N": N, "D": D,
                     "gdtype": rng.choice([dtype, "f32"])})
        return case
    D = _log_int(rng, 1, 8192) if rng.random() < 0.6 else rng.choice([3, 16, 48, 64, 256, 1024, 2000])
    case.update({"n": _log_int(rng, 1, min(2000000, 60000000 // D)), "D": D})
    if op != "pack":
        case["pdtype"] = rng.choice([dtype, "f32"])
    if op in ("rms", "rms_grad"):
        case["residual"] = rng.random() < 0.7
    if op == "rms":
        del case["format"]
        case["out"] = rng.choice(["rows", "rows", "int8", "e4m3"])
        case["keep"] = rng.choice(["", "", "int8", "e4m3"])
    return case


# ------------------------------------------------------------------ inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(values, dtype, pad):
    """`values` [n, D] in `dtype`, each row followed by `pad` unused values."""
    n, D = values.shape
    buf = torch.zeros(n, D + pad, dtype=dtype, device="cuda")
    buf[:, :D].copy_(values)
    return buf[:, :D]


def _activations(case, g):
    """Rows of different sizes, a few columns much larger than the others, and
    one row in 64 all zeros (a splat without a code, a padded token)."""
    n, D = case["n"], case["D"]
    x = _normal(g, n, D) * (0.5 + torch.rand(n, 1, generator=g, device="cuda"))
    x *= torch.where(torch.rand(D, generator=g, device="cuda") < 0.02, 8.0, 1.0)
    x += 0.2 * _normal(g, n, 1)
    if n > 64:
        x *= torch.rand(n, 1, generator=g, device="cuda") >= 1 / 64
    return _rows(x, DTYPES[case["dtype"]], case["pad"])


def _power(s):
    """2^s in float32, for whole s in -126 .. 127."""
    return ((s + 127).to(torch.int32) << 23).view(torch.float32)


def _pack(x, fmt):
    """(held values [n, groups, 32] as they are before their scale, exponents [n, groups])."""
    n, D = x.shape
    groups = -(-D // GROUP)
    v = torch.zeros(n, groups * GROUP, dtype=torch.float32, device=x.device)
    v[:, :D] = x
    v = v.view(n, groups, GROUP)
    m, p = torch.frexp(v.abs().amax(2))                        # m in [1/2, 1), or 0
    top, bits = (127 / 128, 7) if fmt == "int8" else (448 / 512, 9)
    s = (p - bits + (m > top).int()).clamp(min=LEAST)
    s = torch.where(m == 0, torch.full_like(s, LEAST), s)
    z = v * _power(-s)[:, :, None]
    return (z.round() if fmt == "int8" else z.to(torch.float8_e4m3fn).float()), s


def _unpack(held, D):
    v, s = held
    return (v * _power(s)[:, :, None]).reshape(len(v), -1)[:, :D]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    st = {"case": case, "op": case["op"]}
    op, n, D, t = case["op"], case["n"], case["D"], DTYPES[case["dtype"]]
    x = _activations(case, g)
    if own:
        import gaussian_splatting_differentiable_gb300 as ss
    if op == "pack":
        st["x"] = x
        if own:
            st["kept"] = ss.Rows8(n, D, FORMATS[case["format"]])
            st["back"] = torch.empty(n, D, dtype=t, device="cuda")
        return st
    if op == "dense_grad":
        st["dy"] = _rows(_normal(g, n, case["N"]) * 0.1, t, case["pad"])
        if own:
            st["kept"] = ss.Rows8(n, D, FORMATS[case["format"]]).pack(x)
            st["layer"] = ss.DenseGrad(n, case["N"], D, dtype=t, grad_dtype=DTYPES[case["gdtype"]])
        else:
            st["held"] = _pack(x, case["format"])
        return st
    p = DTYPES[case["pdtype"]]
    st["gamma"] = (1 + 0.1 * _normal(g, D)).to(p)
    if op == "rms":
        st["x"] = x
        st["residual"] = _activations(case, g) if case["residual"] else None
        if own:
            st["norm"] = ss.RMSNorm(n, D, eps=EPS, dtype=t, param_dtype=p, residual=case["residual"],
                                    out=FORMATS.get(case["out"]), keep=FORMATS.get(case["keep"]),
                                    backward=False)
            st["values"] = torch.empty(n, D, dtype=torch.bfloat16, device="cuda")
            st["back"] = torch.empty(n, D, dtype=t, device="cuda")
        return st
    st["dy"] = _rows(_normal(g, n, D) * 0.1, t, case["pad"])
    xf = x.float()
    st["mean"] = xf.mean(1)
    c = xf - st["mean"][:, None] if op == "norm_grad" else xf
    st["rstd"] = ((c * c).mean(1) + EPS) ** -0.5
    if op == "rms_grad":
        st["dsum"] = _rows(_normal(g, n, D) * 0.1, t, case["pad"]) if case["residual"] else None
    if own:
        st["kept"] = ss.Rows8(n, D, FORMATS[case["format"]]).pack(x)
        kind = ss.RMSNorm if op == "rms_grad" else ss.LayerNorm
        st["norm"] = kind(n, D, eps=EPS, dtype=t, param_dtype=p, forward=False)
    else:
        st["held"] = _pack(x, case["format"])
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    op = st["op"]
    if op == "pack":
        return {"values": st["kept"].pack(st["x"]).unpack(st["back"])}
    if op == "dense_grad":
        layer = st["layer"]
        layer.backward(st["dy"], st["kept"])
        return {"dweight": layer.grads["dweight"], "dbias": layer.grads["dbias"]}
    norm = st["norm"]
    if op == "rms":
        y = norm.forward(st["x"], st["gamma"], st["residual"])
        out = {"y": y.unpack(st["values"]) if norm.out is not None else y, "rstd": norm.rstd}
        if st["residual"] is not None:
            out["sum"] = norm.sum
        if norm.kept is not None:
            out["kept"] = norm.kept.unpack(st["back"])
        return out
    if op == "rms_grad":
        dx = norm.backward(st["dy"], st["kept"], st["gamma"], st["dsum"], rstd=st["rstd"])
        return {"dx": dx, "dgamma": norm.grads["dgamma"]}
    dx = norm.backward(st["dy"], st["kept"], st["gamma"], st["mean"], st["rstd"])
    return {"dx": dx, "dgamma": norm.grads["dgamma"], "dbeta": norm.grads["dbeta"]}


def _run_plain(st):
    case, op, D = st["case"], st["op"], st["case"]["D"]
    t = DTYPES[case["dtype"]]
    if op == "pack":
        return {"values": _unpack(_pack(st["x"], case["format"]), D).to(t)}
    if op == "dense_grad":
        dy = st["dy"].float()
        g = DTYPES[case["gdtype"]]
        return {"dweight": (dy.t() @ _unpack(st["held"], D)).to(g), "dbias": dy.sum(0).to(g)}
    if op == "rms":
        s = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(t)
        h = s.float()
        rstd = ((h * h).mean(1) + EPS) ** -0.5
        y = h * rstd[:, None] * st["gamma"].float()
        y = y.to(t) if case["out"] == "rows" else _unpack(_pack(y, case["out"]), D).bfloat16()
        out = {"y": y, "rstd": rstd}
        if st["residual"] is not None:
            out["sum"] = s
        if case["keep"]:
            out["kept"] = _unpack(_pack(s, case["keep"]), D).to(t)
        return out
    dy, rstd, p = st["dy"].float(), st["rstd"][:, None], st["gamma"].dtype
    x = _unpack(st["held"], D)
    if op == "rms_grad":
        xh = x * rstd
        w = dy * st["gamma"].float()
        dx = rstd * (w - xh * (w * xh).mean(1, keepdim=True))
        if st["dsum"] is not None:
            dx = dx + st["dsum"].float()
        return {"dx": dx.to(t), "dgamma": (dy * xh).sum(0).to(p)}
    xh = (x - st["mean"][:, None]) * rstd
    dgamma, dbeta = (dy * xh).sum(0), dy.sum(0)
    w = dy * st["gamma"].float()
    dx = rstd * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    return {"dx": dx.to(t), "dgamma": dgamma.to(p), "dbeta": dbeta.to(p)}


# ------------------------------------------------------------------ in 64 bits

def _power64(s):
    """2^s in float64, exactly."""
    return ((s.long() + 1023) << 52).view(torch.float64)


def _held_exactly(x, fmt):
    """What 8 bits hold of x [n, D], in float64, by the definition: the least
    power of two s with max |x| <= Q s, and the nearest number that the format has,
    times s."""
    n, D = x.shape
    x = x.double()
    parts = []
    for c in range(0, D, GROUP):
        v = x[:, c:c + GROUP]
        m, e = torch.frexp(v.abs().max(1, keepdim=True).values / (127.0 if fmt == "int8" else 448.0))
        e = torch.where(m > 0.5, e, e - 1)                     # ceil(log2) of m 2^e, m in [1/2, 1)
        e = torch.where(m > 0, e, torch.full_like(e, LEAST)).clamp(min=LEAST)
        z = v * _power64(-e)
        if fmt == "int8":
            z = torch.round(z)
        else:   # three bits after the leading one, down to 2^-6; below that, steps of 2^-9
            lead = (torch.frexp(z).exponent - 1).clamp(min=-6)
            z = torch.round(z * _power64(3 - lead)) * _power64(lead - 3)
        parts.append(z * _power64(e))
    return torch.cat(parts, 1)


def exact(case, seed):
    st = prepare(dict(case), seed)
    op, n, D = case["op"], case["n"], case["D"]
    if op == "pack":
        return {"values": _held_exactly(st["x"], case["format"])}
    if op == "rms":
        x = st["x"].double()
        out = {}
        if st["residual"] is not None:      # rounded once, as the residual stream keeps it
            x = (x + st["residual"].double()).to(st["x"].dtype).double()
            out["sum"] = x
        rstd = 1.0 / torch.sqrt(torch.einsum("nd,nd->n", x, x) / D + EPS)
        y = torch.einsum("nd,n,d->nd", x, rstd, st["gamma"].double())
        out["y"] = y if case["out"] == "rows" else _held_exactly(y, case["out"])
        out["rstd"] = rstd
        if case["keep"]:
            out["kept"] = _held_exactly(x, case["keep"])
        return out
    dy = st["dy"].double()
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    x = _held_exactly(_activations(case, g), case["format"])
    if op == "dense_grad":
        return {"dweight": torch.einsum("mn,mk->nk", dy, x), "dbias": dy.sum(0)}
    s = st["rstd"].double()[:, None]
    a = dy * st["gamma"].double()
    if op == "rms_grad":
        xh = x * s
        dx = (a - xh * (torch.einsum("nd,nd->n", a, xh) / D)[:, None]) * s
        if st["dsum"] is not None:
            dx += st["dsum"].double()
        return {"dx": dx, "dgamma": torch.einsum("nd,nd->d", dy, xh)}
    xh = (x - st["mean"].double()[:, None]) * s
    both = torch.stack([a.sum(1), torch.einsum("nd,nd->n", a, xh)], 1) / D
    dx = (a - both[:, :1] - xh * both[:, 1:]) * s
    return {"dx": dx, "dgamma": torch.einsum("nd,nd->d", dy, xh), "dbeta": dy.sum(0)}


# ------------------------------------------------------------------ the work

def work(case):
    """Every input once and every output once; what is packed and read back
    within a pass counts once each way."""
    op, n, D, e = case["op"], case["n"], case["D"], BYTES[case["dtype"]]
    held = n * (D + -(-D // GROUP))
    if op == "pack":
        return {"bytes": 2 * n * D * e + 2 * held, "flops": 6 * n * D}
    if op == "dense_grad":
        N, b = case["N"], BYTES[case["gdtype"]]
        return {"bytes": n * N * e + held + (N * D + N) * b, "flops": 2 * n * N * D + n * N}
    p = D * BYTES[case["pdtype"]]
    if op == "rms":
        b = n * D * e * (3 if case["residual"] else 1) + 4 * n + p
        b += n * D * e if case["out"] == "rows" else 2 * held + 2 * n * D
        b += 2 * held + n * D * e if case["keep"] else 0
        return {"bytes": b, "flops": 6 * n * D}
    if op == "rms_grad":
        return {"bytes": n * D * e * (3 if case["residual"] else 2) + held + 4 * n + 2 * p,
                "flops": 12 * n * D}
    return {"bytes": 2 * n * D * e + held + 8 * n + 3 * p, "flops": 14 * n * D}
