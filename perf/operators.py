"""Cases of the operators that learn a scene's code table: the scaled lookup
of code rows and its gradient by sorted ids, layer normalisation forward and
backward, and the clipping of all gradients by their common norm.

A splat that does not own its features names a row of a table; the row is
scaled, normalised and used as the splat's colour coefficients, the gradients
come back the same way, and all of a step's gradients are clipped together.
The sizes are the renderer's own scenes (256, 5,207, 76,363 and 2,000,000
splats; 48 = 16 x 3 degree-3 colour coefficients, 59 trained values a splat)
and generic ones.

`own` false computes the plain forms (elementary torch operations in 32
bits); `own` true calls the package.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
NORM_EPS = 1e-5      # layer norm: added to the variance
CLIP_EPS = 1e-6      # clipping: added to the norm
BUCKET_SEED = 17     # the sizes of a bucket's tensors are part of the case, not of its inputs


def listed():
    return [
        # every splat of the 2M-splat scene takes its 48 colour coefficients from a 64K-row table
        {"name": "lookup 2M x 48 f32", "op": "lookup", "n": 2000000, "V": 65536, "D": 48,
         "dtype": "f32", "ids": "i64", "spread": "uniform", "absent": 0.0, "pad": 0},
        # the smallest scene's splats: one call's latency
        {"name": "lookup 256 x 48 bf16", "op": "lookup", "n": 256, "V": 1000, "D": 48,
         "dtype": "bf16", "ids": "i32", "spread": "uniform", "absent": 0.0, "pad": 0},
        # the 2M splats' gradients summed into a 4K-row code book, a few codes much in use
        {"name": "table grad 2M x 48 f32", "op": "table_grad", "n": 2000000, "V": 4096, "D": 48,
         "dtype": "f32", "gdtype": "f32", "ids": "i64", "spread": "log", "absent": 0.0, "pad": 0},
        # a batch of 8K tokens against a 64,000-row vocabulary, some of them without a row;
        # most of the rows get no gradient
        {"name": "table grad 8191 x 1024 bf16", "op": "table_grad", "n": 8191, "V": 64000,
         "D": 1024, "dtype": "bf16", "gdtype": "bf16", "ids": "i64", "spread": "log",
         "absent": 0.05, "pad": 0},
        # the smallest scene again, its gradient
        {"name": "table grad 256 x 48 f32", "op": "table_grad", "n": 256, "V": 1000, "D": 48,
         "dtype": "f32", "gdtype": "f32", "ids": "i32", "spread": "uniform", "absent": 0.0,
         "pad": 0},
        # every splat's 48 coefficients normalised
        {"name": "norm 2M x 48 f32", "op": "norm", "n": 2000000, "D": 48, "dtype": "f32",
         "pdtype": "f32", "pad": 0},
        # a few rows of an odd width: latency, and no vector alignment
        {"name": "norm 37 x 1001 f16", "op": "norm", "n": 37, "D": 1001, "dtype": "f16",
         "pdtype": "f16", "pad": 0},
        # the 76,363-splat scene's backward, weight gradients from many narrow rows
        {"name": "norm grad 76363 x 48 f32", "op": "norm_grad", "n": 76363, "D": 48,
         "dtype": "f32", "pdtype": "f32", "pad": 0},
        # wide rows in 16 bits with 32-bit weights
        {"name": "norm grad 8191 x 4096 bf16", "op": "norm_grad", "n": 8191, "D": 4096,
         "dtype": "bf16", "pdtype": "f32", "pad": 0},
        # all gradients of the 2M-splat scene: five tensors, 472 MB
        {"name": "clip 2M splats f32", "op": "clip", "kind": "splats", "n": 2000000,
         "dtype": "f32", "share": 0.5},
        # 300 ragged tensors as views of one flat bucket for each type
        {"name": "clip 300 tensors mixed", "op": "clip", "kind": "bucket", "tensors": 300,
         "total": 40000000, "dtype": "mixed", "share": 0.25},
        # the smallest scene's gradients: latency
        {"name": "clip 256 splats f32", "op": "clip", "kind": "splats", "n": 256, "dtype": "f32",
         "share": 0.5},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """The ranges behind the listed cases: one row to two million, widths 1 to
    8192, tables of 1 to 262,144 rows, lists of 1 to 600 tensors."""
    op = rng.choice(["lookup", "table_grad", "table_grad", "norm", "norm_grad", "clip"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "clip":
        if rng.random() < 0.5:
            return {"op": op, "kind": "splats", "n": _log_int(rng, 1, 1900000), "dtype": dtype,
                    "share": rng.choice([0.1, 0.7, 2.0])}
        tensors = _log_int(rng, 1, 600)
        return {"op": op, "kind": "bucket", "tensors": tensors,
                "total": max(tensors, _log_int(rng, 1000, 100000000)),
                "dtype": rng.choice([dtype, "mixed"]), "share": rng.choice([0.1, 0.7, 2.0])}
    D = _log_int(rng, 1, 8192) if rng.random() < 0.6 else rng.choice([3, 16, 48, 64, 256, 1024, 2000])
    cap = 90000000 if op in ("lookup", "norm") else 60000000   # elements of one [n, D] tensor
    n = _log_int(rng, 1, min(2000000, cap // D))
    pad = rng.choice([0, 0, 0, 1, 8])                          # unused values after each row
    case = {"op": op, "n": n, "D": D, "dtype": dtype, "pad": pad}
    if op in ("lookup", "table_grad"):
        case.update({"V": _log_int(rng, 1, min(262144, max(1, cap // D))), "ids": rng.choice(["i32", "i64"]),
                     "spread": rng.choice(["uniform", "log", "log", "one"]),
                     "absent": rng.choice([0.0, 0.0, 0.1])})
        if op == "table_grad":
            case["gdtype"] = rng.choice([dtype, "f32"])
    else:
        case["pdtype"] = rng.choice([dtype, "f32"])
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


def _ids(case, g):
    n, V = case["n"], case["V"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    if case["spread"] == "uniform":
        ids = (u * V).long()
    elif case["spread"] == "log":                      # row k about as often as 1 / (k + 1)
        ids = ((u * math.log(V + 1)).exp() - 1).long()
    else:                                              # nine in ten name one row
        ids = torch.where(u < 0.9, torch.full_like(u, V // 2), (u - 0.9) * 10 * V).long()
    ids = ids.clamp(0, V - 1)
    if case["absent"]:
        gone = torch.rand(n, generator=g, device="cuda") < case["absent"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)


def _bucket_sizes(case):
    rng = random.Random(BUCKET_SEED + case["tensors"])
    w = [math.exp(rng.uniform(0.0, math.log(2000.0))) for _ in range(case["tensors"])]
    s = sum(w)
    return [max(1, int(case["total"] * x / s)) for x in w]


def _clip_tensors(case, g):
    """(gradients, buffers of the same layout for the results, the whole
    buffers, the whole results)."""
    if case["kind"] == "splats":
        n, t = case["n"], DTYPES[case["dtype"]]
        shapes = [(n, 3), (n, 3), (n, 4), (16, 3, n), (n,)]    # mean, scale, rotation, colour, opacity
        sizes = [1e-4, 1e-3, 1e-4, 1e-2, 1e-2]
        if case["dtype"] == "f16":
            sizes = [1e-2] * 5                                 # scaled losses keep 16 bits in range
        grads = [(_normal(g, *s) * k).to(t) for s, k in zip(shapes, sizes)]
        outs = [torch.empty_like(x) for x in grads]
        return grads, outs, grads, outs
    kinds = ["f32", "bf16"] if case["dtype"] == "mixed" else [case["dtype"]]
    lens = [0] * len(kinds)
    where = []
    for i, size in enumerate(_bucket_sizes(case)):
        b = i % len(kinds)
        where.append((b, lens[b], size))
        lens[b] += size
    whole = [(_normal(g, max(1, m)) * 1e-2).to(DTYPES[k]) for m, k in zip(lens, kinds)]
    results = [torch.zeros_like(x) for x in whole]
    return ([whole[b][o:o + s] for b, o, s in where], [results[b][o:o + s] for b, o, s in where],
            [x[:m] for x, m in zip(whole, lens)], [x[:m] for x, m in zip(results, lens)])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    st = {"case": case, "op": case["op"]}
    op = case["op"]
    if op == "clip":
        st["grads"], st["outs"], st["whole"], st["results"] = _clip_tensors(case, g)
        norm = math.sqrt(sum(float(x.double().square().sum()) for x in st["whole"]))
        st["max_norm"] = case["share"] * norm
        if own:
            import gaussian_splatting_differentiable_gb300 as ss
            st["clip"] = ss.GradClip(st["grads"], st["outs"], eps=CLIP_EPS)
        return st
    n, D, t = case["n"], case["D"], DTYPES[case["dtype"]]
    if op in ("lookup", "table_grad"):
        st["scale"] = math.sqrt(D)
        st["ids"] = _ids(case, g)
        if op == "lookup":
            st["table"] = _rows(_normal(g, case["V"], D) / math.sqrt(D), t, case["pad"])
        else:
            st["dout"] = _rows(_normal(g, n, D) * 0.1, t, case["pad"])
        if own:
            import gaussian_splatting_differentiable_gb300 as ss
            st["embed"] = ss.Embedding(n, case["V"], D, scale=st["scale"], dtype=t,
                                       grad_dtype=DTYPES[case.get("gdtype", case["dtype"])],
                                       forward=op == "lookup", backward=op == "table_grad")
        return st
    p = DTYPES[case["pdtype"]]
    x = _normal(g, n, D) * (0.5 + torch.rand(n, 1, generator=g, device="cuda")) + 0.3 * _normal(g, n, 1)
    st["x"] = _rows(x, t, case["pad"])
    st["gamma"] = (1 + 0.1 * _normal(g, D)).to(p)
    st["beta"] = (0.1 * _normal(g, D)).to(p)
    if op == "norm_grad":
        st["dy"] = _rows(_normal(g, n, D) * 0.1, t, case["pad"])
        xf = st["x"].float()
        st["mean"] = xf.mean(1)
        st["rstd"] = (((xf - st["mean"][:, None]) ** 2).mean(1) + NORM_EPS) ** -0.5
    if own:
        import gaussian_splatting_differentiable_gb300 as ss
        st["ln"] = ss.LayerNorm(n, D, eps=NORM_EPS, dtype=t, param_dtype=p,
                                forward=op == "norm", backward=op == "norm_grad")
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    op = st["op"]
    if op == "lookup":
        return {"out": st["embed"].forward(st["table"], st["ids"])}
    if op == "table_grad":
        return {"dtable": st["embed"].backward(st["dout"], st["ids"])}
    if op == "norm":
        ln = st["ln"]
        y = ln.forward(st["x"], st["gamma"], st["beta"])
        return {"y": y, "mean": ln.mean, "rstd": ln.rstd}
    if op == "norm_grad":
        ln = st["ln"]
        dx = ln.backward(st["dy"], st["x"], st["gamma"], st["mean"], st["rstd"])
        return {"dx": dx, "dgamma": ln.grads["dgamma"], "dbeta": ln.grads["dbeta"]}
    return {"norm_coef": st["clip"](st["max_norm"]), "grads": st["results"]}


def _run_plain(st):
    case, op = st["case"], st["op"]
    if op == "lookup":
        ids = st["ids"].long()
        here = (ids >= 0) & (ids < case["V"])
        rows = st["table"][ids.clamp(0, case["V"] - 1)].float() * st["scale"]
        return {"out": torch.where(here[:, None], rows, 0.0).to(st["table"].dtype)}
    if op == "table_grad":
        ids = st["ids"].long()
        here = (ids >= 0) & (ids < case["V"])
        d = torch.where(here[:, None], st["dout"].float(), 0.0)
        dt = torch.zeros(case["V"], case["D"], dtype=torch.float32, device=d.device)
        dt.index_add_(0, ids.clamp(0, case["V"] - 1), d)
        return {"dtable": (dt * st["scale"]).to(DTYPES[case["gdtype"]])}
    if op == "norm":
        x = st["x"].float()
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = ((c * c).mean(1) + NORM_EPS) ** -0.5
        y = c * rstd[:, None] * st["gamma"].float() + st["beta"].float()
        return {"y": y.to(st["x"].dtype), "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        dy, rstd = st["dy"].float(), st["rstd"][:, None]
        xh = (st["x"].float() - st["mean"][:, None]) * rstd
        dgamma, dbeta = (dy * xh).sum(0), dy.sum(0)
        w = dy * st["gamma"].float()
        dx = rstd * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
        p = st["gamma"].dtype
        return {"dx": dx.to(st["x"].dtype), "dgamma": dgamma.to(p), "dbeta": dbeta.to(p)}
    total = torch.stack([(x.float() ** 2).sum() for x in st["whole"]]).sum()
    norm = total.sqrt()
    coef = (st["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    return {"norm_coef": torch.stack([norm, coef]),
            "grads": [(x.float() * coef).to(x.dtype) for x in st["whole"]]}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        flat = [x.reshape(-1).double() for x in st["whole"]]
        norm = math.sqrt(math.fsum(float(torch.dot(x, x)) for x in flat))
        coef = min(1.0, st["max_norm"] / (norm + CLIP_EPS))
        return {"norm_coef": torch.tensor([norm, coef], dtype=torch.float64),
                "grads": [x.double().mul_(coef) for x in st["whole"]]}
    if op == "lookup":
        big = torch.cat([st["table"].double() * st["scale"],
                         torch.zeros(1, case["D"], dtype=torch.float64, device="cuda")])
        ids = st["ids"].long()
        return {"out": big[torch.where((ids < 0) | (ids >= case["V"]), case["V"], ids)]}
    if op == "table_grad":
        # rows of one id side by side; a row's sum is a difference of running sums
        ids = st["ids"].long()
        kept = torch.nonzero((ids >= 0) & (ids < case["V"])).squeeze(1)
        sids, order = torch.sort(ids[kept])
        edge = torch.searchsorted(sids, torch.arange(case["V"] + 1, device="cuda"))
        out = torch.empty(case["V"], case["D"], dtype=torch.float64, device="cuda")
        for c in range(0, case["D"], 512):
            part = st["dout"][:, c:c + 512][kept[order]].double()
            run_ = torch.cat([torch.zeros_like(part[:1]) if len(part) else
                              torch.zeros(1, out[:, c:c + 512].shape[1], dtype=torch.float64,
                                          device="cuda"), part.cumsum(0)])
            out[:, c:c + 512] = (run_[edge[1:]] - run_[edge[:-1]]) * st["scale"]
        return {"dtable": out}
    x = st["x"].double()
    if op == "norm":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + NORM_EPS)
        y = torch.addcmul(st["beta"].double(), (x - mean[:, None]).mul_(rstd[:, None]), st["gamma"].double())
        return {"y": y, "mean": mean, "rstd": rstd}
    # the gradient of sum(dy * y), from mean and rstd as they are given
    dy, s = st["dy"].double(), st["rstd"].double()[:, None]
    xh = (x - st["mean"].double()[:, None]) * s
    a = dy * st["gamma"].double()
    both = torch.stack([a.sum(1), torch.einsum("nd,nd->n", a, xh)], 1) / case["D"]
    dx = (a - both[:, :1] - xh * both[:, 1:]) * s
    return {"dx": dx, "dgamma": torch.einsum("nd,nd->d", dy, xh), "dbeta": dy.sum(0)}


# ------------------------------------------------------------------ the work

def work(case):
    """Every input once and every output once."""
    op = case["op"]
    if op == "clip":
        if case["kind"] == "splats":
            b = 59 * case["n"] * BYTES[case["dtype"]]
            e = 59 * case["n"]
        else:
            kinds = ["f32", "bf16"] if case["dtype"] == "mixed" else [case["dtype"]]
            sizes = _bucket_sizes(case)
            e = sum(sizes)
            b = sum(s * BYTES[kinds[i % len(kinds)]] for i, s in enumerate(sizes))
        return {"bytes": 2 * b + 8, "flops": 3 * e}
    n, D, e = case["n"], case["D"], BYTES[case["dtype"]]
    if op in ("lookup", "table_grad"):
        idb = n * (4 if case["ids"] == "i32" else 8)
        if op == "lookup":
            return {"bytes": idb + min(n, case["V"]) * D * e + n * D * e, "flops": n * D}
        return {"bytes": idb + n * D * e + case["V"] * D * BYTES[case["gdtype"]],
                "flops": n * D + case["V"] * D}
    p = D * BYTES[case["pdtype"]]
    if op == "norm":
        return {"bytes": 2 * n * D * e + 8 * n + 2 * p, "flops": 8 * n * D}
    return {"bytes": 3 * n * D * e + 8 * n + 3 * p, "flops": 14 * n * D}
