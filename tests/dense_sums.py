"""What the sums of a dense layer's weight gradient may lose, and inputs that show it.

The products are exact.  A step of the tensor cores adds 16 of them to a sum in float32 and
cuts the result off, so it loses less than a unit of the sum's last place, 2 u of it with
u = 2^-24; a chain of J steps (CHAIN / 16; CHAIN16 / 16 where the result has 16 bits) ends, and
from there on sums are rounded to nearest, u each.

`graded`: positive dy and x of many exponents, independent and alike over the rows.  A chain's
sum grows evenly; its values after the steps add up to (J + 1) / 2 times the last, give or take
0.3 J times the spread of one summand, 1.4 of its mean, over the root of 16 J of them: 0.05 J is
over 5 such deviations for a full chain of 128 steps, and a shorter one loses less.  So a chain
loses at most 0.55 J 2 u of its sum.

`coarse`: dy's upper part 1 or 1.5 and x 1 or 2, so that sums of hi x are multiples of 1/2
below 2^23 and no addition of them is cut off or rounded; all that is lost is lost by the rests,
which are below 2^-7 of it: two additions a step at most, each 2 u of the rests' sum so far,
2 J 2 u of their sum R in a chain."""
import numpy as np

CHAIN, CHAIN16 = 2048, 16384
U32 = 2.0 ** -24
JOINS = 48     # additions that join chains and ranges: 32 slices of up to 16 of them


def graded(n, N, D, generator, device, dtype):
    """dy = 2^(-6 .. 0), x = 2^(-3 .. 0)."""
    import torch
    dy = (-6 * torch.rand(n, N, generator=generator, device=device)).exp2().to(dtype)
    return dy, (-3 * torch.rand(n, D, generator=generator, device=device)).exp2()


def coarse(n, N, D, generator, device, dtype):
    """(dy, its upper part, x); dy has 17 or more bits in float32, 11 in float16."""
    import torch
    r = lambda *s: torch.rand(*s, generator=generator, device=device)  # noqa: E731
    hi = 1 + 0.5 * (r(n, N) < 0.5)
    dy = (hi + 2.0 ** -7 * (0.05 + 0.9 * r(n, N))).to(dtype)
    return dy, hi, 1.0 + (r(n, D) < 0.5)


def graded_limit(want, sixteen=False, joins=JOINS):
    """Of sums `want` of graded inputs, without the rounding to 16 bits."""
    steps = (CHAIN16 if sixteen else CHAIN) // 16
    return (0.55 * steps * 2 + joins + 3) * U32 * want


def coarse_limit(want, rests, rows, joins=JOINS):
    """Of sums `want` of coarse inputs whose rests add up to `rests`, chains of `rows` at most."""
    steps = -(-min(rows, CHAIN) // 16)
    return 2 * steps * 2 * U32 * rests + (joins + 3) * U32 * want


# ---- the sums as they are formed, in float64

def cut(v):
    """v towards zero to float32's 24 bits."""
    m, e = np.frexp(v)
    return np.ldexp(np.trunc(np.ldexp(m, 24)), e - 24)


def parts_of(dy):
    """float32 dy as three values of 8 bits each that add up to it."""
    out, rest = [], dy.astype(np.float32)
    for _ in range(3):
        hi = (rest.view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)
        out.append(hi.astype(np.float64))
        rest = rest - hi
    return out


def chained(dy, x, chain=CHAIN, parts=3, one_set=False):
    """dW = dy^T x of one range of rows, its chains added up in float32."""
    n = len(dy)
    p = parts_of(dy)[:parts]
    total = np.zeros((dy.shape[1], x.shape[1]), np.float32)
    for c in range(0, n, chain):
        sums = [np.zeros(total.shape) for _ in range(1 if one_set else 2)]
        for r in range(c, min(c + chain, n), 16):
            s = slice(r, min(r + 16, c + chain, n))
            for k, q in enumerate(p):
                a = 0 if one_set or k == 0 else 1
                sums[a] = cut(sums[a] + q[s].T @ x[s])
        for s in sums[1:]:
            sums[0] = (sums[0] + s).astype(np.float32).astype(np.float64)
        total = total + sums[0].astype(np.float32)
    return total.astype(np.float64)
