"""Shared by the GPU tests of the operators for activations in 8 bits: rows
with what can go wrong in them, and Rows8 buffers whose surroundings are watched."""
import numpy as np

FORMATS = ("int8", "e4m3")


def torch_format(fmt):
    import torch
    return {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[fmt]


def activations(r, n, D, t):
    """Rows of very different sizes; zeros, single values, borders of a scale."""
    big = 4.0 if t == "f16" else 30.0
    x = r.normal(size=(n, D)) * np.exp(r.uniform(-big, big / 2, (n, 1)))
    if n > 3:
        x[1] = 0.0
        x[2] = 0.0
        x[2, r.integers(D)] = -3.0
        x[3] = 0.25 * r.integers(-508, 508, D)          # ties, in both formats
        x[3, 0] = 127.0
    if n > 5:
        x[4] = 448.0 * r.choice([-1.0, 1.0], D)         # a scale's border
        x[5] = np.where(r.random(D) < 0.9, 0.0, r.normal(size=D))
    if n > 7 and t != "f16":
        x[6] = 1e-36 * r.normal(size=D)                 # below the least scale's reach
        x[7] = 2.0e38 * r.choice([-1.0, 1.0], D)
    return x


class Guarded:
    """A Rows8 of the binding whose buffers are pieces of larger ones."""

    def __init__(self, ss, n, D, fmt, extra_q=0, extra_s=0):
        import torch
        self.n, self.D, self.fmt = n, D, fmt
        self.held, self.G = (D + 7) // 8 * 8, (D + 31) // 32
        self.qs, self.ss_ = self.held + extra_q, self.G + extra_s
        self.qbuf = torch.full((16 + n * self.qs + 16,), 0xA5, dtype=torch.uint8, device="cuda")
        self.sbuf = torch.full((3 + n * self.ss_ + 5,), 0x5A, dtype=torch.uint8, device="cuda")
        r = ss.Rows8(n, D, torch_format(fmt))
        r._buf = self.qbuf[16:16 + n * self.qs].view(n, self.qs)
        r._q = r._buf.view(torch_format(fmt))[:, :D]
        r._scales = self.sbuf[3:3 + n * self.ss_].view(n, self.ss_)[:, :self.G]
        r._c.q, r._c.q_stride = self.qbuf.data_ptr() + 16, self.qs
        r._c.scales, r._c.scale_stride = self.sbuf.data_ptr() + 3, self.ss_
        self.rows = r

    def check_untouched(self):
        """Nothing written outside the rows; the bytes past D are zeros."""
        n, D = self.n, self.D
        q, s = self.qbuf.cpu().numpy(), self.sbuf.cpu().numpy()
        assert (q[:16] == 0xA5).all() and (q[16 + n * self.qs:] == 0xA5).all()
        assert (s[:3] == 0x5A).all() and (s[3 + n * self.ss_:] == 0x5A).all()
        q = q[16:16 + n * self.qs].reshape(n, self.qs)
        s = s[3:3 + n * self.ss_].reshape(n, self.ss_)
        assert (q[:, D:self.held] == 0).all() and (q[:, self.held:] == 0xA5).all()
        assert (s[:, self.G:] == 0x5A).all()
