"""Plain 64-bit forms of the group norm and the Muon step, and the tolerances of
their tests.

Tolerances.  u = 2^-24 is the half step of fp32.  A kernel's sum of K values is a
chain of at most CHAIN additions (a thread's own values, then trees over lanes,
waves and partial sums), so it is off by at most CHAIN u times the sum of the
magnitudes.  Every elementwise formula takes fewer than 16 roundings.  An output
of 16 bits is rounded once more, by half a step (eps / 2) of its type.
"""
import math

import torch

U = 2.0 ** -24
CHAIN = 128
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def act64(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    return z


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def half_step(ref, dtype):
    """Half a step of a 16-bit output at the reference's values (0 for fp32,
    whose rounding is counted with the others)."""
    if dtype == torch.float32:
        return 0.0
    f = torch.finfo(dtype)
    return ref.abs() * f.eps / 2 + f.smallest_normal * f.eps / 2


class Norm64:
    """The norm of x (N, C, H, W, any type) in fp64 with its intermediates."""

    def __init__(self, x, groups, gamma, beta, eps, act):
        n, c, h, w = x.shape
        self.shape, self.groups, self.act = (n, c, h, w), groups, act
        self.x = x.double().reshape(n, groups, -1)
        self.mean = self.x.mean(2)
        self.var = (self.x - self.mean[..., None]).square().mean(2)
        self.rstd = 1 / torch.sqrt(self.var + eps)
        self.ga = (torch.ones(c, dtype=torch.float64) if gamma is None else gamma.double()).view(1, c, 1, 1)
        self.be = (torch.zeros(c, dtype=torch.float64) if beta is None else beta.double()).view(1, c, 1, 1)
        self.xh = ((self.x - self.mean[..., None]) * self.rstd[..., None]).view(n, c, h, w)
        self.z = self.ga * self.xh + self.be
        self.y = act64(self.z, act)

    def per_element(self, t):
        """(N, groups) values as (N, C, 1, 1)."""
        n, c = self.shape[:2]
        return t.repeat_interleave(c // self.groups, 1).view(n, c, 1, 1)

    def y_tol(self, dtype):
        # mean: CHAIN u E|x|; rstd: (CHAIN + 8) / 2 u relative; the activations'
        # slopes are at most 1.13 and their own formulas 16 u (1 + |z|)
        ex = self.per_element(self.x.abs().mean(2) * self.rstd)
        z_err = U * (self.ga.abs() * (CHAIN * ex + (CHAIN / 2 + 8) * self.xh.abs()) + 4 * self.z.abs())
        return 1.13 * z_err + 16 * U * (1 + self.z.abs()) + half_step(self.y, dtype)

    def backward(self, dy):
        n, c, h, w = self.shape
        dy = dy.double()
        self.dz = dy * slope64(self.z, self.act)
        self.dbeta = self.dz.sum((0, 2, 3))
        self.dgamma = (self.dz * self.xh).sum((0, 2, 3))
        t = self.ga * self.dz
        g = lambda v: self.per_element(v.reshape(n, self.groups, -1).mean(2))
        self.dx = self.per_element(self.rstd) * (t - g(t) - self.xh * g(t * self.xh))
        # an element's dz is off by 16 roundings of dy slope and by the slope's
        # own change (at most 1) with z's error, (|gamma| 8 |xh| + 4 |z|) u
        e = dy.abs() * U * (16 * (1 + self.z.abs()) + 8 * self.ga.abs() * self.xh.abs() + 4 * self.z.abs())
        te = self.ga.abs() * e
        self.dbeta_tol = (e + CHAIN * U * self.dz.abs()).sum((0, 2, 3))
        xt = (self.dz * self.xh).abs()
        self.dgamma_tol = (e * self.xh.abs() + (CHAIN + 8) * U * xt).sum((0, 2, 3))
        a, b = g(te + CHAIN * U * t.abs()), g(te * self.xh.abs() + (CHAIN + 8) * U * (t * self.xh).abs())
        mag = t.abs() + g(t).abs() + (self.xh * g(t * self.xh)).abs()
        self.dx_err = self.per_element(self.rstd) * (te + a + self.xh.abs() * b + 8 * U * mag)
        return self.dx, self.dgamma, self.dbeta

    def dx_tol(self, dtype):
        return self.dx_err + half_step(self.dx, dtype)


COEF = (3.4445, -4.7750, 2.0315)


def ortho64(g, steps=5, eps=1e-7):
    """The iteration on a (..., rows, cols) stack in fp64 (coefficients as the
    fp32 values the kernels hold)."""
    a, b, c = (float(torch.tensor(v, dtype=torch.float32)) for v in COEF)
    x = g.double()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    x = x / (torch.linalg.matrix_norm(x, keepdim=True) + eps)
    for _ in range(steps):
        p = x @ x.mT
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.mT if tall else x


def ortho_tol(ref, steps, dtype):
    """Bound on the Frobenius norm of a result's error, per matrix.  A product
    with factors of 22 bits is off by 2^-22 of its norm; a step magnifies an
    error by at most a = 3.4445, so one made at X_0 (of norm 1) arrives as
    2^-22 a^steps, and the three products of every step add in squares.  An
    output's own rounding comes on top."""
    norm = torch.linalg.matrix_norm(ref)
    own = U if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    return 2.0 ** -22 * COEF[0] ** steps * math.sqrt(3 * steps) + own * norm
