"""Plain 64-bit forms of the root-mean-square norm, the gated product and the
clipping, and the tolerances of their tests.

Tolerances.  u = 2^-24 is the half step of fp32; an output of 16 bits is rounded
once more, by half a step of its type (half_step).  Sums of a row's squares and
products are chains of at most CHAIN additions (64 in a thread, then trees).

A product of K terms runs in instructions of 16 terms: one rounding of the
running sum for each instruction and at most 4 levels inside one, so it is off by
at most (n K / 16 + 16) u of the sum of its terms' magnitudes, n the instructions
for 16 terms (1, fp32 factors 6).  fp32 factors are whole in their three numbers;
the three products that are left out are at most 2^-8 2^-16, 2^-16 2^-8 and 2^-16
2^-16 of the first, with bits cut off (not rounded) twice that: below 2^-21.
"""
import math

import torch

from tests.train_util import CHAIN, DTYPES, U, act64, half_step, slope64  # noqa: F401


def rms64(h, gamma, eps):
    """y and rstd of the rows of h (fp64)."""
    h = h.double()
    rstd = 1 / torch.sqrt(h.square().mean(-1) + eps)
    y = h * rstd[..., None]
    return (y if gamma is None else y * gamma.double()), rstd


def rms_tol(y, dtype):
    return y.abs() * (CHAIN / 2 + 16) * U + half_step(y, dtype)


def rms_back64(h, dy, dh, gamma, rstd):
    """dx, dgamma and their tolerances; rstd as it is given to the call."""
    dtype = h.dtype
    c = h.shape[-1]
    h, dy, rs = h.double(), dy.double(), rstd.double()[..., None]
    hh = h * rs
    t = dy if gamma is None else dy * gamma.double()
    mean = (t * hh).sum(-1, keepdim=True) / c
    dx = rs * (t - hh * mean)
    mean_err = (CHAIN + 8) * U * (t * hh).abs().sum(-1, keepdim=True) / c
    tol = rs * (4 * U * t.abs() + hh.abs() * (mean_err + 8 * U * mean.abs()))
    if dh is not None:
        dx = dx + dh.double()
    tol = tol + 2 * U * dx.abs() + half_step(dx, dtype)
    terms = (dy * hh).reshape(-1, c)
    # 64 rows of a slot, up to 256 slots one after the other, then fp64
    return dx, tol, terms.sum(0), (64 + 256 + 8) * U * terms.abs().sum(0)


class Gated64:
    """h, and with dh the gradients, in fp64 with bounds on a call's errors."""

    def __init__(self, x, wg, wu, bg, bu, act):
        self.dtype, self.act = x.dtype, act
        self.n = 6 if x.dtype == torch.float32 else 1
        self.lost = 2.0 ** -21 if x.dtype == torch.float32 else 0.0
        self.x, self.wg, self.wu = x.double(), wg.double(), wu.double()
        zero = torch.zeros(wg.shape[0], dtype=torch.float64, device=x.device)
        self.bg, self.bu = (zero if b is None else b.double() for b in (bg, bu))
        self.g, self.g_err = self.project(self.wg, self.bg)
        self.u, self.u_err = self.project(self.wu, self.bu)
        self.a, self.slope = act64(self.g, act), slope64(self.g, act)
        # the activations' slopes are at most 1.13, their own formulas 16 u (1 + |g|)
        self.a_err = 1.13 * self.g_err + 16 * U * (1 + self.g.abs())
        self.h = self.a * self.u

    def rate(self, k):
        return (self.n * k / 16 + 16) * U + self.lost

    def project(self, w, b):
        v = self.x @ w.t() + b
        return v, self.rate(w.shape[1]) * (self.x.abs() @ w.t().abs()) + 2 * U * v.abs()

    def h_tol(self):
        return self.u.abs() * self.a_err + self.a.abs() * self.u_err + 4 * U * self.h.abs() + half_step(self.h, self.dtype)

    def backward(self, dh):
        """{name: (value, tolerance)}"""
        dh = dh.double()
        dg, du = dh * self.u * self.slope, dh * self.a
        # a slope changes by at most its argument's error and is off by 16 roundings
        s_err = 1.0 * self.g_err + 16 * U * (1 + self.g.abs())
        dg_err = dh.abs() * (self.slope.abs() * self.u_err + self.u.abs() * s_err) + 4 * U * dg.abs()
        du_err = dh.abs() * self.a_err + 4 * U * du.abs()
        # ... and both are rounded to the type before the products
        dg_all, du_all = dg_err + half_step(dg, self.dtype), du_err + half_step(du, self.dtype)
        f, m = self.wg.shape[0], dh.shape[0]
        out = {}
        mag = dg.abs() @ self.wg.abs() + du.abs() @ self.wu.abs()
        dx = dg @ self.wg + du @ self.wu
        out["dx"] = dx, (dg_all @ self.wg.abs() + du_all @ self.wu.abs() + (self.rate(2 * f) + 64 * U) * mag +
                         half_step(dx, self.dtype) + U * dx.abs())
        for name, v, e in (("dw_gate", dg, dg_all), ("dw_up", du, du_all)):
            w = v.t() @ self.x
            out[name] = w, (e.t() @ self.x.abs() + (self.rate(m) + 64 * U) * (v.abs().t() @ self.x.abs()) +
                            half_step(w, self.dtype) + U * w.abs())
        for name, v, e in (("db_gate", dg, dg_err), ("db_up", du, du_err)):
            out[name] = v.sum(0), (e + 32 * U * v.abs()).sum(0)
        return out


def check(name, got, ref, tol):
    """Whether every element of got is within tol of ref (a NaN is not)."""
    assert got.shape == ref.shape, (name, tuple(got.shape), tuple(ref.shape))
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    if bool(bad.any()):
        i = int((err / tol).nan_to_num(nan=math.inf).argmax())
        raise AssertionError("%s: %d of %d outside; worst at %d: %g against %g, tolerance %g" % (
            name, int(bad.sum()), bad.numel(), i, float(got.flatten()[i]), float(ref.flatten()[i]),
            float(tol.expand_as(ref).flatten()[i])))
