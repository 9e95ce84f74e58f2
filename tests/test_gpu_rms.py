"""Root-mean-square norm on the GPU against its formulas in fp64."""
import pytest
import torch

import level_haar_wavelet_amd as wt
from level_haar_wavelet_amd.module import RMSNorm
from tests.block_util import DTYPES, check, rms64, rms_back64, rms_tol, U

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(rows, c, dtype, seed, offset=0):
    """x, residual, dy, dh (rows, c), each `offset` elements behind an aligned address, and gamma."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for i in range(4):
        v = torch.randn(rows, c, generator=g) * (1 + (i == 1) * torch.randn(1, c, generator=g).abs())
        t = torch.empty(rows * c + offset, dtype=DTYPES[dtype], device="cuda")[offset:].view(rows, c)
        t.copy_(v)
        out.append(t)
    return out + [(1 + 0.2 * torch.randn(c, generator=g)).cuda()]


# rows; lengths that a few lanes hold, a wave, a workgroup with 1, 2, 4 and 8
# accesses, and longer ones; lengths that no access divides
SHAPES = [(1, 1), (3, 7), (5, 8), (300, 96), (257, 128), (1000, 33), (65, 1024), (9, 2047), (4, 4096), (7, 5003),
          (2, 8192), (3, 16384), (2, 16391), (1, 40000), (4099, 16)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,c", SHAPES)
@pytest.mark.parametrize("offset", [0, 1])
def test_both_directions(rows, c, dtype, offset):
    x, r, dy, dh, gamma = make(rows, c, dtype, rows + c, offset)
    for res, ga in ((r, gamma), (None, None)):
        y, h, rstd = wt.wtconv_rms_norm_forward(x, res, ga, eps=EPS)
        want = x if res is None else (x.float() + res.float()).to(x.dtype)
        assert torch.equal(h, want) and (res is not None or h is x)
        ref, rs = rms64(want, ga, EPS)
        check("y", y, ref, rms_tol(ref, x.dtype))
        check("rstd", rstd, rs, rs * 80 * U)
        d2 = dh if res is not None else None
        dx, dgamma = wt.wtconv_rms_norm_backward(h, dy, rstd, ga, dh=d2)
        ref, tol, gref, gtol = rms_back64(h, dy, d2, ga, rstd)
        check("dx", dx, ref, tol)
        check("dgamma", dgamma, gref, gtol)


@pytest.mark.parametrize("rows,c,dtype", [(200000, 16, "bf16"), (70000, 96, "f32"), (300000, 9, "f16")])
def test_many_rows(rows, c, dtype):
    x, r, dy, dh, gamma = make(rows, c, dtype, 3)
    y, h, rstd = wt.wtconv_rms_norm_forward(x, r, gamma, eps=EPS)
    ref, _ = rms64(h, gamma, EPS)
    check("y", y, ref, rms_tol(ref, x.dtype))
    dx, dgamma = wt.wtconv_rms_norm_backward(h, dy, rstd, gamma, dh=dh)
    ref, tol, gref, gtol = rms_back64(h, dy, dh, gamma, rstd)
    check("dx", dx, ref, tol)
    check("dgamma", dgamma, gref, gtol)
    again = wt.wtconv_rms_norm_backward(h, dy, rstd, gamma, dh=dh)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dgamma)


@pytest.mark.parametrize("rows,c", [(2200000, 1000), (2200000, 1001), (70000, 33000)])
def test_beyond_2_31_elements(rows, c):
    """Rows repeat, and so do their outputs wherever they lie."""
    few = 40  # whole periods of a row's start
    x = torch.randn(few, c, device="cuda").bfloat16().repeat(rows // few, 1)
    assert x.numel() > 2 ** 31
    y, h, rstd = wt.wtconv_rms_norm_forward(x, x)
    dx, dgamma = wt.wtconv_rms_norm_backward(h, x, rstd)
    del h
    small, hs, rs = wt.wtconv_rms_norm_forward(x[:few], x[:few])
    ds, gs = wt.wtconv_rms_norm_backward(hs, x[:few], rs)
    assert bool((y.view(-1, few, c) == small).all()) and bool((rstd.view(-1, few) == rs).all())
    assert bool((dx.view(-1, few, c) == ds).all())
    assert float((dgamma.double() - gs.double() * (rows // few)).norm() / dgamma.double().norm()) < 1e-5


@pytest.mark.parametrize("c", [100, 103, 20000])
def test_in_place(c):
    x, r, dy, dh, gamma = make(37, c, "bf16", 5)
    y, h, rstd = wt.wtconv_rms_norm_forward(x, r, gamma)
    into = r.clone()
    y2, h2, _ = wt.wtconv_rms_norm_forward(x, into, gamma, h=into)
    assert h2 is into and torch.equal(into, h) and torch.equal(y2, y)
    dx, dgamma = wt.wtconv_rms_norm_backward(h, dy, rstd, gamma, dh=dh)
    into = dh.clone()
    dx2, dgamma2 = wt.wtconv_rms_norm_backward(h, dy, rstd, gamma, dh=into, dx=into)
    assert dx2 is into and torch.equal(dx2, dx) and torch.equal(dgamma2, dgamma)


def test_values():
    """A bad row stays in its row; zeros, infinities and squares out of range."""
    x = torch.randn(6, 64, device="cuda")
    good = wt.wtconv_rms_norm_forward(x)[0]
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    x[3] = 0.0
    x[4] = 1e30
    y, _, rstd = wt.wtconv_rms_norm_forward(x)
    assert torch.equal(y[0], good[0]) and torch.equal(y[5], good[5])
    assert bool(y[1].isnan().all()) and bool(y[2, 7].isnan()) and bool((y[2, :7] == 0).all())
    assert bool((y[3] == 0).all()) and float(rstd[3]) == pytest.approx(1e3, rel=1e-6)
    assert bool((y[4] == 0).all()) and float(rstd[4]) == 0
    dx, _ = wt.wtconv_rms_norm_backward(x, torch.ones_like(x), rstd)
    assert bool(dx[0].isfinite().all()) and bool(dx[5].isfinite().all()) and bool(dx[1].isnan().all())


def test_module_gradients():
    """Both outputs' gradients through the module, against fp64 autograd of the formula and against differences."""
    torch.manual_seed(0)
    norm = RMSNorm(48, device="cuda")
    with torch.no_grad():
        norm.gamma.add_(0.3 * torch.randn_like(norm.gamma))
    x = torch.randn(3, 5, 48, device="cuda", requires_grad=True)
    r = torch.randn(3, 5, 48, device="cuda", requires_grad=True)
    a, b = torch.randn(3, 5, 48, device="cuda"), torch.randn(3, 5, 48, device="cuda")

    def loss64(xx, rr, ga):
        h = xx + rr
        y = ga * h / torch.sqrt(h.square().mean(-1, keepdim=True) + norm.eps)
        return (y * a.double()).sum() + (h * b.double()).sum()

    y, h = norm(x, r)
    ((y * a).sum() + (h * b).sum()).backward()
    v = [t.detach().double().requires_grad_() for t in (x, r, norm.gamma)]
    loss64(*v).backward()
    for name, got, ref in zip(("x", "residual", "gamma"), (x.grad, r.grad, norm.gamma.grad), v):
        assert float((got - ref.grad).norm() / ref.grad.norm()) < 1e-6, name
    d = [torch.randn_like(t) for t in v]
    with torch.no_grad():
        step = 1e-5
        diff = (loss64(*(t + step * q for t, q in zip(v, d))) - loss64(*(t - step * q for t, q in zip(v, d)))) / (2 * step)
        own = sum((got.double() * q).sum() for got, q in zip((x.grad, r.grad, norm.gamma.grad), d))
    assert float(own) == pytest.approx(float(diff), rel=1e-5, abs=1e-4)
    # y alone, h alone, no residual
    for use in ("y", "h", "plain"):
        x.grad = None
        out = norm(x) if use == "plain" else norm(x, r)["yh".index(use)]
        (out * a).sum().backward()
        v = [t.detach().double().requires_grad_() for t in (x, r)]
        h = v[0] if use == "plain" else v[0] + v[1]
        o = h if use == "h" else norm.gamma.detach().double() * h / torch.sqrt(h.square().mean(-1, keepdim=True) + norm.eps)
        (o * a.double()).sum().backward()
        assert float((x.grad - v[0].grad).norm() / v[0].grad.norm()) < 1e-6, use


def test_strided_inputs_and_streams():
    norm = RMSNorm(24, device="cuda")
    x = torch.randn(2, 24, 6, 6, device="cuda").permute(0, 2, 3, 1)
    assert torch.equal(norm(x), norm(x.contiguous()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, _, _ = wt.wtconv_rms_norm_forward(x.contiguous(), gamma=norm.gamma.detach(), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, norm(x).detach())
