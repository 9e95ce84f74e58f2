"""The gated product's digits and ranges on the GPU: fp32 factors in full, fp16
gradients that are small or large."""
import pytest
import torch

import level_haar_wavelet_amd as wt
from tests.block_util import U, Gated64, check
from tests.test_gpu_gated import NAMES, make

pytestmark = pytest.mark.gpu


def spread(*shape, seed=0):
    """fp32 values with random last bits, of both signs and several powers of two."""
    g = torch.Generator().manual_seed(seed)
    v = (1 + torch.rand(shape, generator=g)) * 2.0 ** torch.randint(-3, 4, shape, generator=g)
    return (v * (1 - 2 * torch.randint(0, 2, shape, generator=g))).cuda()


def single(rows, cols, values):
    """Rows with one value each, the r-th in column r modulo cols."""
    t = torch.zeros(rows, cols, device="cuda")
    r = torch.arange(rows, device="cuda")
    t[r, r % cols] = values
    return t


# Sums of one product each, so that nothing but that product is off.  Of its factors' nine
# partial products three are left out: with each number the nearest to what is left
# before it, they are at most 2 2^-8 2^-17 + 2^-34 of the whole.  The sums of the five
# smaller ones are below 2^-7 of it, five roundings of 2 U each; the last sum's rounding
# is at most 2 U, to whichever side it goes.
ONE = (1 + 2.0 ** -9 + 10 * 2.0 ** -7 + 2) * U


# few rows, short rows (32 and 192 channels), longer ones, rows that no access divides
@pytest.mark.parametrize("m,c,f", [(40, 32, 64), (200, 32, 256), (300, 192, 304), (200, 200, 204), (130, 33, 135)])
def test_fp32_products_keep_their_digits(m, c, f):
    wg, wu = spread(f, c, seed=1), torch.zeros(f, c, device="cuda")
    up = torch.ones(f, device="cuda")  # u = 1
    x = single(m, c, spread(m, seed=2))
    x[3, 3] = 0.999999 * torch.finfo(torch.float32).max  # beyond the largest bf16 number
    wg_small = wg / 16
    h = wt.wtconv_gated_forward(x, wg_small, wu, None, up, act="none")
    col = torch.arange(m, device="cuda") % c
    want = x.double().sum(1, keepdim=True) * wg_small.double()[:, col].t()
    check("h", h, want, ONE * want.abs())

    x, v = spread(m, c, seed=3), spread(m, seed=4)
    dh = single(m, f, v)  # f >= m: a column has one row
    dx, dw, _, _, _ = wt.wtconv_gated_backward(x, dh, wg, wu, None, up, act="none")
    want = v.double()[:, None] * wg.double()[:m]
    check("dx", dx, want, ONE * want.abs())
    want = v.double()[:, None] * x.double()
    check("dw_gate", dw[:m], want, ONE * want.abs())
    assert not bool(dw[m:].any())


# dg and du below 2^-14 have steps of 2^-24 (half_step counts them), below 2^-25 they are zero;
# the biases' gradients sum them before that
@pytest.mark.parametrize("scale", [1e-4, 2e-6, 1e3])
@pytest.mark.parametrize("m,c,f", [(5, 64, 40), (150, 96, 72), (140, 33, 65), (300, 264, 130)])
def test_fp16_gradients_of_any_size(m, c, f, scale):
    x, wg, wu, bg, bu, dh = make(m, c, f, "f16", seed=m)
    dh = (dh.float() * scale).half()
    want = Gated64(x, wg, wu, bg, bu, "silu").backward(dh)
    # (the weights' gradients in float32: at the largest size some of them pass 65504)
    for name, got in zip(NAMES, wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu, dw_dtype=torch.float32)):
        check(name, got, *want[name])
    # ... and beyond fp16's range in the weights' gradients alone
    if scale > 1:
        x = x.abs()
        dh = (dh.float().abs() * 8).clamp(max=3e4).half()
        wu.zero_()
        want = Gated64(x, wg, wu, None, torch.ones_like(bu), "none").backward(dh)
        out = wt.wtconv_gated_backward(x, dh, wg, wu, None, torch.ones_like(bu), act="none", dw_dtype=torch.float32)
        check("dw_gate", out[1], *want["dw_gate"])
        own = wt.wtconv_gated_backward(x, dh, wg, wu, None, torch.ones_like(bu), act="none")
        assert torch.equal(own[1], out[1].half())
        if m > 100:
            assert float(out[1].min()) > 65504 and bool(own[1].isinf().all())


def test_fp16_gradients_beyond_their_range():
    """dg beyond 65504 is infinite, and with it the row of dx that it is in; no other row."""
    x, wg, wu, bg, bu, dh = make(200, 64, 48, "f16", seed=5)
    good = wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu)
    dh[7] = 6e4
    x[7] *= 8
    dx, _, _, dbg, _ = wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu)
    rows = [i for i in range(200) if i != 7]
    assert torch.equal(dx[rows], good[0][rows])
    want = Gated64(x, wg, wu, bg, bu, "silu").backward(dh)["db_gate"]
    check("db_gate", dbg, *want)  # sums of fp32
    assert not bool(dx[7].isfinite().any())
