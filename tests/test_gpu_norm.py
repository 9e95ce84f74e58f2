"""Group norm with activation on the GPU against its formulas in fp64."""
import pytest
import torch

import level_haar_wavelet_amd as wt
from tests.train_util import DTYPES, Norm64

pytestmark = pytest.mark.gpu

LAYOUTS = [(False, False), (True, True), (False, True), (True, False)]
ACTS = ["none", "relu", "silu", "gelu"]

# n, c, h, w, groups: one value a group; groups of one channel, of all; channel
# counts that 16-byte vectors do and do not divide; planes shorter than a wave,
# odd ones, ones that several workgroups share; many images
SHAPES = [
    (1, 1, 1, 1, 1), (2, 1, 9, 10, 1), (2, 6, 1, 1, 3), (3, 5, 1, 7, 5), (2, 8, 16, 16, 4), (2, 8, 4, 4, 1), (1, 24, 3, 5, 24),
    (2, 33, 9, 11, 3), (3, 100, 37, 23, 20), (2, 96, 28, 28, 32), (1, 192, 14, 14, 32), (2, 64, 56, 56, 8),
    (1, 12, 131, 67, 4), (1, 16, 200, 200, 2), (70, 4, 6, 10, 2), (1, 256, 31, 33, 16), (2, 1030, 3, 3, 5),
    (1, 8, 256, 256, 1), (1, 520, 64, 64, 65),
    # accesses of 8 bytes: four (two) elements divide the channels, the pixels or both
    (2, 12, 14, 14, 3), (2, 36, 6, 7, 9), (1, 20, 66, 66, 5), (2, 10, 50, 62, 2), (1, 100, 64, 66, 4),
]


def layout(t, last):
    return t.contiguous(memory_format=torch.channels_last) if last else t.contiguous()


def inputs(shape, dtype, seed, offset=0.0):
    n, c, h, w, groups = shape
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, c, h, w, generator=g) * (0.5 + torch.rand(1, c, 1, 1, generator=g)) \
        + torch.randn(1, c, 1, 1, generator=g) + offset
    dy = torch.randn(n, c, h, w, generator=g)
    gamma = 1 + 0.3 * torch.randn(c, generator=g)
    beta = 0.3 * torch.randn(c, generator=g)
    return x.to(DTYPES[dtype]), dy.to(DTYPES[dtype]), gamma, beta


def within(got, ref, tol, what):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), what + ": not finite"
    over = (got - ref).abs() / torch.as_tensor(tol).clamp(min=1e-300)
    assert over.max() <= 1, "%s: %.3g times its tolerance" % (what, over.max())


def check(shape, dtype, act, lx, ly, seed, offset=0.0, affine=True, eps=1e-5):
    n, c, h, w, groups = shape
    x, dy, gamma, beta = inputs(shape, dtype, seed, offset)
    if not affine:
        gamma = beta = None
    ref = Norm64(x, groups, gamma, beta, eps, act)
    cu = lambda t: None if t is None else t.cuda()
    xd, dyd = layout(x.cuda(), lx), layout(dy.cuda(), ly)
    y, mean, rstd = wt.wtconv_group_norm_forward(xd, groups, cu(gamma), cu(beta), eps=eps, act=act, channels_last=ly)
    what = "%s %s %s %s->%s" % (shape, dtype, act, lx, ly)
    assert y.is_contiguous(memory_format=torch.channels_last if ly else torch.contiguous_format)
    within(y, ref.y, ref.y_tol(x.dtype), what + " y")
    ex = ref.x.abs().mean(2)
    within(mean, ref.mean, 2.0 ** -24 * 128 * ex + 1e-30, what + " mean")
    # rstd: half of var's relative error, which is CHAIN u and twice the mean's
    # (squared differences from a rounded mean add its error squared)
    within(rstd, ref.rstd, ref.rstd * 2.0 ** -24 * (64 + 8) + ref.rstd ** 3 * (2.0 ** -24 * 128 * ex) ** 2,
           what + " rstd")
    # the backward call takes the reference's statistics, rounded to fp32
    ref.backward(dy)
    m32, r32 = ref.mean.float().cuda(), ref.rstd.float().cuda()
    dx, dg, db = wt.wtconv_group_norm_backward(xd, dyd, groups, m32, r32, cu(gamma), cu(beta), act=act)
    # the rounded mean moves xh by u |mean| rstd, the rounded rstd by u |xh|
    drift = ref.per_element(ref.mean.abs() * ref.rstd) * 2.0 ** -24
    slack = (1 + ref.ga.abs()) ** 2 * (dy.double().abs() + ref.dz.abs()) * (drift + 2.0 ** -24 * ref.xh.abs())
    g = lambda v: ref.per_element(v.reshape(n, groups, -1).mean(2))
    rs = ref.per_element(ref.rstd)
    dx_slack = rs * (slack + g(slack) + ref.xh.abs() * g(slack * (1 + ref.xh.abs())) +
                     drift * g((ref.ga * ref.dz * ref.xh).abs()))
    within(dx, ref.dx, ref.dx_tol(x.dtype) + dx_slack, what + " dx")
    within(dg, ref.dgamma, ref.dgamma_tol + (slack * (1 + ref.xh.abs())).sum((0, 2, 3)), what + " dgamma")
    within(db, ref.dbeta, ref.dbeta_tol + slack.sum((0, 2, 3)), what + " dbeta")


@pytest.mark.parametrize("layouts", LAYOUTS, ids=lambda l: "%s_%s" % tuple("last" if v else "planes" for v in l))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_the_formulas(shape, layouts):
    i = SHAPES.index(shape) + LAYOUTS.index(layouts)
    for k, dtype in enumerate(DTYPES):
        act = ACTS[(i + k) % 4]
        print(shape, layouts, dtype, act, flush=True)
        check(shape, dtype, act, *layouts, seed=i * 10 + k)


@pytest.mark.parametrize("layouts", LAYOUTS, ids=lambda l: "%s_%s" % tuple("last" if v else "planes" for v in l))
@pytest.mark.parametrize("shape", [(2, 3, 8, 8, 1), (2, 6, 8, 8, 3), (2, 4, 8, 8, 2), (3, 2, 16, 12, 1), (2, 7, 24, 16, 7),
                                   (1, 5, 64, 64, 1)], ids=lambda s: "x".join(map(str, s)))
def test_fewer_channels_than_an_access_has_elements(shape, layouts):
    # rows of pixels allow accesses of 8 or 16 bytes, rows of channels do not
    for k, dtype in enumerate(DTYPES):
        print(shape, layouts, dtype, flush=True)
        check(shape, dtype, ACTS[k + 1], *layouts, seed=500 + k)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_every_activation_in_every_type(act, dtype):
    check((2, 24, 19, 21, 6), dtype, act, True, True, seed=77)
    check((2, 24, 19, 21, 6), dtype, act, False, False, seed=78, affine=False)
    check((2, 40, 20, 20, 8), dtype, act, False, True, seed=79, eps=0.1)


@pytest.mark.parametrize("layouts", LAYOUTS, ids=str)
@pytest.mark.parametrize("shape,dtype", [((18, 64, 96, 96, 8), "f32"), ((29, 64, 97, 96, 16), "bf16")], ids=str)
def test_tensors_larger_than_the_caches(shape, dtype, layouts):
    check(shape, dtype, "gelu", *layouts, seed=11)


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("shape", [(2, 16, 40, 40, 4), (1, 8, 256, 256, 2)], ids=str)
def test_a_mean_far_from_zero_does_not_cancel(shape, last):
    # sum x^2 - K mean^2 in fp32 would lose every digit of the variance here
    check(shape, "f32", "silu", last, last, seed=5, offset=3000.0)


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("shape", [(2, 16, 40, 40, 4), (2, 16, 8, 8, 4), (1, 8, 256, 16, 2)], ids=str)
def test_a_mean_whose_square_overflows(shape, last):
    # the values' spread, 1e17, has a finite variance: K 1e34 is the largest sum
    n, c, h, w, groups = shape
    x = 1e20 + 1e17 * torch.randn(n, c, h, w, generator=torch.Generator().manual_seed(8), dtype=torch.float64)
    x = x.float()
    ref = Norm64(x, groups, None, None, 1e-5, "none")
    _, mean, rstd = wt.wtconv_group_norm_forward(layout(x.cuda(), last), groups)
    # as in check(); the mean's error there is 128 u 1e20 / 1e17 = 0.8 % of the spread, squared in rstd
    ex = ref.x.abs().mean(2)
    within(mean, ref.mean, 2.0 ** -24 * 128 * ex, "mean")
    within(rstd, ref.rstd, ref.rstd * 2.0 ** -24 * (64 + 8) + ref.rstd ** 3 * (2.0 ** -24 * 128 * ex) ** 2, "rstd")


def test_a_constant_group_gives_beta_and_finite_gradients():
    x = torch.full((2, 8, 6, 6), 3.0, device="cuda")
    beta = torch.randn(8, device="cuda")
    y, mean, rstd = wt.wtconv_group_norm_forward(x, 2, None, beta)
    assert torch.equal(y, beta.view(1, 8, 1, 1).expand_as(y))
    assert torch.equal(mean, torch.full_like(mean, 3.0))
    dx, dg, db = wt.wtconv_group_norm_backward(x, torch.randn_like(x), 2, mean, rstd, None, beta)
    assert torch.isfinite(dx).all() and torch.equal(dg, torch.zeros_like(dg))


@pytest.mark.parametrize("layouts", LAYOUTS, ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_value_stays_in_its_group(bad, layouts):
    lx, ly = layouts
    for act in ACTS:
        x, dy, gamma, beta = inputs((2, 24, 17, 18, 6), "f32", 3)
        clean, _, _ = wt.wtconv_group_norm_forward(layout(x.cuda(), lx), 6, gamma.cuda(), beta.cuda(), act=act,
                                                   channels_last=ly)
        x[1, 9, 4, 5] = bad
        xd = layout(x.cuda(), lx)
        y, mean, rstd = wt.wtconv_group_norm_forward(xd, 6, gamma.cuda(), beta.cuda(), act=act, channels_last=ly)
        dx, _, _ = wt.wtconv_group_norm_backward(xd, layout(dy.cuda(), ly), 6, mean, rstd, gamma.cuda(), beta.cuda(),
                                                 act=act)
        hit = torch.zeros(2, 24, 1, 1, dtype=torch.bool)
        hit[1, 8:12] = True
        hit = hit.expand_as(x).cuda()
        assert torch.isnan(y[hit]).all() and torch.isnan(dx[hit]).all(), act
        assert torch.equal(y[~hit], clean[~hit]) and torch.isfinite(dx[~hit]).all(), act


def test_large_negative_values_of_the_activations():
    # exp(-z) overflows: the limit is taken, not a NaN
    x = torch.tensor([-1.0, 1.0], device="cuda").repeat(8).view(1, 2, 2, 4)
    gamma = torch.full((2,), 300.0, device="cuda")
    for act in ("silu", "gelu"):
        y, mean, rstd = wt.wtconv_group_norm_forward(x, 1, gamma, None, act=act)
        ref = torch.where(x < 0, 0.0, 300.0 * rstd.item())
        assert torch.allclose(y, ref, atol=1e-4), act
        dx, dg, db = wt.wtconv_group_norm_backward(x, torch.ones_like(x), 1, mean, rstd, gamma, None, act=act)
        assert torch.isfinite(dx).all() and torch.isfinite(dg).all(), act


@pytest.mark.parametrize("layouts", LAYOUTS, ids=str)
def test_unaligned_buffers_and_what_lies_behind_them(layouts):
    """Views one element into a buffer; nothing outside the outputs changes."""
    lx, ly = layouts
    for shape in ((2, 16, 12, 12, 4), (1, 15, 7, 9, 5)):
        for dtype in DTYPES.values():
            n, c, h, w, groups = shape
            k = n * c * h * w

            def view(buf, last):
                v = buf[1:k + 1]
                return v.view(n, h, w, c).permute(0, 3, 1, 2) if last else v.view(n, c, h, w)

            g = torch.Generator(device="cuda").manual_seed(1)
            bufs = [torch.randn(k + 40, generator=g, device="cuda").to(dtype) for _ in range(4)]
            x, dy, y, dx = (view(b, l) for b, l in zip(bufs, (lx, ly, ly, lx)))
            yr, mean, rstd = wt.wtconv_group_norm_forward(layout(x.clone(), lx), groups, act="silu", channels_last=ly)
            dxr, dgr, dbr = wt.wtconv_group_norm_backward(layout(x.clone(), lx), layout(dy.clone(), ly), groups, mean,
                                                          rstd, act="silu")
            edge = [b[[0] + list(range(k + 1, k + 40))].clone() for b in bufs]
            wt.wtconv_group_norm_forward(x, groups, act="silu", y=y)
            _, dg, db = wt.wtconv_group_norm_backward(x, dy, groups, mean, rstd, act="silu", dx=dx)
            tol = 1e-5 if dtype == torch.float32 else 4 * torch.finfo(dtype).eps
            assert torch.allclose(y.float(), yr.float(), atol=tol, rtol=tol)
            assert torch.allclose(dx.float(), dxr.float(), atol=tol, rtol=tol)
            assert torch.allclose(dg, dgr, atol=1e-3, rtol=1e-4) and torch.allclose(db, dbr, atol=1e-3, rtol=1e-4)
            for b, e in zip(bufs, edge):
                assert torch.equal(b[[0] + list(range(k + 1, k + 40))], e)


def test_refusals_on_the_gpu():
    x = torch.randn(2, 8, 4, 4, device="cuda")
    with pytest.raises(ValueError):
        wt.wtconv_group_norm_forward(x, 2, act="tanh")
    with pytest.raises(TypeError):
        wt.wtconv_group_norm_forward(x[:, ::2], 2)
    with pytest.raises(TypeError):
        wt.wtconv_group_norm_forward(x.double(), 2)
    with pytest.raises(TypeError):
        wt.wtconv_group_norm_forward(x, 2, torch.ones(4, device="cuda"))
    with pytest.raises(TypeError):
        wt.wtconv_group_norm_forward(x, 2, torch.ones(8))
    with pytest.raises(TypeError):
        wt.wtconv_group_norm_forward(x, 2, y=torch.empty_like(x), channels_last=True)
    with pytest.raises(wt._native.WtconvError):
        wt.wtconv_group_norm_forward(x, 3)
    with pytest.raises(wt._native.WtconvError):
        wt.wtconv_group_norm_forward(x, 2, y=x)
    with pytest.raises(wt._native.WtconvError):
        wt.wtconv_group_norm_forward(x[:0], 2)
    y, mean, rstd = wt.wtconv_group_norm_forward(x, 2)
    with pytest.raises(TypeError):
        wt.wtconv_group_norm_backward(x, y[:1], 2, mean, rstd)
    with pytest.raises(TypeError):
        wt.wtconv_group_norm_backward(x, y.half(), 2, mean, rstd)
    with pytest.raises(TypeError):
        wt.wtconv_group_norm_backward(x, y, 2, mean[:1], rstd)
    with pytest.raises(TypeError):
        wt.wtconv_group_norm_backward(x, y, 2, mean, rstd, dx=layout(torch.empty_like(x), True))


def test_gradients_against_differences():
    """<dx, v> against the forward call's own difference along v (fp64 sums of
    fp32 outputs: an output is off by about 4 u |y| ~ 2^-22, so a difference
    over 2 h = 0.02 by 2^-22 sqrt(K) / 0.02; its own h^2 error is about 1e-4)."""
    from level_haar_wavelet_amd.module import GroupNormAct2d

    for act in ("silu", "gelu", "none"):
        torch.manual_seed(2)
        m = GroupNormAct2d(4, 16, act=act, channels_last=True, device="cuda")
        with torch.no_grad():
            m.gamma.add_(0.3 * torch.randn(16, device="cuda"))
            m.beta.add_(0.3 * torch.randn(16, device="cuda"))
        x = torch.randn(2, 16, 9, 11, device="cuda", requires_grad=True)
        w = torch.randn(2, 16, 9, 11, device="cuda")
        (m(x) * w).sum().backward()
        for t, grad in ((x, x.grad), (m.gamma, m.gamma.grad), (m.beta, m.beta.grad)):
            v = torch.randn_like(t)
            h, keep, out = 0.01, t.detach().clone(), []
            with torch.no_grad():
                for s in (h, -h):
                    t.copy_(keep + s * v)
                    out.append((m(x).double() * w.double()).sum().item())
                t.copy_(keep)
            diff, dot = (out[0] - out[1]) / (2 * h), (grad.double() * v.double()).sum().item()
            size = grad.double().norm().item() * v.double().norm().item()
            assert abs(diff - dot) <= 2e-3 * size ** 0.5 + 2e-3 * abs(dot) + 1e-3 * size / t.numel() ** 0.5, act


def test_module_layouts_and_frozen_parts():
    from level_haar_wavelet_amd.module import GroupNormAct2d

    x = torch.randn(2, 12, 10, 14, device="cuda", dtype=torch.bfloat16)
    for cl in (None, True, False):
        m = GroupNormAct2d(3, 12, act="gelu", channels_last=cl, device="cuda")
        for last in (False, True):
            xi = layout(x.clone(), last).requires_grad_()
            y = m(xi)
            assert y.is_contiguous(memory_format=torch.channels_last) == (last if cl is None else cl)
            y.sum().backward()  # dy is an expanded scalar: no layout of its own
            assert xi.grad.shape == x.shape and m.gamma.grad is not None
    strided = torch.randn(2, 24, 10, 14, device="cuda")[:, ::2].requires_grad_()
    m = GroupNormAct2d(3, 12, device="cuda")
    ref = torch.nn.functional.group_norm(strided, 3, eps=1e-5)
    assert torch.allclose(m(strided), ref, atol=1e-5)
    m.gamma.requires_grad_(False)
    m(strided.detach()).sum().backward()
    assert m.gamma.grad is None and m.beta.grad is not None


def test_same_bits_every_time_and_on_another_stream():
    x, dy, gamma, beta = (t.cuda() for t in inputs((8, 64, 56, 56, 8), "f16", 9))
    for last in (False, True):
        xl, dyl = layout(x, last), layout(dy, last)
        y0, mean, rstd = wt.wtconv_group_norm_forward(xl, 8, gamma, beta, act="gelu")
        b0 = wt.wtconv_group_norm_backward(xl, dyl, 8, mean, rstd, gamma, beta, act="gelu")
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(3):
            got = []
            for s in streams:  # two calls in flight, each with its own workspace
                s.wait_stream(torch.cuda.current_stream())
                f = wt.wtconv_group_norm_forward(xl, 8, gamma, beta, act="gelu", stream=s)
                got.append((f, wt.wtconv_group_norm_backward(xl, dyl, 8, f[1], f[2], gamma, beta, act="gelu",
                                                             stream=s)))
            torch.cuda.synchronize()
            for f, b in got:
                assert torch.equal(f[0], y0) and all(torch.equal(p, q) for p, q in zip(b, b0))


def test_a_call_on_another_stream_takes_no_block_of_the_current_one():
    # the allocator hands a freed block to the next request on the same stream,
    # whose work orders it; a call on another stream does not wait for that work
    x = torch.randn(4, 8, 64, 64, device="cuda")
    g = torch.randn(512, 600, device="cuda")
    w, m = torch.zeros_like(g), torch.zeros_like(g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    freed = []
    for t in (x, g):
        freed.append(torch.empty_like(t))
    freed = {t.untyped_storage().data_ptr() for t in freed}
    y, mean, rstd = wt.wtconv_group_norm_forward(x, 2, stream=s)
    s.synchronize()
    dx = wt.wtconv_group_norm_backward(x, x, 2, mean, rstd, stream=s)[0]
    o = wt.wtconv_orthogonalize(g, stream=s)
    wt.wtconv_muon_step(w, g, m, lr=0.1, stream=s)
    s.synchronize()
    assert not freed & {t.untyped_storage().data_ptr() for t in (y, dx, o)}
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, wt.wtconv_group_norm_forward(x, 2)[0]) and torch.equal(o, wt.wtconv_orthogonalize(g))


@pytest.mark.parametrize("shape", [(2, 24, 20, 18, 6), (4, 64, 28, 28, 8), (1, 16, 200, 200, 2)], ids=str)
@pytest.mark.parametrize("layouts", LAYOUTS, ids=str)
def test_captured_calls_replay_on_new_inputs(shape, layouts):
    lx, ly = layouts
    groups = shape[-1]
    x, dy, gamma, beta = (t.cuda() for t in inputs(shape, "f32", 4))
    x, dy = layout(x, lx), layout(dy, ly)

    def step():
        y, mean, rstd = wt.wtconv_group_norm_forward(x, groups, gamma, beta, act="silu", channels_last=ly)
        return (y, mean, rstd) + wt.wtconv_group_norm_backward(x, dy, groups, mean, rstd, gamma, beta, act="silu")

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(4):
        nx, ndy, _, _ = inputs(shape, "f32", 20 + r)
        x.copy_(nx)
        dy.copy_(ndy)
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_offsets_beyond_32_bits():
    """Five images of 2^29 values each: the last one's offsets pass 2^31.  The
    image alone is cut into other ranges: its statistics may differ by the
    rounding of their sums (CHAIN u E|x| = 128 2^-24 0.8 = 6e-6), its outputs
    by that and one fp16 step (2^-10 of the value), as two neighbouring
    roundings do."""
    x = torch.empty(5, 2, 1 << 14, 1 << 14, device="cuda", dtype=torch.float16)
    for i in range(5):
        x[i].normal_()
    y, mean, rstd = wt.wtconv_group_norm_forward(x, 2, act="relu")
    dx, dg, db = wt.wtconv_group_norm_backward(x, x, 2, mean, rstd, act="relu")
    torch.cuda.synchronize()
    y1, m1, r1 = wt.wtconv_group_norm_forward(x[4:].clone(), 2, act="relu")
    dx1, _, _ = wt.wtconv_group_norm_backward(x[4:].clone(), x[4:].clone(), 2, m1, r1, act="relu")
    assert torch.allclose(m1, mean[4:], atol=6e-6, rtol=0)
    for a, b in ((y1, y[4:]), (dx1, dx[4:])):
        assert ((a - b).abs() <= b.abs() * 2.0 ** -10 + 4e-5).all()
    v = x[4, 1].double()
    assert abs(v.mean().item() - m1[0, 1].item()) < 1e-5


def stats64(x, groups):
    """mean, biased variance and E|x| of every group in fp64, on the GPU image by image."""
    out = []
    for v in x:
        v = v.double().reshape(groups, -1)
        m = v.mean(1)
        out.append((m, (v - m[:, None]).square().mean(1), v.abs().mean(1)))
    return [torch.stack(t).cpu() for t in zip(*out)]


@pytest.mark.parametrize("dtype,last,shape", [("f32", False, (64, 4, 1024, 1024, 4)), ("f16", False, (64, 4, 1448, 1448, 4)),
                                              ("f32", False, (2, 3, 3000, 3000, 3)), ("f32", True, (8, 4, 2048, 2048, 1)),
                                              ("f32", True, (1, 2, 8192, 8192, 2))], ids=str)
def test_long_planes_whose_first_rows_differ(dtype, last, shape):
    """Every thread's first values are a border's: shifted by 1000 spreads from
    the rest.  Tolerances as in check(): chains of at most 128 additions."""
    n, c, h, w, groups = shape
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(n, c, h, w, generator=g, device="cuda")
    x[:, :, :2 if not last else 1] += 1000.0
    x = layout(x.to(DTYPES[dtype]), last)
    _, mean, rstd = wt.wtconv_group_norm_forward(x, groups)
    m, var, ex = stats64(x, groups)
    r = 1 / torch.sqrt(var + 1e-5)
    within(mean, m, 2.0 ** -24 * 128 * ex, "mean")
    within(rstd, r, r * 2.0 ** -24 * (64 + 8) + r ** 3 * (2.0 ** -24 * 128 * ex) ** 2, "rstd")


@pytest.mark.parametrize("shape,dtype,layouts", [
    ((64, 4, 1024, 1024, 4), "f32", (False, False)), ((2, 2, 4096, 4096, 2), "f32", (True, True)),
    ((65536, 8, 8, 8, 2), "f32", (True, True)), ((65536, 8, 7, 9, 2), "f32", (False, False)),
    ((1, 64, 4096, 4096, 8), "f32", (False, True)), ((1, 64, 4096, 4096, 8), "bf16", (True, False)),
    ((1, 33, 4001, 2999, 3), "f16", (False, True)),
], ids=str)
def test_long_sums_of_equal_gradients(shape, dtype, layouts):
    """dy = 0.3 everywhere: each addition to a growing sum is rounded the same
    way, so that a chain of 2000 is off by 350 u.  dbeta and dgamma within the
    bounds of Norm64.backward (act none: the slope is 1), dx's two means through
    dx itself, which is zero for a constant dy but for their error."""
    n, c, h, w, groups = shape
    lx, ly = layouts
    g = torch.Generator(device="cuda").manual_seed(4)
    x = layout(torch.randn(n, c, h, w, generator=g, device="cuda").to(DTYPES[dtype]), lx)
    dy = layout(torch.full((n, c, h, w), 0.3, device="cuda", dtype=DTYPES[dtype]), ly)
    step = max(1, 2 ** 26 // (c * h * w))
    sums = torch.zeros(3, c, dtype=torch.float64, device="cuda")
    mean, rstd = (torch.empty(n, groups, device="cuda") for _ in range(2))
    for i in range(0, n, step):
        v = x[i:i + step].double().reshape(-1, groups, c // groups * h * w)
        m = v.mean(2)
        r = 1 / torch.sqrt((v - m[..., None]).square().mean(2) + 1e-5)
        mean[i:i + step], rstd[i:i + step] = m, r
        # from the rounded statistics, as the call gets them
        xh = (v - mean[i:i + step].double()[..., None]) * rstd[i:i + step].double()[..., None]
        xh = xh.view(-1, c, h * w)
        sums[0] += xh.sum((0, 2))
        sums[1] += xh.abs().sum((0, 2))
        sums[2] += xh.square().sum((0, 2))
    d = dy.flatten()[0].item()
    count = n * h * w
    sx, sa, sq = (t.cpu() for t in sums)
    dx, dg, db = wt.wtconv_group_norm_backward(x, dy, groups, mean, rstd)
    u = 2.0 ** -24
    # e = |dy| u (16 (1 + |z|) + 8 |xh| + 4 |z|), z = xh
    within(db, torch.full((c,), d * count, dtype=torch.float64), u * d * (16 * count + 28 * sa + 128 * count), "dbeta")
    within(dg, d * sx, u * d * (16 * sa + 28 * sq + 136 * sa), "dgamma")
    # E[t xh] is about 0 as well, so dx = rstd (t - E[t] - xh E[t xh]): errors of
    # E[t] and of E[t xh] (of magnitudes |t| and |t| E|xh|, E|xh| < 1), 8 u of |t|
    # for the rest, xh up to 7; half a step of 16 bits is below that
    tol = rstd.max().item() * d * u * ((16 + 28 + 128 + 8) + 7 * (16 + 28 + 136 + 8))
    assert dx.float().abs().max().item() <= tol


@pytest.mark.parametrize("layouts", LAYOUTS, ids=str)
@pytest.mark.parametrize("shape", [(2, 16, 40, 40, 4), (2, 16, 8, 8, 4), (1, 8, 256, 16, 2), (300, 2, 64, 64, 2),
                                   (1, 512, 64, 64, 1)], ids=str)
def test_a_variance_beyond_fp32(shape, layouts):
    """A spread of 1e20: the variance is infinite, as include/wtconv.h says."""
    n, c, h, w, groups = shape
    lx, ly = layouts
    g = torch.Generator(device="cuda").manual_seed(6)
    x = layout(1e20 * torch.randn(n, c, h, w, generator=g, device="cuda"), lx)
    beta = torch.randn(c, generator=g, device="cuda")
    y, mean, rstd = wt.wtconv_group_norm_forward(x, groups, None, beta, channels_last=ly)
    assert torch.equal(rstd, torch.zeros_like(rstd)) and torch.isfinite(mean).all()
    assert torch.equal(y, beta.view(1, c, 1, 1).expand_as(y))
    dx, _, _ = wt.wtconv_group_norm_backward(x, layout(torch.ones_like(x), ly), groups, mean, rstd, None, beta)
    assert torch.equal(dx, torch.zeros_like(dx))


@pytest.mark.parametrize("layouts", LAYOUTS, ids=str)
@pytest.mark.parametrize("shape", [(1, 512, 64, 64, 1), (2, 1024, 7, 8, 512), (1, 6, 600, 600, 2)], ids=str)
def test_a_bad_value_in_groups_of_many_channels_and_of_few(shape, layouts):
    """Groups whose ranges a kernel between the walks joins, a workgroup or a wave
    each: the bad value, in the first set of its group or a later one, stays there."""
    n, c, h, w, groups = shape
    lx, ly = layouts
    x, dy, gamma, beta = inputs(shape, "f32", 12)
    clean = wt.wtconv_group_norm_forward(layout(x.cuda(), lx), groups, gamma.cuda(), beta.cuda(), act="silu",
                                         channels_last=ly)[0]
    per = c // groups
    for bad in (float("nan"), float("inf"), -float("inf")):
        for ch, row in ((0, 0), (per - 1, h - 1)):
            v = x.clone()
            v[n - 1, ch, row, w - 1] = bad
            v = layout(v.cuda(), lx)
            y, mean, rstd = wt.wtconv_group_norm_forward(v, groups, gamma.cuda(), beta.cuda(), act="silu",
                                                         channels_last=ly)
            dx, _, _ = wt.wtconv_group_norm_backward(v, layout(dy.cuda(), ly), groups, mean, rstd, gamma.cuda(),
                                                     beta.cuda(), act="silu")
            hit = torch.zeros(n, c, 1, 1, dtype=torch.bool)
            hit[n - 1, :per] = True
            hit = hit.expand_as(x).cuda()
            assert torch.isnan(y[hit]).all() and torch.isnan(dx[hit]).all(), (bad, ch)
            assert torch.equal(y[~hit], clean[~hit]) and torch.isfinite(dx[~hit]).all(), (bad, ch)
