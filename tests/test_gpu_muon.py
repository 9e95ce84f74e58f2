"""Newton-Schulz orthogonalisation and the Muon step on the GPU against their
formulas in fp64."""
import math

import pytest
import torch

import level_haar_wavelet_amd as wt
from tests.train_util import DTYPES, U, ortho64, ortho_tol

pytestmark = pytest.mark.gpu

# batch, rows, cols: single values and vectors, both orientations, around the
# tile sizes 16, 32, 64, 128, odd sizes, the layer's parameters, stacks
SHAPES = [
    (1, 1, 1), (3, 1, 7), (2, 9, 1), (1, 2, 3), (5, 3, 2), (2, 16, 16), (1, 15, 17), (2, 31, 33), (1, 32, 500),
    (3, 384, 25), (1, 96, 25), (4, 32, 9), (2, 200, 49), (1, 49, 49), (2, 63, 65), (1, 64, 64), (2, 66, 64),
    (1, 96, 384), (1, 127, 129), (1, 128, 128), (2, 130, 300), (1, 257, 255), (1, 100, 1999), (1, 2500, 40),
    (1, 384, 1536), (2, 512, 512), (1, 700, 333), (1, 1, 5000), (1, 4097, 2),
    # one workgroup's limits: 256, 512, 1024 and 2048 columns of 32 rows, 512 of 64
    (2, 27, 256), (1, 25, 257), (2, 513, 30), (1, 32, 1025), (1, 2048, 32), (1, 20, 2049), (2, 64, 256), (1, 40, 300),
    (1, 512, 64), (1, 60, 513), (1, 65, 70),
]


# with those above, every kernel instance of the tiled path (tests/test_muon_plan.py):
# products and joins of tiles of 32, 64 and 128, stages of both depths, whole
# rounds of tiles with a last one cut along k, cuts over several matrices
LARGE = [
    (4, 1024, 1024), (1, 2048, 2048), (6, 1024, 700), (1, 1999, 3001), (6, 1675, 1632), (8, 3416, 483),
    (1, 1644, 1904), (4, 2570, 225), (4, 2892, 65), (1, 611, 3325), (1, 385, 397), (2, 1796, 1818), (4, 4201, 612),
    (8, 1282, 1241), (8, 673, 641), (3, 635, 1010),
]


def gradient(shape, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    b, r, c = shape
    k = min(r, c, 3)
    v = torch.randn(b, r, c, generator=g) + torch.randn(b, r, k, generator=g) @ torch.randn(b, k, c, generator=g)
    return (1e-3 * v).to(dtype)


def within(got, ref, steps, dtype, what):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape and torch.isfinite(got).all(), what
    over = torch.linalg.matrix_norm(got - ref) / ortho_tol(ref, steps, dtype)
    assert over.max() <= 1, "%s: %.3g times its tolerance" % (what, over.max())


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_the_formula(shape):
    for k, dtype in enumerate(DTYPES.values()):
        g = gradient(shape, 10 * SHAPES.index(shape) + k, dtype)
        print(shape, dtype, flush=True)
        within(wt.wtconv_orthogonalize(g.cuda()), ortho64(g), 5, dtype, "%s %s" % (shape, dtype))


@pytest.mark.parametrize("shape", [(1, 25, 96), (2, 100, 80), (1, 130, 600), (1, 300, 300)], ids=str)
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6, 7])
def test_number_of_steps(shape, steps):
    g = gradient(shape, steps)
    within(wt.wtconv_orthogonalize(g.cuda(), steps=steps), ortho64(g, steps), steps, torch.float32, str(shape))


@pytest.mark.parametrize("shape", [(40, 40), (25, 384), (160, 200), (90, 700)], ids=str)
def test_ranks_that_are_not_full(shape):
    """One row of values, a matrix of rank 2, repeated rows: directions with
    no value of their own stay empty."""
    torch.manual_seed(0)
    one = torch.zeros(shape)
    one[shape[0] // 2] = torch.randn(shape[1])
    low = torch.randn(shape[0], 2) @ torch.randn(2, shape[1])
    same = torch.randn(1, shape[1]).expand(shape).contiguous()
    for g in (one, low, same, one.mT.contiguous(), low.mT.contiguous()):
        got = wt.wtconv_orthogonalize(g.cuda())
        within(got, ortho64(g), 5, torch.float32, str(shape))
    assert torch.equal(wt.wtconv_orthogonalize(one.cuda())[0], torch.zeros(shape[1], device="cuda"))


@pytest.mark.parametrize("shape", [(2, 25, 64), (2, 150, 170), (2, 90, 700)], ids=str)
@pytest.mark.parametrize("size", [1e-30, 1e-12, 1.0, 1e15, 1e30])
def test_size_of_the_gradient(shape, size):
    """The norm's square passes fp32's range at both ends."""
    g = gradient(shape, 3) / 1e-3 * size
    within(wt.wtconv_orthogonalize(g.cuda()), ortho64(g), 5, torch.float32, "%g" % size)
    within(wt.wtconv_orthogonalize(g.cuda(), eps=0.0), ortho64(g, eps=0.0), 5, torch.float32, "%g, eps 0" % size)


@pytest.mark.parametrize("shape", [(25, 64), (150, 170), (90, 700), (700, 90)], ids=str)
def test_zero_and_bad_matrices_of_a_stack(shape):
    g = gradient((4,) + shape, 8)
    clean = wt.wtconv_orthogonalize(g.cuda())
    g[0] = 0
    g[2, 3, 4] = float("nan")
    g[3, 1, 1] = float("inf")
    got = wt.wtconv_orthogonalize(g.cuda())
    assert torch.equal(got[0], torch.zeros_like(got[0]))
    assert torch.equal(got[1], clean[1])
    assert torch.isnan(got[2]).all() and torch.isnan(got[3]).all()


def plain_muon(w, g, m, lr, mu, wd, scale, nesterov, steps, eps):
    g, m, w = g.double(), m.double(), w.double()
    m = mu * m + (1 - mu) * g
    u = (1 - mu) * g + mu * m if nesterov else m
    return (1 - lr * wd) * w - lr * scale * ortho64(u, steps, eps), m


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape", [(1, 96, 25), (3, 64, 25), (1, 1, 9), (2, 100, 128), (1, 333, 200), (1, 120, 900)],
                         ids=str)
def test_muon_step(shape, nesterov):
    for k, dtype in enumerate(DTYPES.values()):
        g = gradient(shape, k, dtype)
        torch.manual_seed(k)
        w, m = 0.1 * torch.randn(shape), 1e-3 * torch.randn(shape)
        # fp32 values of the hyperparameters, as the entry point takes them
        lr, mu, wd, scale = (float(torch.tensor(v)) for v in (0.5, 0.9, 0.01, 1.5))
        rw, rm = plain_muon(w, g, m, lr, mu, wd, scale, nesterov, 5, 1e-7)
        wd_, gd, md = w.cuda(), g.cuda(), m.cuda()
        wo, mo = torch.full_like(wd_, 9.0), torch.full_like(md, 9.0)
        kw = dict(lr=lr, mu=mu, weight_decay=wd, scale=scale, nesterov=nesterov)
        a = wt.wtconv_muon_step(wd_, gd, md, weight_out=wo, momentum_out=mo, **kw)
        assert a[0] is wo and a[1] is mo
        assert torch.equal(wd_.cpu(), w) and torch.equal(md.cpu(), m) and torch.equal(gd.cpu(), g)
        # momentum: four roundings of its two terms
        assert ((mo.cpu().double() - rm).abs() <= 4 * U * (mu * m.double().abs() + (1 - mu) * g.double().abs())
                + 1e-40).all()
        err = torch.linalg.matrix_norm(wo.cpu().double() - rw)
        # the update's error times lr scale, and four roundings of the weight;
        # U itself is off by 8 u, which the iteration magnifies as X_0's
        tol = lr * scale * (ortho_tol(rw, 5, torch.float32) + 8 * U * 3.4445 ** 5) \
            + 4 * U * torch.linalg.matrix_norm(w.double())
        assert (err <= tol).all(), (shape, dtype, err / tol)
        b = wt.wtconv_muon_step(wd_, gd, md, **kw)  # in place
        assert b[0] is wd_ and b[1] is md and torch.equal(wd_, wo) and torch.equal(md, mo)


@pytest.mark.parametrize("shape", [(1, 25, 64), (1, 150, 171), (2, 90, 701), (1, 333, 77)], ids=str)
def test_unaligned_buffers_and_what_lies_behind_them(shape):
    k = math.prod(shape)
    for dtype in DTYPES.values():
        bufs = [torch.randn(k + 30, device="cuda").to(dtype) for _ in range(2)]
        g, out = (b[1:k + 1].view(shape) for b in bufs)
        ref = wt.wtconv_orthogonalize(g.clone())
        edge = [b[[0] + list(range(k + 1, k + 30))].clone() for b in bufs]
        wt.wtconv_orthogonalize(g, out=out)
        tol = 1e-4 if dtype == torch.float32 else 4 * torch.finfo(dtype).eps
        assert torch.allclose(out.float(), ref.float(), atol=tol, rtol=tol)
        for b, e in zip(bufs, edge):
            assert torch.equal(b[[0] + list(range(k + 1, k + 30))], e)
    f = [torch.randn(k + 30, device="cuda") for _ in range(5)]
    w, g, m, wo, mo = (b[1:k + 1].view(shape) for b in f)
    edge = [b[[0] + list(range(k + 1, k + 30))].clone() for b in f]
    rw, rm = wt.wtconv_muon_step(w.clone(), g.clone(), m.clone(), lr=0.1)
    wt.wtconv_muon_step(w, g, m, lr=0.1, weight_out=wo, momentum_out=mo)
    assert torch.allclose(wo, rw, atol=1e-4) and torch.equal(mo, rm)
    for b, e in zip(f, edge):
        assert torch.equal(b[[0] + list(range(k + 1, k + 30))], e)


def test_refusals_on_the_gpu():
    g = torch.randn(8, 12, device="cuda")
    for bad in (g.t(), g[0], g.double(), g.view(1, 2, 4, 12)):
        with pytest.raises(TypeError):
            wt.wtconv_orthogonalize(bad)
    with pytest.raises(TypeError):
        wt.wtconv_orthogonalize(g, out=torch.empty_like(g, dtype=torch.float16))
    for kw in (dict(steps=0), dict(steps=17), dict(eps=-1.0), dict(out=g)):
        with pytest.raises(wt._native.WtconvError):
            wt.wtconv_orthogonalize(g, **kw)
    with pytest.raises(wt._native.WtconvError):
        wt.wtconv_orthogonalize(g[:0])
    with pytest.raises(wt._native.WtconvError):
        wt.wtconv_orthogonalize(torch.randn(80, 90, device="cuda"),
                                workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    w, m = g.clone(), g.clone()
    with pytest.raises(TypeError):
        wt.wtconv_muon_step(w.half(), g, m, lr=0.1)
    with pytest.raises(TypeError):
        wt.wtconv_muon_step(w[:4], g, m, lr=0.1)
    with pytest.raises(TypeError):
        wt.wtconv_muon_step(w, g, m.cpu(), lr=0.1)
    with pytest.raises(wt._native.WtconvError):
        wt.wtconv_muon_step(w, g, w, lr=0.1)  # one buffer for both


@pytest.mark.parametrize("shape", [(2, 96, 25), (1, 300, 260), (2, 100, 900)], ids=str)
def test_same_bits_every_time_and_on_other_streams(shape):
    g = gradient(shape, 5).cuda()
    ref = wt.wtconv_orthogonalize(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            got.append(wt.wtconv_orthogonalize(g, stream=s))
        torch.cuda.synchronize()
        assert all(torch.equal(t, ref) for t in got)


@pytest.mark.parametrize("shape", [(2, 96, 25), (1, 300, 260), (2, 100, 900), (1, 64, 90)], ids=str)
def test_captured_steps_replay_on_new_gradients(shape):
    w, g, m = torch.randn(shape, device="cuda"), gradient(shape, 1).cuda(), torch.zeros(shape, device="cuda")
    w2, m2 = w.clone(), m.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        wt.wtconv_muon_step(w.clone(), g, m.clone(), lr=0.1)
        wt.wtconv_orthogonalize(g)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wt.wtconv_muon_step(w, g, m, lr=0.1)
        o = wt.wtconv_orthogonalize(g)
    for r in range(4):
        g.copy_(gradient(shape, 30 + r))
        o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        wt.wtconv_muon_step(w2, g, m2, lr=0.1)
        assert torch.equal(w, w2) and torch.equal(m, m2) and torch.equal(o, wt.wtconv_orthogonalize(g))


def test_optimizer_on_the_layer_and_its_state():
    from level_haar_wavelet_amd.module import WTConv2d
    from level_haar_wavelet_amd.optim import Muon

    torch.manual_seed(0)
    layer = WTConv2d(16, 5, 2, device="cuda")
    lin = torch.nn.Linear(16, 40, device="cuda")
    params = [layer.w_base, layer.w_lvl, lin.weight]
    opt = Muon(params, lr=0.1, weight_decay=0.1)
    ref = [(p.detach().cpu(), torch.zeros(p.shape)) for p in params]
    for it in range(3):
        for i, p in enumerate(params):
            p.grad = 1e-2 * torch.randn(p.shape, device="cuda")
            if i == 2:
                p.grad = p.grad.t().contiguous().t()  # a gradient that is not contiguous
        if it == 1:
            params[0].grad = None  # left as it is
        opt.step()
        for i, p in enumerate(params):
            if p.grad is None:
                assert torch.equal(p.detach().cpu(), ref[i][0])
                continue
            b, r, c = ((1, 16, 25), (2, 64, 25), (1, 40, 16))[i]
            v = lambda t: t.reshape(b, r, c)
            rw, rm = plain_muon(v(ref[i][0]), v(p.grad.cpu()), v(ref[i][1]), 0.1, 0.95, 0.1, max(1, r / c) ** 0.5,
                                True, 5, 1e-7)
            assert torch.allclose(v(p.detach().cpu()).double(), rw, atol=1e-5)
            assert torch.allclose(v(opt.state[p]["momentum_buffer"].cpu()).double(), rm, atol=1e-8)
            ref[i] = (p.detach().cpu().clone(), opt.state[p]["momentum_buffer"].cpu().clone())
    again = Muon(params, lr=0.1)
    again.load_state_dict(opt.state_dict())
    assert torch.equal(again.state[params[1]]["momentum_buffer"], opt.state[params[1]]["momentum_buffer"])


def test_a_first_step_is_not_captured():
    from level_haar_wavelet_amd.optim import Muon

    p = torch.nn.Parameter(torch.randn(8, 12, device="cuda"))
    p.grad = torch.randn_like(p)
    opt = Muon([p], lr=0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin()
        with pytest.raises(RuntimeError, match="cannot be captured"):
            opt.step()
        p.grad.mul_(1.0)  # a capture that holds something
        graph.capture_end()
    torch.cuda.current_stream().wait_stream(s)
    before = p.detach().clone()
    opt.step()  # and an ordinary step still runs
    assert not torch.equal(p, before)


def test_two_graphs_with_their_own_workspaces_run_side_by_side():
    """Two captured orthogonalisations replayed on two streams at once: each has
    its own workspace and gives its own result, every time."""
    gs = [gradient((1, 300, 260), k).cuda() for k in (1, 2)]
    ref = [wt.wtconv_orthogonalize(g) for g in gs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for g in gs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(wt.wtconv_orthogonalize(g))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in gs]
    for _ in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for o, r in zip(outs, ref))


def test_a_long_narrow_matrix_and_a_large_stack():
    """2^20 columns of 3 rows (the sum over k is long), and 4000 matrices of 7 x 9
    in one call."""
    for shape in ((1, 3, 1 << 20), (4000, 7, 9)):
        g = gradient(shape, 3)
        within(wt.wtconv_orthogonalize(g.cuda()), ortho64(g), 5, torch.float32, str(shape))


@pytest.mark.parametrize("bad", ["channels_last", "cpu", "too_large", "no_stack"])
def test_a_parameter_that_is_refused_stops_a_step_before_its_first_update(bad):
    from level_haar_wavelet_amd.optim import Muon

    good = torch.nn.Parameter(torch.randn(8, 8, device="cuda"))
    if bad == "channels_last":
        last = torch.nn.Parameter(torch.zeros(8, 4, 3, 3, device="cuda").contiguous(memory_format=torch.channels_last))
    elif bad == "cpu":
        last = torch.nn.Parameter(torch.zeros(8, 4, 3, 3))
    elif bad == "too_large":  # more columns than the entry point takes
        last = torch.nn.Parameter(torch.zeros(1, (1 << 22) + 1, device="cuda"))
    else:
        last = torch.nn.Parameter(torch.zeros(8, 4, 3, 3, device="cuda"))
    opt = Muon([good, last], lr=0.1, batch_dims=0)
    if bad == "no_stack":
        opt.param_groups[0]["batch_dims"] = 7
    good.grad, last.grad = torch.randn_like(good), torch.zeros_like(last)
    before, version = good.detach().clone(), good._version
    with pytest.raises((TypeError, ValueError, wt._native.WtconvError)):
        opt.step()
    assert torch.equal(good, before) and good._version == version and not opt.state


def test_ordinary_convolution_weights():
    """(out, in, k, k) and (out, in, 1, 1), batch_dims=0, against the formula."""
    from level_haar_wavelet_amd.optim import Muon

    for k in (1, 3):
        torch.manual_seed(k)
        conv = torch.nn.Conv2d(12, 20, k, device="cuda")
        opt = Muon([conv.weight], lr=0.1, batch_dims=0)
        old = conv.weight.detach().cpu()
        conv.weight.grad = 1e-2 * torch.randn_like(conv.weight)
        opt.step()
        r, c = 20, 12 * k * k
        v = lambda t: t.detach().cpu().reshape(1, r, c)
        rw, _ = plain_muon(v(old), v(conv.weight.grad), torch.zeros(1, r, c), 0.1, 0.95, 0.0, max(1, r / c) ** 0.5, True,
                           5, 1e-7)
        # lr scale <= 0.13 times the iteration's bound, and 4 u of the weights
        tol = 0.13 * (ortho_tol(rw, 5, torch.float32) + 8 * U * 3.4445 ** 5) + 4 * U * v(old).norm().item()
        assert (torch.linalg.matrix_norm(v(conv.weight).double() - rw) <= tol).all()


def ortho64_gpu(g, **kw):
    """ortho64 of a stack, on the GPU matrix by matrix."""
    return torch.stack([ortho64(m.cuda(), **kw).cpu() for m in g])


@pytest.mark.parametrize("shape", LARGE, ids=lambda s: "x".join(map(str, s)))
def test_every_instance_of_the_products(shape):
    i = LARGE.index(shape)
    half = (torch.float16, torch.bfloat16)[i % 2]
    for d in (torch.float32, half):
        g = gradient(shape, 900 + i, d)
        print(shape, d, flush=True)
        got = wt.wtconv_orthogonalize(g.cuda())
        within(got, ortho64_gpu(g), 5, d, "%s %s" % (shape, d))
        assert torch.equal(got, wt.wtconv_orthogonalize(g.cuda()))  # the same bits each time
    # a 16-bit result is the fp32 one of the same values, rounded once
    assert torch.equal(got, wt.wtconv_orthogonalize(g.cuda().float()).to(half))


@pytest.mark.parametrize("shape", [(1, 2048, 2048), (6, 1024, 700), (1, 1999, 3001), (6, 1675, 1632), (4, 1024, 1024)],
                         ids=lambda s: "x".join(map(str, s)))
def test_muon_step_of_large_matrices(shape):
    dtype = torch.float32 if shape[0] == 1 else torch.bfloat16
    g = gradient(shape, 3, dtype)
    torch.manual_seed(3)
    w, m = 0.1 * torch.randn(shape), 1e-3 * torch.randn(shape)
    lr, mu, wd, scale = (float(torch.tensor(v)) for v in (0.5, 0.9, 0.01, 1.5))
    wo, mo = wt.wtconv_muon_step(w.cuda(), g.cuda(), m.cuda(), lr=lr, mu=mu, weight_decay=wd, scale=scale)
    rm = mu * m.double() + (1 - mu) * g.double()
    rw = (1 - lr * wd) * w.double() - lr * scale * ortho64_gpu((1 - mu) * g.double() + mu * rm)
    # as in test_muon_step
    assert ((mo.cpu().double() - rm).abs() <= 4 * U * (mu * m.double().abs() + (1 - mu) * g.double().abs())
            + 1e-40).all()
    tol = lr * scale * (ortho_tol(rw, 5, torch.float32) + 8 * U * 3.4445 ** 5) + 4 * U * torch.linalg.matrix_norm(w.double())
    err = torch.linalg.matrix_norm(wo.cpu().double() - rw)
    assert (err <= tol).all(), (shape, err / tol)


@pytest.mark.parametrize("n", [30, 60, 130], ids=["one_block", "two_blocks", "tiles"])
def test_small_entries_next_to_large_ones(n):
    """One step on diag(d), d from 1 down to 2^-44: element i comes out as
    p(x_i) = a x + b x^3 + c x^5, x = d / |d|.  x is off by 2^-22 x or, below 2^-28
    (hi is a subnormal fp16 number of x 2^14, whose rest, up to 2^-25, is held to
    half of 2^-24 2^-11), by 2^-50; the diagonal of the polynomial's matrix by 2^-22
    of 3.45 and by about 40 2^-22 x^2 from x^2 and x^4; the fp32 sums add 2^-22 p
    at most.  The lo lo that is left out is 2^-22 p too, and below 2^-28, where lo
    holds a rest of up to 2^-39, 2^-11 3.45 of that: another 3.45 2^-50."""
    torch.manual_seed(n)
    d = (1 + torch.rand(n)) * torch.pow(2.0, -torch.arange(n) * 44.0 / (n - 1))
    for copies in ((1, 1), (1, 2), (2, 1)):  # two equal blocks: sums over both, singular values sqrt 2 larger
        g = torch.diag(d).repeat(copies)
        got = wt.wtconv_orthogonalize(g.cuda(), steps=1, eps=0.0).cpu().double()
        ref = ortho64(g, 1, 0.0)
        x = (d.double() * math.sqrt(max(copies)) / g.double().norm()).repeat(copies[0])
        tol = 2.0 ** -22 * (3.45 * 4 * x + 40 * x ** 3) + 3.45 * 2.0 ** -49
        assert ((got - ref).abs() <= tol[:, None]).all(), ((got - ref).abs() / tol[:, None]).max()
        assert torch.equal(got[ref == 0], torch.zeros_like(got[ref == 0]))


@pytest.mark.parametrize("shape", [(25, 384), (64, 512), (64, 1024), (384, 1536), (1030, 300), (1, 2048, 2048)], ids=str)
def test_rows_graded_over_many_powers_of_two(shape):
    """Every row keeps its own digits.  Row i of size x_i among others of up to 1:
    its entries and the polynomial's are off by 2^-22 of themselves (down to
    2^-28; here 2^-24 2^-6), lo lo by as much, and A_ij, about x_i x_j, by 2^-22 of
    itself, which P X brings to row i as 4.8 2^-22 x_i x_j^2, with sum x_j^2 = 1:
    8 2^-22 a step, five steps."""
    g = torch.Generator().manual_seed(1)
    *b, r, c = shape
    n = min(r, c)
    scale = torch.pow(2.0, -torch.arange(n) * 24.0 / (n - 1))
    m = torch.randn(shape, generator=g) * (scale[:, None] if r <= c else scale)
    got = wt.wtconv_orthogonalize(m.cuda()).cpu().double().view(r, c)
    ref = ortho64(m.view(r, c).cuda()).cpu()
    dim = 1 if r <= c else 0
    over = (got - ref).norm(dim=dim) / ref.norm(dim=dim) / (40 * 2.0 ** -22)
    assert over.max() <= 1, over.max()
