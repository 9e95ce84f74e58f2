"""The gated product on the GPU against its formulas in fp64."""
import pytest
import torch

import level_haar_wavelet_amd as wt
from level_haar_wavelet_amd.module import GatedLinear
from tests.block_util import DTYPES, Gated64, check

pytestmark = pytest.mark.gpu
NAMES = ("dx", "dw_gate", "dw_up", "db_gate", "db_up")


def make(m, c, f, dtype, seed=0, bias=True, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, scale=1.0, dt=DTYPES[dtype]):
        n = 1
        for q in shape:
            n *= q
        t = torch.empty(n + offset, dtype=dt, device="cuda")[offset:].view(shape)
        return t.copy_(scale * torch.randn(shape, generator=g, device="cuda"))

    f32 = torch.float32
    return (rand(m, c), rand(f, c, scale=c ** -0.5), rand(f, c, scale=c ** -0.5),
            rand(f, scale=0.3, dt=f32) if bias else None, rand(f, scale=0.3, dt=f32) if bias else None, rand(m, f))


def run(m, c, f, dtype, act, seed=0, bias=True, offset=0):
    x, wg, wu, bg, bu, dh = make(m, c, f, dtype, seed, bias, offset)
    ref = Gated64(x, wg, wu, bg, bu, act)
    # what the workspace holds before the call has no part in it
    code = {"f32": 0, "f16": 1, "bf16": 2}[dtype]
    work = [torch.full((wt.wtconv_gated_workspace_size(x.shape, f, code, op),), 255, dtype=torch.uint8, device="cuda")
            for op in (0, 3)]
    h = wt.wtconv_gated_forward(x, wg, wu, bg, bu, act=act, workspace=work[0])
    check("h", h, ref.h, ref.h_tol())
    outs = wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu, act=act, workspace=work[1])
    for name, got in zip(NAMES, outs):
        check(name, got, *ref.backward(dh)[name])
    return h, outs


# single rows and few (each number of row groups), ragged against every tile, rows
# that no access divides, one of everything
SHAPES = [(1, 1, 1), (1, 64, 48), (16, 72, 40), (17, 256, 100), (33, 100, 64), (64, 512, 96), (65, 64, 64),
          (130, 96, 192), (200, 72, 129), (129, 33, 65), (257, 136, 260), (300, 301, 77), (1000, 8, 8), (500, 40, 500)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,c,f", SHAPES)
def test_shapes(m, c, f, dtype):
    run(m, c, f, dtype, "silu", seed=m + c + f)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("m", [5, 150])
def test_activations(act, bias, m, dtype):
    run(m, 96, 70, dtype, act, seed=2, bias=bias)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m", [9, 140])
def test_relu(dtype, m):
    """Sums that are exact in fp32, so that a gate's sign is the formula's: small whole numbers; zeros among the gates."""
    g = torch.Generator().manual_seed(7)
    x = torch.randint(-2, 3, (m, 40), generator=g).to(DTYPES[dtype]).cuda()
    wg, wu = (torch.randint(-2, 3, (72, 40), generator=g).to(DTYPES[dtype]).cuda() for _ in range(2))
    dh = torch.randint(-1, 2, (m, 72), generator=g).to(DTYPES[dtype]).cuda()
    gate, up = (x.double() @ w.double().t() for w in (wg, wu))
    assert bool((gate == 0).any())
    h = wt.wtconv_gated_forward(x, wg, wu, act="relu")
    assert torch.equal(h.double(), (gate.clamp(min=0) * up).to(h.dtype).double())
    dg, du = dh.double() * up * (gate > 0), dh.double() * gate.clamp(min=0)
    dx, dwg, dwu, dbg, dbu = wt.wtconv_gated_backward(x, dh, wg, wu, act="relu")
    # whole numbers below 256: exact in every type until the outputs' own rounding
    assert float(torch.stack([dg.abs().max(), du.abs().max()]).max()) < 256
    for got, ref in ((dx, dg @ wg.double() + du @ wu.double()), (dwg, dg.t() @ x.double()), (dwu, du.t() @ x.double())):
        assert torch.equal(got.double(), ref.to(got.dtype).double())
    assert torch.equal(dbg.double(), dg.sum(0)) and torch.equal(dbu.double(), du.sum(0))


# the tiles of 256, for each product, and sums cut into slices
@pytest.mark.parametrize("m,c,f,dtype", [
    (8200, 72, 1032, "bf16"), (8200, 72, 520, "f32"), (65600, 64, 72, "f16"), (65600, 40, 40, "f32"),
    (100, 4096, 2056, "bf16"), (70, 136, 4100, "f16"), (66, 140, 2000, "f32"), (20000, 24, 40, "bf16"),
])
def test_large(m, c, f, dtype):
    run(m, c, f, dtype, "silu")


# outputs and gradients beyond 2 GB, columns that end inside a tile: every part of the
# rows comes out as it does by itself, and nothing is written behind its place
@pytest.mark.parametrize("m,c,f,dtype", [(1100000, 16, 1028, "bf16"), (1100000, 264, 1026, "f16"),
                                         (560000, 32, 1028, "f32")])
def test_beyond_2_gb(m, c, f, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    dt = DTYPES[dtype]
    x = torch.randn(m, c, generator=g, device="cuda").to(dt)
    wg, wu = ((torch.randn(f, c, generator=g, device="cuda") / c ** 0.5).to(dt) for _ in range(2))
    dh = torch.empty(m, f, dtype=dt, device="cuda")
    for part in dh.split(100000):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    assert dh.numel() * dh.element_size() > 2 ** 31
    h = wt.wtconv_gated_forward(x, wg, wu)
    dx = wt.wtconv_gated_backward(x, dh, wg, wu, need=(True, False, False))[0]
    for at in range(0, m, 204800):  # whole tiles
        rows = slice(at, at + 204800)
        assert torch.equal(h[rows], wt.wtconv_gated_forward(x[rows], wg, wu)), at
        assert torch.equal(dx[rows], wt.wtconv_gated_backward(x[rows], dh[rows], wg, wu, need=(True, False, False))[0]), at


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,c,f", [(3, 64, 40), (150, 64, 40), (150, 61, 43)])
def test_addresses(m, c, f, dtype):
    run(m, c, f, dtype, "gelu", offset=1)


def test_needs_and_given_outputs():
    x, wg, wu, bg, bu, dh = make(300, 64, 96, "bf16")
    full = wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu)
    assert all(torch.equal(a, b) for a, b in zip(full, wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu)))
    for need in ((True, False, False), (False, True, False), (False, False, True), (True, False, True)):
        part = wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu, need=need)
        wanted = (need[0], need[1], need[1], need[2], need[2])
        for w, a, b in zip(wanted, part, full):
            assert torch.equal(a, b) if w else a is None
    given = {n: torch.full_like(t, 7.0) for n, t in zip(NAMES, full)}
    part = wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu, **given)
    assert all(a is given[n] and torch.equal(a, b) for n, a, b in zip(NAMES, part, full))
    # one weight for both projections, and leading dimensions
    both = wt.wtconv_gated_forward(x.view(3, 2, 50, 64), wg, wg, bg, bg, act="none")
    ref = Gated64(x, wg, wg, bg, bg, "none")
    check("h", both.view(300, 96), ref.h, ref.h_tol())


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("m", [40, 300])
def test_bad_rows(m, dtype):
    """A bad row stays in its row of h and dx."""
    x, wg, wu, bg, bu, dh = make(m, 72, 80, dtype)
    good = wt.wtconv_gated_forward(x, wg, wu, bg, bu), wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu)[0]
    x[3, 5], x[m - 1, 71] = float("nan"), float("inf")
    h = wt.wtconv_gated_forward(x, wg, wu, bg, bu)
    dx, dwg, _, dbg, _ = wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu)
    rows = [i for i in range(m) if i not in (3, m - 1)]
    assert torch.equal(h[rows], good[0][rows]) and torch.equal(dx[rows], good[1][rows])
    for t in (h, dx):
        assert bool(t[3].isnan().all()) and not bool(t[m - 1].isfinite().any())
    assert not bool(dwg.isfinite().any()) and not bool(dbg.isfinite().any())


def test_graded_rows():
    """fp32 rows of very different sizes keep their own digits."""
    x, wg, wu, _, _, dh = make(200, 96, 64, "f32", bias=False)
    x *= 2.0 ** torch.linspace(-60, 20, 200, device="cuda")[:, None]
    ref = Gated64(x, wg, wu, None, None, "none")
    h = wt.wtconv_gated_forward(x, wg, wu, act="none")
    for row in (h - ref.h).norm(dim=1) / ref.h.norm(dim=1):
        assert float(row) < 1e-6


def test_captured():
    """Replays beside eager calls and another captured call, each against the eager result."""
    sets = [make(300, 64, 96, "bf16", seed=1), make(130, 33, 40, "f32", seed=2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x, wg, wu, bg, bu, dh in sets:
            wt.wtconv_gated_forward(x, wg, wu, bg, bu)
            wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for x, wg, wu, bg, bu, dh in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append((wt.wtconv_gated_forward(x, wg, wu, bg, bu),) + wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu))
    for _ in range(4):
        for s in sets:
            s[0].mul_(-0.9)
            s[5].mul_(1.1)
        for g in graphs:
            g.replay()
        for (x, wg, wu, bg, bu, dh), out in zip(sets, outs):
            eager = (wt.wtconv_gated_forward(x, wg, wu, bg, bu),) + wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, eager))


def test_two_streams():
    """Two calls at once, each with its own workspace from its stream's pool."""
    sets = [make(2000, 64, 96, "bf16", seed=i) for i in range(2)]
    want = [wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu) for x, wg, wu, bg, bu, dh in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = [wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu, stream=s)
               for s, (x, wg, wu, bg, bu, dh) in zip(streams, sets)]
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", DTYPES)
def test_module_gradients(dtype):
    """The module's gradients (float32 parameters) against the formula's and differences."""
    torch.manual_seed(0)
    layer = GatedLinear(40, 56, act="gelu", device="cuda")
    with torch.no_grad():
        layer.b_gate.normal_()
        layer.b_up.normal_()
    x = torch.randn(2, 70, 40, device="cuda").to(DTYPES[dtype]).requires_grad_()
    a = torch.randn(2, 70, 56, device="cuda").to(DTYPES[dtype])
    layer(x).backward(a)
    params = (layer.w_gate, layer.w_up, layer.b_gate, layer.b_up)
    w16 = [p.detach().to(x.dtype) for p in params[:2]]
    ref = Gated64(x.detach().view(140, 40), *w16, layer.b_gate.detach(), layer.b_up.detach(), "gelu")
    want = ref.backward(a.view(140, 56))
    check("dx", x.grad.view(140, 40), *want["dx"])
    for p, name in zip(params, NAMES[1:]):
        assert p.grad.dtype == torch.float32
        check(name, p.grad, *want[name])
    if dtype == "f32":
        with torch.no_grad():
            v = [t.detach().double() for t in (x, *params)]
            d = [torch.randn_like(t) for t in v]

            def value(t):
                q = Gated64(t[0].view(140, 40), *t[1:], "gelu")
                return (q.h * a.double().view(140, 56)).sum()

            s = 1e-5
            diff = (value([t + s * q for t, q in zip(v, d)]) - value([t - s * q for t, q in zip(v, d)])) / (2 * s)
            own = sum((g.double() * q).sum() for g, q in zip((x.grad, *(p.grad for p in params)), d))
        assert float(own) == pytest.approx(float(diff), rel=1e-5)
    # frozen parts
    for p in params:
        p.grad = None
    layer.w_gate.requires_grad_(False)
    layer.b_up.requires_grad_(False)
    y = x.detach()
    layer(y).backward(a)
    assert layer.w_gate.grad is None and layer.b_up.grad is None
    check("dw_up", layer.w_up.grad, *want["dw_up"])
    check("db_gate", layer.b_gate.grad, *want["db_gate"])
