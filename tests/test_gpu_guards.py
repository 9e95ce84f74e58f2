"""What the calls around the layer write lies in their outputs and workspaces, and what
they read in their inputs, at the sizes that end inside a tile or an access: outputs and
workspaces lie between bytes that have to stay, inputs between NaNs that would show."""
import pytest
import torch

import level_haar_wavelet_amd as wt
from tests.block_util import DTYPES, Gated64, check, rms64, rms_back64, rms_tol
from tests.guard_util import Guards, among_nan

pytestmark = pytest.mark.gpu
CODES = {"f32": 0, "f16": 1, "bf16": 2}
NAMES = ("dx", "dw_gate", "dw_up", "db_gate", "db_up")

# few rows, short rows and long ones; one of everything; one row behind a tile's last;
# columns that end inside an access; (8193, 72, 1036) fills the chip with tiles of 256
GATED = [(1, 1, 1), (3, 1, 5), (17, 40, 33), (64, 129, 30), (65, 1, 7), (65, 64, 64), (65, 300, 64), (129, 33, 65),
         (129, 192, 68), (130, 40, 1), (257, 136, 260), (257, 96, 131), (257, 264, 131), (100, 300, 77),
         (8193, 72, 1036), (8193, 300, 1030)]


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,c,f", GATED)
def test_gated(m, c, f, dtype, offset):
    dt, f32 = DTYPES[dtype], torch.float32
    gen = torch.Generator(device="cuda").manual_seed(m + c + f)

    def rand(*shape, scale=1.0, of=dt):
        return among_nan((scale * torch.randn(shape, generator=gen, device="cuda")).to(of), offset)

    x, wg, wu, dh = rand(m, c), rand(f, c, scale=c ** -0.5), rand(f, c, scale=c ** -0.5), rand(m, f)
    bg, bu = rand(f, scale=0.3, of=f32), rand(f, scale=0.3, of=f32)
    ref = Gated64(x, wg, wu, bg, bu, "silu")
    want = ref.backward(dh)
    g = Guards()
    work = [g.workspace(wt.wtconv_gated_workspace_size((m, c), f, CODES[dtype], op)) for op in (0, 3)]
    h = g.output((m, f), dt, offset)
    wt.wtconv_gated_forward(x, wg, wu, bg, bu, h=h, workspace=work[0])
    check("h", h, ref.h, ref.h_tol())
    for dw in (dt, f32):
        outs = [g.output(s, t, offset) for s, t in (((m, c), dt), ((f, c), dw), ((f, c), dw), ((f,), f32), ((f,), f32))]
        wt.wtconv_gated_backward(x, dh, wg, wu, bg, bu, workspace=work[1], dw_dtype=dw, **dict(zip(NAMES, outs)))
        for name, got in zip(NAMES, outs):
            check(name, got, *want[name])
    g.assert_whole()


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,c", [(1, 1), (3, 7), (257, 9), (300, 96), (257, 33), (65, 1024), (9, 2047), (7, 5003),
                                    (5, 8200), (3, 16391), (2050, 17)])
def test_rms(rows, c, dtype, offset):
    dt, f32 = DTYPES[dtype], torch.float32
    gen = torch.Generator(device="cuda").manual_seed(rows + c)
    x, r, dy, dh = (among_nan(torch.randn(rows, c, generator=gen, device="cuda").to(dt), offset) for _ in range(4))
    gamma = among_nan(1 + 0.2 * torch.randn(c, generator=gen, device="cuda"), offset)
    g = Guards()
    y, h, rstd = g.output((rows, c), dt, offset), g.output((rows, c), dt, offset), g.output((rows,), f32, offset)
    wt.wtconv_rms_norm_forward(x, r, gamma, y=y, h=h, rstd=rstd)
    sums = (x.float() + r.float()).to(dt)
    assert torch.equal(h, sums)
    want, _ = rms64(sums, gamma, 1e-6)
    check("y", y, want, rms_tol(want, dt))
    dx, dgamma = g.output((rows, c), dt, offset), g.output((c,), f32, offset)
    work = g.workspace(wt.wtconv_rms_norm_workspace_size((rows, c), CODES[dtype], 3))
    h, rs = among_nan(sums, offset), among_nan(rstd, offset)
    wt.wtconv_rms_norm_backward(h, dy, rs, gamma, dh=dh, dx=dx, dgamma=dgamma, workspace=work)
    want, tol, gwant, gtol = rms_back64(h, dy, dh, gamma, rs)
    check("dx", dx, want, tol)
    check("dgamma", dgamma, gwant, gtol)
    g.assert_whole()


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", [[1], [7, 0, 8, 9, 255, 2049], [8193, 3, 100003], [1 + 37 * i % 301 for i in range(300)]],
                         ids=len)
def test_clip(sizes, dtype, offset):
    dt = DTYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(len(sizes))
    pad = 4096 // (len(sizes) // 100 + 1)
    grads = []
    for n in sizes:  # NaNs beside every gradient
        raw = torch.full((n + offset + 2 * pad,), float("nan"), dtype=dt, device="cuda")
        grads.append(raw[pad + offset:pad + offset + n].copy_(torch.randn(n, generator=gen, device="cuda")))
    norm = float(torch.cat([t.double() for t in grads]).norm())
    g = Guards()
    # the outputs in one buffer, three elements between two of them
    flat = g.output((sum(n + 3 for n in sizes) + offset,), dt)
    flat.fill_(-7.0)
    out, between, at = [], [], offset
    for n in sizes:
        out.append(flat[at:at + n])
        between.append(flat[at + n:at + n + 3])
        at += n + 3
    total = g.output((), torch.float32, offset)
    work = g.workspace(wt.wtconv_grad_norm_workspace_size(len(sizes)))
    wt.wtconv_clip_grad_norm(grads, 0.3 * norm, out=out, norm=total, workspace=work)
    assert float(total) == pytest.approx(norm, rel=2.0 ** -23)
    for t, o in zip(grads, out):
        want = t.double() * min(1.0, 0.3 * norm / (norm + 1e-6))
        check("out", o, want, want.abs() * (3 * 2.0 ** -24 + (0 if dtype == "f32" else torch.finfo(dt).eps / 2)) + 2.0 ** -25)
    assert bool((torch.cat(between) == -7.0).all()) and bool((flat[:offset] == -7.0).all())
    wt.wtconv_grad_norm(grads, norm=total, workspace=work)
    assert float(total) == pytest.approx(norm, rel=2.0 ** -23)
    g.assert_whole()


# dg and du beyond 2 GB (16 bits: beyond 4), columns that end inside a tile.  Small whole numbers,
# whose sums are exact in fp32: gradients come out bit by bit, every row's part among them
@pytest.mark.parametrize("m,c,f,dtype", [(1100000, 16, 1028, "bf16"), (1100000, 264, 1026, "f16"),
                                         (560000, 32, 1028, "f32")])
def test_weights_gradients_beyond_2_gb(m, c, f, dtype):
    dt = DTYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(1)

    def ints(*shape):
        return torch.randint(-1, 2, shape, generator=g, device="cuda", dtype=torch.int8)

    x = ints(m, c).to(dt)
    wg, wu = ints(f, c).to(dt), ints(f, c).to(dt)
    dh = torch.empty(m, f, dtype=dt, device="cuda")
    for part in dh.split(100000):
        part.copy_(ints(*part.shape))
    _, dwg, dwu, dbg, dbu = wt.wtconv_gated_backward(x, dh, wg, wu, act="none", need=(False, True, True),
                                                     dw_dtype=torch.float32)
    want = [torch.zeros(f, c, dtype=torch.float64, device="cuda") for _ in range(2)]
    bias = [torch.zeros(f, dtype=torch.float64, device="cuda") for _ in range(2)]
    for xs, ds in zip(x.split(50000), dh.split(50000)):
        xs, ds = xs.double(), ds.double()
        for i, w in enumerate((wu, wg)):  # dg = dh u, du = dh g
            d = ds * (xs @ w.double().t())
            assert float(d.abs().max()) <= 256  # whole in every type
            want[i] += d.t().contiguous() @ xs
            bias[i] += d.sum(0)
    for got, ref in zip((dwg, dwu, dbg, dbu), want + bias):
        assert float(ref.abs().max()) < 2 ** 20 and torch.equal(got.double(), ref)
