"""Weights' gradients in float32 under 16-bit activations."""
import ctypes

import pytest
import torch

import level_haar_wavelet_amd as wt
from level_haar_wavelet_amd import _native
from level_haar_wavelet_amd.module import GatedFunction, GatedLinear
from tests.block_util import DTYPES, Gated64, check, half_step

pytestmark = pytest.mark.gpu


def wide_tol(want, dtype):
    """The tolerance of a gradient that is not rounded to the activations' type."""
    value, tol = want
    return value, tol - half_step(value, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,c,f", [(140, 40, 56), (5, 33, 17), (3000, 264, 96)])
def test_module_keeps_the_sums(dtype, m, c, f):
    """float32 parameters get the float32 sums, not those rounded to the activations' type."""
    torch.manual_seed(m)
    layer = GatedLinear(c, f, act="silu", device="cuda")
    x = torch.randn(m, c, device="cuda").to(DTYPES[dtype])
    a = torch.randn(m, f, device="cuda").to(DTYPES[dtype])
    layer(x).backward(a)
    ref = Gated64(x, layer.w_gate.detach().to(x.dtype), layer.w_up.detach().to(x.dtype), layer.b_gate.detach(),
                  layer.b_up.detach(), "silu").backward(a)
    for p, name in ((layer.w_gate, "dw_gate"), (layer.w_up, "dw_up")):
        check(name, p.grad, *wide_tol(ref[name], x.dtype))
        # more digits than the activations' type has
        assert not torch.equal(p.grad, p.grad.to(x.dtype).float())


def test_module_sums_beyond_fp16():
    torch.manual_seed(0)
    layer = GatedLinear(24, 40, act="none", device="cuda")
    with torch.no_grad():
        layer.b_up.fill_(40.0)
    x = torch.randn(4096, 24, device="cuda").abs().half()
    a = torch.randn(4096, 40, device="cuda").abs().half()
    layer(x).backward(a)
    ref = Gated64(x, layer.w_gate.detach().half(), layer.w_up.detach().half(), layer.b_gate.detach(),
                  layer.b_up.detach(), "none").backward(a)
    assert float(ref["dw_gate"][0].abs().min()) > torch.finfo(torch.float16).max
    check("dw_gate", layer.w_gate.grad, *wide_tol(ref["dw_gate"], x.dtype))


# whole tiles and cut ones, of each size; rows that no access divides
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,c,f", [(1, 8, 8), (130, 96, 192), (257, 33, 65), (8200, 520, 1032), (20000, 24, 40),
                                   (70, 2056, 4100)])
def test_sums_are_those_that_are_rounded(dtype, m, c, f):
    """The float32 gradients rounded to the activations' type are that call's own."""
    g = torch.Generator(device="cuda").manual_seed(m)
    x, wg, wu, dh = (torch.randn(s, generator=g, device="cuda").to(DTYPES[dtype]) for s in ((m, c), (f, c), (f, c), (m, f)))
    wg, wu = wg * c ** -0.5, wu * c ** -0.5
    own = wt.wtconv_gated_backward(x, dh, wg, wu)
    wide = wt.wtconv_gated_backward(x, dh, wg, wu, dw_dtype=torch.float32)
    assert wide[1].dtype == wide[2].dtype == torch.float32 and wide[0].dtype == x.dtype
    for a, b in zip(own, wide):
        assert torch.equal(a, b.to(a.dtype))
    given = [torch.full((f, c), 7.0, device="cuda") for _ in range(2)]
    out = wt.wtconv_gated_backward(x, dh, wg, wu, dw_gate=given[0], dw_up=given[1], dw_dtype=torch.float32,
                                   need=(False, True, False))
    assert out[1] is given[0] and out[2] is given[1] and out[0] is None
    assert torch.equal(given[0], wide[1]) and torch.equal(given[1], wide[2])


def test_types_are_checked():
    x, w, dh = torch.randn(9, 8, device="cuda").half(), torch.randn(6, 8, device="cuda").half(), torch.randn(9, 6).cuda().half()
    for bad in (torch.bfloat16, torch.float64):
        with pytest.raises(ValueError, match="dw_dtype"):
            wt.wtconv_gated_backward(x, dh, w, w, dw_dtype=bad)
    with pytest.raises(TypeError, match="dw_gate"):
        wt.wtconv_gated_backward(x, dh, w, w, dw_gate=torch.empty_like(w), dw_dtype=torch.float32)
    with pytest.raises(TypeError, match="dw_up"):
        wt.wtconv_gated_backward(x, dh, w, w, dw_up=torch.empty(6, 8, device="cuda"))


def test_captured_module():
    """Replays of a captured backward pass with float32 parameters under fp16."""
    torch.manual_seed(0)
    layer = GatedLinear(32, 48, device="cuda")
    x, a = torch.randn(200, 32, device="cuda").half(), torch.randn(200, 48, device="cuda").half()
    params = list(layer.parameters())

    def step():
        return torch.autograd.grad(layer(x), params, a)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(4):
        x.mul_(-0.9)
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))


def test_weights_of_two_types():
    """Each weight's gradient comes back in its own type, from the float32 sums."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, wg, wu, a = (torch.randn(s, generator=g, device="cuda").half() for s in ((90, 24), (40, 24), (40, 24), (90, 40)))
    wide = wt.wtconv_gated_backward(x, a, wg, wu, dw_dtype=torch.float32)
    for types in ((torch.float32, torch.float16), (torch.float16, torch.float64), (torch.bfloat16, torch.bfloat16)):
        w = [t.clone().to(d) for t, d in zip((wg, wu), types)]
        if torch.bfloat16 in types:
            wide = wt.wtconv_gated_backward(x, a, *(t.half() for t in w), dw_dtype=torch.float32)
        for t in w:
            t.requires_grad_()
        GatedFunction.apply(x, *w, None, None, "silu").backward(a)
        for t, ref in zip(w, wide[1:3]):
            assert t.grad.dtype == t.dtype and torch.equal(t.grad, ref.to(t.dtype))


def test_entry_point_in_fp32():
    """The C call with fp32 gradients and fp32 activations is the other one."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x, wg, wu, dh = (torch.randn(s, generator=g, device="cuda") for s in ((130, 33), (65, 33), (65, 33), (130, 65)))
    want = wt.wtconv_gated_backward(x, dh, wg, wu, act="gelu")
    got = [torch.empty_like(t) for t in want]
    n = wt.wtconv_gated_workspace_size(x.shape, 65, _native.F32, _native.OP_BWD)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    d = _native.GatedDesc(130, 33, 65, _native.F32, _native.ACTS["gelu"])
    st = _native.load().wtconv_gated_backward_f32_grads(
        ctypes.byref(d), x.data_ptr(), dh.data_ptr(), wg.data_ptr(), wu.data_ptr(), None, None,
        *(t.data_ptr() for t in got), work.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
