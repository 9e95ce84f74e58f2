"""Gradient norm and clipping on the GPU against fp64."""
import math

import pytest
import torch

import level_haar_wavelet_amd as wt
from level_haar_wavelet_amd import _native
from level_haar_wavelet_amd.optim import clip_grad_norm_
from tests.block_util import DTYPES, U, check, half_step

pytestmark = pytest.mark.gpu


def make(sizes, types, seed=0, offset=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.empty(n + offset, dtype=DTYPES[types[i % len(types)]], device="cuda")[offset:]
        t.copy_(scale * 10.0 ** (i % 4 - 2) * torch.randn(n, generator=g))
        out.append(t)
    return out


def norm64(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


def scaled(grads, norm, max_norm, eps=1e-6):
    return [g.double() * min(1.0, max_norm / (norm + eps)) for g in grads]


def check_all(got, ref):
    for i, (a, b) in enumerate(zip(got, ref)):
        # the factor, the product and the output are rounded once each
        check("tensor %d" % i, a, b, 3 * U * b.abs() + half_step(b, a.dtype) + 2.0 ** -149)


LISTS = {
    "one": [1], "small": [1, 7, 8, 9, 255, 256, 257], "ragged": [2047, 2048, 2049, 8191, 8192, 8193, 100003],
    "empty among": [0, 5, 0, 0, 9000, 0], "many": [1 + 37 * i % 3001 for i in range(500)], "large": [20000003, 33],
    "more ranges than a workgroup joins": [3] * 4200,
}


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("types", [("f32",), ("f16",), ("bf16",), ("f32", "bf16", "f16")], ids="-".join)
@pytest.mark.parametrize("name", LISTS)
def test_norm_and_clip(name, types, offset):
    grads = make(LISTS[name], types, offset=offset)
    n = norm64(grads)
    assert float(wt.wtconv_grad_norm(grads)) == pytest.approx(n, rel=2 * U)
    keep = [g.clone() for g in grads]
    for max_norm in (0.37 * n, 2.0 * n):
        out = [torch.empty_like(g) for g in grads]
        norm, back = wt.wtconv_clip_grad_norm(grads, max_norm, out=out)
        assert back == out or all(a is b for a, b in zip(back, out))
        assert norm.shape == () and float(norm) == pytest.approx(n, rel=2 * U)
        check_all(out, scaled(grads, n, max_norm))
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    wt.wtconv_clip_grad_norm(grads, 2.0 * n)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    wt.wtconv_clip_grad_norm(grads, 0.37 * n)
    check_all(grads, scaled(keep, n, 0.37 * n))


def test_beyond_2_31_elements():
    g = torch.randn(1 << 20, device="cuda").bfloat16()
    big = [g.repeat(2200), torch.randn(1000, device="cuda")]
    n = math.sqrt(2200 * norm64([g]) ** 2 + norm64(big[1:]) ** 2)
    norm, _ = wt.wtconv_clip_grad_norm(big, 1.0)
    assert float(norm) == pytest.approx(n, rel=2 * U)
    small = (g.float() * (1.0 / (n + 1e-6))).bfloat16()
    diff = (big[0].view(2200, -1).float() - small.float()).abs()
    assert bool((diff <= torch.finfo(torch.bfloat16).eps * small.float().abs()).all())


def test_no_tensors():
    norm, out = wt.wtconv_clip_grad_norm([], 1.0)
    assert float(norm) == 0 and out == [] and float(wt.wtconv_grad_norm([])) == 0
    assert float(wt.wtconv_grad_norm([torch.empty(0, device="cuda")])) == 0


def test_values():
    """fp32's range of values has no effect on the sum; NaN and infinity come through."""
    for scale in (1e-30, 1e30):
        g = make([1000], ("f32",), scale=100 * scale)
        assert float(wt.wtconv_grad_norm(g)) == pytest.approx(norm64(g), rel=2 * U)
        wt.wtconv_clip_grad_norm(g, scale, eps=0.0)
        assert norm64(g) == pytest.approx(scale, rel=1e-6)
    huge = [torch.full((4096,), 3e38, device="cuda")]
    norm, _ = wt.wtconv_clip_grad_norm(huge, 1.0)
    assert math.isinf(float(norm)) and norm64(huge) == pytest.approx(1.0, rel=1e-6)
    a, b = torch.randn(50, device="cuda"), torch.randn(60, device="cuda")
    a[3] = float("inf")
    norm, _ = wt.wtconv_clip_grad_norm([a, b], 1.0)
    assert math.isinf(float(norm)) and bool((b == 0).all()) and bool(a[3].isnan()) and bool((a[:3] == 0).all())
    a, b = torch.randn(50, device="cuda"), torch.randn(60, device="cuda")
    a[3] = float("nan")
    norm, _ = wt.wtconv_clip_grad_norm([a, b], 1.0)
    assert math.isnan(float(norm)) and bool(a.isnan().all()) and bool(b.isnan().all())
    z = [torch.zeros(9, device="cuda")]
    norm, _ = wt.wtconv_clip_grad_norm(z, 1.0, eps=0.0)
    assert float(norm) == 0 and bool((z[0] == 0).all())
    g = [torch.randn(9, device="cuda")]
    wt.wtconv_clip_grad_norm(g, 0.0)
    assert bool((g[0] == 0).all())


def test_repeats_and_overlaps():
    g = torch.randn(100, device="cuda")
    assert float(wt.wtconv_grad_norm([g, g])) == pytest.approx(math.sqrt(2) * norm64([g]), rel=1e-6)
    for grads, out in (([g, g], None), ([g, g[50:]], None), ([g[:60]], [g[10:70]]),
                       ([g[:50], g[50:]], [g[50:], g[:50]])):
        with pytest.raises(_native.WtconvError, match="ALIAS"):
            wt.wtconv_clip_grad_norm(grads, 1.0, out=out)
    # neighbours in one buffer are apart
    keep = g.clone()
    wt.wtconv_clip_grad_norm([g[50:], g[:50]], 0.5)
    check_all([g], scaled([keep], norm64([keep]), 0.5))


def test_captured():
    """Replays of a captured call follow the gradients' values, beside another captured call."""
    grads, others = make([5000, 33, 100000], ("f32", "bf16")), make([77, 20000], ("f16",), seed=2)
    out, out2 = [torch.empty_like(g) for g in grads], [torch.empty_like(g) for g in others]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        wt.wtconv_clip_grad_norm(grads, 1.0, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        n1, _ = wt.wtconv_clip_grad_norm(grads, 1.0, out=out)
    with torch.cuda.graph(graphs[1]):
        n2, _ = wt.wtconv_clip_grad_norm(others, 0.5, out=out2)
    for i in range(4):
        for g in grads + others:
            g.mul_(1.5)
        for graph in graphs:
            graph.replay()
        eager = [wt.wtconv_grad_norm(grads), wt.wtconv_grad_norm(others)]
        torch.cuda.synchronize()
        assert torch.equal(n1, eager[0]) and torch.equal(n2, eager[1])
        check_all(out, scaled(grads, norm64(grads), 1.0))
        check_all(out2, scaled(others, norm64(others), 0.5))


def test_parameters():
    torch.manual_seed(0)
    params = [torch.nn.Parameter(torch.randn(s, device="cuda")) for s in ((3, 4), (5,), (2, 2), (6, 8))]
    params[0].grad, params[1].grad = torch.randn(3, 4, device="cuda"), torch.randn(5, device="cuda")
    params[3].grad = torch.randn(8, 6, device="cuda").t()  # strided
    keep = [p.grad.clone() for p in params if p.grad is not None]
    n = norm64(keep)
    norm = clip_grad_norm_(iter(params + [params[0]]), 0.7)
    assert float(norm) == pytest.approx(n, rel=2 * U) and params[2].grad is None
    check_all([p.grad for p in params if p.grad is not None], scaled(keep, n, 0.7))
    assert float(clip_grad_norm_(params[1], 1e9)) == pytest.approx(norm64([params[1].grad]), rel=2 * U)
    assert float(clip_grad_norm_([params[2]], 1.0)) == 0
    # a graph that saved a gradient notices
    w = torch.randn(5, device="cuda", requires_grad=True)
    loss = (w * params[1].grad).sum()
    clip_grad_norm_([params[1]], 0.1)
    with pytest.raises(RuntimeError, match="modified"):
        loss.backward()
