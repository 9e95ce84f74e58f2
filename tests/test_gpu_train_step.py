"""The operators together, as a training step of a block uses them: the WTConv
layer, the group norm with its activation written channels last, a product over
the channels, the backward pass of all, and the Muon update."""
import math

import numpy as np
import pytest
import torch

from level_haar_wavelet_amd.synthetic import make_inputs
from tests.train_util import Norm64, ortho64

pytestmark = pytest.mark.gpu

N, C, H, W, K, L, GROUPS, OUT = 3, 12, 20, 28, 5, 2, 4, 24


def build():
    from level_haar_wavelet_amd.module import GroupNormAct2d, WTConv2d

    torch.manual_seed(1)
    conv = WTConv2d(C, K, L, device="cuda")
    norm = GroupNormAct2d(GROUPS, C, act="gelu", channels_last=True, device="cuda")
    lin = torch.nn.Linear(C, OUT, bias=False, device="cuda")
    return conv, norm, lin


def forward(conv, norm, lin, x):
    y = norm(conv(x))
    assert y.is_contiguous(memory_format=torch.channels_last)
    return lin(y.permute(0, 2, 3, 1))  # (N, H, W, OUT), no copy


def test_training_step_against_fp64(orc):
    from level_haar_wavelet_amd.optim import Muon

    conv, norm, lin = build()
    inp = make_inputs(N, C, H, W, K, L, seed=3)
    x = torch.from_numpy(inp.x).cuda().requires_grad_()
    tgt = torch.randn(N, H, W, OUT, generator=torch.Generator().manual_seed(4))
    muon = Muon([conv.w_base, conv.w_lvl, lin.weight], lr=0.05)
    before = [p.detach().cpu().clone() for p in (conv.w_base, conv.w_lvl, lin.weight)]
    out = forward(conv, norm, lin, x)
    loss = (out - tgt.cuda()).square().sum()
    loss.backward()
    grads = [p.grad.clone() for p in (conv.w_base, conv.w_lvl, lin.weight)]
    muon.step()

    # the same step in fp64: the layer by the oracle, the rest by formulas
    f64 = lambda p: p.detach().cpu().double()
    p = [f64(t).numpy() for t in (conv.s_base, conv.s_lvl)]
    wb, wl = (b.double().numpy() for b in before[:2])
    bias = f64(conv.bias).numpy()
    x64 = inp.x.astype(np.float64)
    a = torch.from_numpy(orc.forward(x64, wb, bias, p[0], wl, p[1], K, L))
    ref = Norm64(a, GROUPS, f64(norm.gamma), f64(norm.beta), norm.eps, "gelu")
    rows = ref.y.permute(0, 2, 3, 1).reshape(-1, C)
    lw = before[2].double()
    o64 = rows @ lw.T
    d = 2 * (o64 - tgt.double().view(-1, OUT))
    dy = (d @ lw).view(N, H, W, C).permute(0, 3, 1, 2)
    dx1, dgamma, dbeta = ref.backward(dy)
    dx = orc.backward_data(dx1.contiguous().numpy(), wb, p[0], wl, p[1], K, L)
    dw = orc.backward_weight(x64, dx1.contiguous().numpy(), wb, bias, p[0], wl, p[1], K, L)

    def close(got, want, what):
        want = torch.as_tensor(want)
        err = (got.detach().cpu().double() - want).norm() / want.norm()
        assert err <= 1e-4, (what, float(err))  # the layer's own tolerance of fp32 gradients

    close(out.view(-1, OUT), o64, "out")
    close(x.grad, dx, "dx")
    close(norm.gamma.grad, dgamma, "dgamma")
    close(norm.beta.grad, dbeta, "dbeta")
    close(conv.w_base.grad, dw[0], "dw_base")
    close(conv.s_base.grad, dw[2], "ds_base")
    close(conv.w_lvl.grad, dw[3], "dw_lvl")
    close(conv.s_lvl.grad, dw[4], "ds_lvl")
    close(lin.weight.grad, d.T @ rows, "dlin")
    # bias of the layer: a shift of a channel, not of its group
    # the update, from the gradients that the step saw
    for param, old, g, shape in zip((conv.w_base, conv.w_lvl, lin.weight), before, grads,
                                    ((1, C, K * K), (L, 4 * C, K * K), (1, OUT, C))):
        o = ortho64(g.cpu().view(shape))
        want = old.double().view(shape) - 0.05 * math.sqrt(max(1, shape[1] / shape[2])) * o
        close(param.view(shape), want, "update")


def test_captured_training_step_replays():
    """Forward, backward and update in one graph, replayed on new inputs between
    eager steps of a second copy.  The gradients of the captured step are its
    own: no eager backward pass of these leaves is alive at the capture."""
    from level_haar_wavelet_amd.optim import Muon

    sides = []
    for _ in range(2):
        mods = build()
        params = [mods[0].w_base, mods[0].w_lvl, mods[2].weight]
        for m in mods:
            for q in m.parameters():
                q.requires_grad_(any(q is t for t in params))
        opt = Muon(params, lr=0.05, weight_decay=0.1)
        for q in params:
            opt.state[q]["momentum_buffer"] = torch.zeros_like(q)
        sides.append((mods, params, opt, torch.zeros(N, C, H, W, device="cuda")))

    def step(side):
        mods, params, opt, x = side
        out = forward(*mods, x).square().mean()
        for q, g in zip(params, torch.autograd.grad(out, params)):
            q.grad = g
        opt.step()
        return out.detach()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    keep = [t.detach().clone() for t in sides[0][1]]
    with torch.cuda.stream(s):
        sides[0][3].normal_()
        step(sides[0])
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step(sides[0])
    with torch.no_grad():
        for q, t in zip(sides[0][1], keep):
            q.copy_(t)
            sides[0][2].state[q]["momentum_buffer"].zero_()
    for r in range(4):
        x = torch.randn(N, C, H, W, generator=torch.Generator().manual_seed(r)).cuda()
        for side in sides:
            side[3].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        want = step(sides[1])
        torch.cuda.synchronize()
        assert torch.allclose(loss, want, rtol=1e-6)
        for p, q in zip(sides[0][1], sides[1][1]):
            assert torch.allclose(p, q, rtol=1e-5, atol=1e-6), r


def test_autograd_sees_the_update_of_saved_weights():
    """A backward pass through weights that a step has changed since the forward
    pass is refused, as after any optimiser of torch."""
    from level_haar_wavelet_amd.optim import Muon

    for pick in (lambda m: [m[0].w_base], lambda m: [m[0].w_lvl], lambda m: [m[2].weight]):
        mods = build()
        params = pick(mods)
        x = torch.randn(N, C, H, W, device="cuda", requires_grad=True)
        opt = Muon(params, lr=0.1)
        loss = forward(*mods, x).square().mean()
        loss.backward(retain_graph=True)
        opt.step()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        forward(*mods, x).square().mean().backward()  # a graph recorded after it is fine


def test_versions_of_the_tensors_a_call_writes_into():
    """Every tensor of the caller's that a call writes counts as modified, once
    the call is accepted; its inputs do not."""
    import level_haar_wavelet_amd as wt

    def changes(call, written, read):
        before = [t._version for t in written + read]
        call()
        after = [t._version for t in written + read]
        assert all(a > b for a, b in zip(after[:len(written)], before))
        assert after[len(written):] == before[len(written):]

    x, y, dx = (torch.randn(2, 8, 6, 6, device="cuda") for _ in range(3))
    mean, rstd = (torch.ones(2, 4, device="cuda") for _ in range(2))
    gamma, beta, dg, db = (torch.ones(8, device="cuda") for _ in range(4))
    changes(lambda: wt.wtconv_group_norm_forward(x, 4, gamma, beta, y=y, mean=mean, rstd=rstd), [y, mean, rstd],
            [x, gamma, beta])
    changes(lambda: wt.wtconv_group_norm_backward(x, y, 4, mean, rstd, gamma, beta, dx=dx, dgamma=dg, dbeta=db),
            [dx, dg, db], [x, y, mean, rstd, gamma, beta])
    g, w, m, wo, mo, out = (torch.randn(12, 20, device="cuda") for _ in range(6))
    changes(lambda: wt.wtconv_orthogonalize(g, out=out), [out], [g])
    changes(lambda: wt.wtconv_muon_step(w, g, m, lr=0.1, weight_out=wo, momentum_out=mo), [wo, mo], [w, g, m])
    changes(lambda: wt.wtconv_muon_step(w, g, m, lr=0.1), [w, m], [g])
    changes(lambda: wt.wtconv_muon_step(w, g, m, lr=0.1, stream=torch.cuda.Stream()), [w, m], [g])
    torch.cuda.synchronize()

    def refused():
        with pytest.raises(wt._native.WtconvError):
            wt.wtconv_muon_step(w, g, m, lr=0.1, steps=0)
        with pytest.raises(wt._native.WtconvError):
            wt.wtconv_orthogonalize(g, out=g)

    changes(refused, [], [w, g, m])
    with torch.inference_mode():  # such tensors have no counter
        u = torch.randn(12, 20, device="cuda")
        wt.wtconv_muon_step(u, g, torch.zeros_like(u), lr=0.1)
