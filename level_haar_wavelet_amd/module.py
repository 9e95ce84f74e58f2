"""PyTorch autograd wrapper and nn.Module over libwtconv.

The layer (the depthwise base convolution with bias and scale, plus L levels of
orthonormal Haar analysis, per-level depthwise convolutions over the 4C
subbands with per-band scales, and the synthesis cascade) is the one described
in "Fast and Memory-Efficient Wavelet Convolutions via I/O-Aware
Reformulation" (arXiv 2608.10805), technical summary, Methodology, and the
WTConv layer it reformulates.  Forward, data backward and parameter gradients
all run in libwtconv's kernels (wtconv_forward, wtconv_backward_data,
wtconv_backward_weight); this module only hands tensors to them.  The layer
saves only its input for the backward pass.

GroupNormAct2d is the normalisation and activation that follow the layer in a
block, in the same manner.
"""
from __future__ import annotations

import math

import torch

from . import _native
from . import (wtconv_backward_data, wtconv_backward_weight, wtconv_forward, wtconv_group_norm_backward,
               wtconv_group_norm_forward)

__all__ = ["WTConvFunction", "WTConv2d", "GroupNormActFunction", "GroupNormAct2d"]


class WTConvFunction(torch.autograd.Function):
    """y = WTConv(x; w_base, bias, s_base, w_lvl, s_lvl).

    x: (N, C, H, W) float32 or float16, contiguous, on the GPU (sides 2^L
    does not divide: odd level maps zero-padded at the bottom / right, each
    level's synthesis cropped back).  Parameters are float32: w_base (C, k, k), bias (C,) or
    None, s_base (C,), w_lvl (L, 4C, k, k) and s_lvl (L, 4C), or None for
    both when L = 0.
    """

    @staticmethod
    def forward(ctx, x, w_base, bias, s_base, w_lvl, s_lvl):
        x = x.contiguous()
        y = wtconv_forward(x, w_base, bias, s_base, w_lvl, s_lvl)
        ctx.save_for_backward(x, w_base, bias, s_base, w_lvl, s_lvl)
        ctx.has_bias = bias is not None
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w_base, bias, s_base, w_lvl, s_lvl = ctx.saved_tensors
        dy = dy.contiguous().to(x.dtype)
        need = ctx.needs_input_grad
        dx = wtconv_backward_data(dy, w_base, s_base, w_lvl, s_lvl) if need[0] else None
        dw0 = db0 = ds0 = dwl = dsl = None
        if any(need[1:]):
            dw0, db0, ds0, dwl, dsl = wtconv_backward_weight(x, dy, w_base, bias, s_base, w_lvl, s_lvl)
        return (dx, dw0 if need[1] else None, db0 if (ctx.has_bias and need[2]) else None,
                ds0 if need[3] else None, dwl if need[4] else None, dsl if need[5] else None)


class WTConv2d(torch.nn.Module):
    """Drop-in WTConv layer: a depthwise k x k convolution with an L-level
    Haar wavelet branch (same channels in and out, stride 1, 'same' padding).

    Initialisation: weights N(0, 0.05^2), bias zero, base scale 1 and
    level scales 0.1 (the wavelet branch starts small next to the base
    convolution).
    """

    def __init__(self, channels: int, kernel_size: int = 5, levels: int = 1, bias: bool = True,
                 device=None):
        super().__init__()
        if kernel_size not in (1, 3, 5, 7):
            raise ValueError("kernel_size must be 1, 3, 5 or 7")
        if levels < 0:
            raise ValueError("levels must be >= 0")
        c, k = channels, kernel_size
        f = dict(device=device, dtype=torch.float32)
        self.channels, self.kernel_size, self.levels = c, k, levels
        self.w_base = torch.nn.Parameter(torch.randn(c, k, k, **f) * 0.05)
        self.bias = torch.nn.Parameter(torch.zeros(c, **f)) if bias else None
        self.s_base = torch.nn.Parameter(torch.ones(c, **f))
        if levels > 0:
            self.w_lvl = torch.nn.Parameter(torch.randn(levels, 4 * c, k, k, **f) * 0.05)
            self.s_lvl = torch.nn.Parameter(torch.full((levels, 4 * c), 0.1, **f))
        else:
            self.register_parameter("w_lvl", None)
            self.register_parameter("s_lvl", None)
        self._mark_matrices()

    def _mark_matrices(self):
        # for optim.Muon: the first dimension counts matrices
        if self.w_lvl is not None:
            self.w_lvl.matrix_batch_dims = 1

    def __setstate__(self, state):  # a copied parameter is a new one
        super().__setstate__(state)
        self._mark_matrices()

    def forward(self, x):
        return WTConvFunction.apply(x, self.w_base, self.bias, self.s_base, self.w_lvl, self.s_lvl)

    def extra_repr(self):
        return "channels=%d, kernel_size=%d, levels=%d, bias=%s" % (self.channels, self.kernel_size, self.levels,
                                                                   self.bias is not None)


class GroupNormActFunction(torch.autograd.Function):
    """y = act(group_norm(x)) (wtconv_group_norm_forward / _backward).

    x: (N, C, H, W) float32, float16 or bfloat16 on the GPU, contiguous or
    channels last (other strides are made contiguous); gamma, beta: (C,)
    float32 or None; channels_last: the layout of y (None: x's).  Saves x and the
    groups' mean and rstd."""

    @staticmethod
    def forward(ctx, x, gamma, beta, groups, eps, act, channels_last):
        if not (x.is_contiguous() or x.is_contiguous(memory_format=torch.channels_last)):
            x = x.contiguous()
        y, mean, rstd = wtconv_group_norm_forward(x, groups, gamma, beta, eps=eps, act=act,
                                                  channels_last=channels_last)
        ctx.save_for_backward(x, gamma, beta, mean, rstd)
        ctx.groups, ctx.act = groups, act
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, gamma, beta, mean, rstd = ctx.saved_tensors
        dy = dy.to(x.dtype)
        if not (dy.is_contiguous() or dy.is_contiguous(memory_format=torch.channels_last)):
            dy = dy.contiguous()
        dx, dgamma, dbeta = wtconv_group_norm_backward(x, dy, ctx.groups, mean, rstd, gamma, beta, act=ctx.act)
        need = ctx.needs_input_grad
        return (dx if need[0] else None, dgamma if need[1] else None, dbeta if need[2] else None, None, None, None,
                None)


class GroupNormAct2d(torch.nn.Module):
    """Group norm with its activation, as it follows a WTConv2d: `groups`
    groups of neighbouring channels, act "none", "relu", "silu" or "gelu".
    channels_last=True writes the output channels last whatever the input's
    layout is (what a product over the channels reads); None keeps the input's.
    Initialisation: gamma one, beta zero (none with affine=False).  Both stay
    float32, whatever the input's type; an empty batch is refused.
    """

    def __init__(self, groups: int, channels: int, eps: float = 1e-5, act: str = "none", affine: bool = True,
                 channels_last=None, device=None):
        super().__init__()
        if groups < 1 or channels % groups:
            raise ValueError("groups must divide channels")
        if act not in _native.ACTS:
            raise ValueError("act must be one of %s, got %r" % (", ".join(sorted(_native.ACTS)), act))
        if not 0 < eps < math.inf:
            raise ValueError("eps must be positive and finite")
        f = dict(device=device, dtype=torch.float32)
        self.groups, self.channels, self.eps, self.act, self.channels_last = groups, channels, eps, act, channels_last
        if affine:
            self.gamma = torch.nn.Parameter(torch.ones(channels, **f))
            self.beta = torch.nn.Parameter(torch.zeros(channels, **f))
        else:
            self.register_parameter("gamma", None)
            self.register_parameter("beta", None)

    def forward(self, x):
        if x.dim() != 4 or x.shape[1] != self.channels:
            raise ValueError("expected (N, C, H, W) with C = %d channels, got %s" % (self.channels, tuple(x.shape)))
        return GroupNormActFunction.apply(x, self.gamma, self.beta, self.groups, self.eps, self.act,
                                          self.channels_last)

    def extra_repr(self):
        return "groups=%d, channels=%d, eps=%g, act=%s, affine=%s, channels_last=%s" % (
            self.groups, self.channels, self.eps, self.act, self.gamma is not None, self.channels_last)
