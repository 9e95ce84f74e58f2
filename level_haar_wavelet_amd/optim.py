"""The Muon optimiser over libwtconv: every update is the momentum of the
gradient, orthogonalised by the Newton-Schulz iteration (wtconv_muon_step).

It is for parameters that are matrices: the layer's convolution weights and the
products next to it.  A parameter of shape (*batch, rows, *rest) is a stack of
matrices of rows x prod(rest):
    WTConv2d.w_base (C, k, k)       one matrix of C x k^2,
    WTConv2d.w_lvl  (L, 4C, k, k)   L matrices of 4C x k^2,
    a product's weight (out, in)    itself.
`batch_dims` says how many leading dimensions are the stack's; by default none,
and one for WTConv2d.w_lvl.  Other 4-d parameters need it: 0 for the (out, in,
k, k) weight of an ordinary convolution, 1 for a stack laid out as w_lvl is (a
parameter whose attribute `matrix_batch_dims` is 1 counts as one by itself).
Biases and the scales s_base and s_lvl are no matrices in that sense: leave them
to another optimiser.
"""
from __future__ import annotations

import math

import torch

from . import _native, _train, wtconv_muon_step

__all__ = ["Muon"]


def _matrices(shape, batch_dims):
    """(batch, rows, cols) of a parameter's shape."""
    if batch_dims is None:
        batch_dims = 1 if len(shape) == 4 else 0
    if batch_dims < 0 or len(shape) < batch_dims + 2 or 0 in shape:
        raise ValueError("Muon takes matrices: shape %s has none behind %d batch dimensions" % (tuple(shape),
                                                                                               batch_dims))
    return math.prod(shape[:batch_dims]), shape[batch_dims], math.prod(shape[batch_dims + 1:])


def _matrices_of(p, batch_dims):
    """The same of a parameter.  Nothing in a 4-d shape tells a convolution's
    weight from a stack, and each taken for the other is updated wrongly."""
    if batch_dims is None and p.dim() == 4:
        batch_dims = getattr(p, "matrix_batch_dims", None)
        if batch_dims is None:
            raise ValueError("a parameter of shape %s needs batch_dims: 0 for a convolution's weight (out, in, k, k), "
                             "1 for a stack of matrices (L, rows, k, k)" % (tuple(p.shape),))
    return _matrices(p.shape, batch_dims)


class Muon(torch.optim.Optimizer):
    """momentum <- mu momentum + (1 - mu) grad; u = mu momentum + (1 - mu) grad
    (nesterov) or momentum; weight <- (1 - lr weight_decay) weight - lr s O(u),
    with O the Newton-Schulz iteration of `steps` steps and
    s = sqrt(max(1, rows / cols)).  Parameters are contiguous float32 tensors on
    the GPU.  The hyperparameters go by value: a step captured into a graph
    replays with those it was captured with, and only after a step outside one
    (the momentum's zeros would be part of the graph)."""

    def __init__(self, params, lr=0.02, momentum=0.95, weight_decay=0.0, nesterov=True, steps=5, eps=1e-7,
                 batch_dims=None):
        super().__init__(params, dict(lr=lr, momentum=momentum, weight_decay=weight_decay, nesterov=nesterov,
                                      steps=steps, eps=eps, batch_dims=batch_dims))

    def add_param_group(self, group):
        super().add_param_group(group)
        group = self.param_groups[-1]
        try:
            if not group["lr"] >= 0 or not group["weight_decay"] >= 0 or not 0 <= group["momentum"] < 1:
                raise ValueError("lr and weight_decay must be >= 0 and momentum in [0, 1)")
            if not 1 <= group["steps"] <= 16 or not 0 <= group["eps"] < math.inf:
                raise ValueError("steps must be 1 to 16 and eps >= 0 and finite")
            for p in group["params"]:
                _matrices_of(p, group["batch_dims"])
                if p.dtype != torch.float32:
                    raise TypeError("Muon takes float32 parameters, got %s" % p.dtype)
        except (TypeError, ValueError):
            self.param_groups.pop()
            raise

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        # everything is checked before the first update
        todo = []
        for group in self.param_groups:
            for p in group["params"]:
                if p.grad is None:
                    continue
                shape = _matrices_of(p, group["batch_dims"])
                if not p.is_contiguous():
                    raise TypeError("Muon takes contiguous parameters")
                if not p.is_cuda:
                    raise TypeError("Muon takes parameters on the GPU")
                # the step's own plan: sizes, steps and eps that the call would refuse
                _train._ortho_plan(*shape, _native.F32, int(group["steps"]), float(group["eps"]))
                if "momentum_buffer" not in self.state.get(p, ()) and torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("the first step of a parameter cannot be captured: every replay would "
                                       "start from a momentum of zero")
                todo.append((group, p, shape))
        for group, p, shape in todo:
            state = self.state[p]
            if "momentum_buffer" not in state:
                state["momentum_buffer"] = torch.zeros_like(p)
            wtconv_muon_step(p.view(shape), p.grad.contiguous().view(shape), state["momentum_buffer"].view(shape),
                             lr=group["lr"], mu=group["momentum"], weight_decay=group["weight_decay"],
                             scale=math.sqrt(max(1.0, shape[1] / shape[2])), nesterov=group["nesterov"],
                             steps=group["steps"], eps=group["eps"])
        return loss
