"""Binding of the operators around the layer in a training step: the group norm
with its activation, and the Newton-Schulz orthogonalisation and Muon step of
the weights' update.  Argument checks and marshalling only; the functions carry
the names of the C entry points in include/wtconv.h and are re-exported by the
package.

A call is enqueued on `stream`, or on the current stream of the device that its
tensors lie on; that device need not be the current one.  Its buffers are the
caller's: a tensor that was made on another stream needs that stream's own
ordering (torch.cuda.Stream.wait_stream, Tensor.record_stream), as with any
torch operation.  Those that it writes count as modified for autograd: a
backward pass that saved one of them raises instead of reading the new values.
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.graph import increment_version

from . import _native

_DTYPES = {torch.float32: _native.F32, torch.float16: _native.F16, torch.bfloat16: _native.BF16}
_F32 = torch.float32
_Tensor = torch.Tensor


def _dtype_code(t, name):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be float32, float16 or bfloat16, got %s" % (name, t.dtype))
    return code


def _ptr(t):
    return None if t is None else t.data_ptr()


def _gpu_tensor(t, name, device=None):
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError("%s must be a GPU tensor" % name)
    if device is not None and t.device != device:
        raise TypeError("%s lies on %s, the other tensors on %s" % (name, t.device, device))


def _f32(t, name, shape, device):
    if t is None:
        return
    if not isinstance(t, _Tensor) or t.dtype is not _F32 or t.shape != shape or t.device != device or \
            not t.is_contiguous():
        _gpu_tensor(t, name, device)
        raise TypeError("%s must be a contiguous float32 tensor of shape %s" % (name, tuple(shape)))


def _workspace(workspace, need, device):
    """The caller's workspace, or a new one; (tensor or None, bytes)."""
    if workspace is None:
        if need == 0:
            return None, 0
        return torch.empty(need, dtype=torch.uint8, device=device), need
    _gpu_tensor(workspace, "workspace", device)
    if not workspace.is_contiguous():
        raise TypeError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def _written(*tensors):
    """The kernels write through addresses, which torch does not see."""
    given = [t for t in tensors if t is not None]
    if given:
        increment_version(given)


class _On:
    """The device of the tensors as the current one, and the stream's handle.
    What a call with a stream of its own allocates comes from that stream's pool
    (a block of the current stream's may still be in use there, and the call
    does not wait for it); `made` marks the results as used on the current
    stream too, which their caller is likely to read them on."""

    __slots__ = ("handle", "guard", "current")

    def __init__(self, device, stream):
        cuda = torch.cuda
        self.current = None
        self.guard = None if cuda.current_device() == device.index else cuda.device(device)
        if stream is None:
            # the current stream's handle without a Stream object (2 us less)
            self.handle = torch._C._cuda_getCurrentRawStream(device.index)
        elif stream.device != device:
            raise TypeError("the stream belongs to %s, the tensors lie on %s" % (stream.device, device))
        else:
            self.handle = stream.cuda_stream
            self.current = cuda.current_stream(device)
            self.guard = cuda.stream(stream)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def made(self, *tensors):
        if self.current is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.current)


# ---- group norm --------------------------------------------------------------

def _layout_of(t, name):
    """WTCONV_NCHW or WTCONV_NHWC of a 4-d tensor without gaps."""
    if t.dim() != 4:
        raise TypeError("%s must be an (N, C, H, W) tensor" % name)
    if t.is_contiguous():
        return _native.NCHW
    if t.is_contiguous(memory_format=torch.channels_last):
        return _native.NHWC
    raise TypeError("%s must be contiguous or channels_last" % name)


def _one_layout(t):
    """Whether planes and channels last are the same order for this shape."""
    return t.shape[1] == 1 or t.shape[2] * t.shape[3] == 1


def _like(t, layout):
    fmt = torch.channels_last if layout == _native.NHWC else torch.contiguous_format
    return torch.empty_like(t, memory_format=fmt)


@functools.lru_cache(maxsize=512)
def _norm_plan(op, n, c, h, w, groups, dtype, act, x_layout, y_layout, eps):
    """The descriptor of these sizes (as ctypes takes it) and op's workspace."""
    if act not in _native.ACTS:
        raise ValueError("act must be one of %s, got %r" % (", ".join(sorted(_native.ACTS)), act))
    d = _native.NormDesc(n, c, h, w, groups, dtype, _native.ACTS[act], x_layout, y_layout, eps)
    out = ctypes.c_size_t(0)
    _native.check(_native.load().wtconv_group_norm_workspace_size(ctypes.byref(d), op, ctypes.byref(out)),
                  "wtconv_group_norm_workspace_size")
    return ctypes.byref(d), out.value


def wtconv_group_norm_workspace_size(shape, groups, dtype_code, op, x_layout=_native.NCHW, y_layout=_native.NCHW,
                                     act="none") -> int:
    """Bytes of workspace of the forward (OP_FWD) or backward (OP_BWD) call."""
    n, c, h, w = shape
    return _norm_plan(op, n, c, h, w, groups, dtype_code, act, x_layout, y_layout, 1e-5)[1]


def wtconv_group_norm_forward(x, groups, gamma=None, beta=None, eps=1e-5, act="none", channels_last=None, y=None,
                              mean=None, rstd=None, workspace=None, stream=None):
    """(y, mean, rstd) of y = act(gamma (x - mean) rstd + beta), the statistics
    over the C / groups channels and the H x W pixels of a group.

    x is (N, C, H, W) float32, float16 or bfloat16, contiguous or channels
    last; y comes in the same layout, or channels last / contiguous where
    `channels_last` is True / False (or in the layout of `y`, if given).  gamma,
    beta: (C,) float32 or None.  act: "none", "relu", "silu" or "gelu" (erf).
    mean, rstd: (N, groups) float32, for the backward call."""
    lib = _native.load()
    _gpu_tensor(x, "x")
    xl = _layout_of(x, "x")
    if y is not None:
        _gpu_tensor(y, "y", x.device)
        if y.shape != x.shape or y.dtype != x.dtype:
            raise TypeError("y must match x in shape and dtype")
        yl = _layout_of(y, "y")
        if channels_last is not None and yl != (_native.NHWC if channels_last else _native.NCHW) and \
                not _one_layout(y):
            raise TypeError("y is not in the layout that channels_last asks for")
    else:
        yl = xl if channels_last is None else _native.NHWC if channels_last else _native.NCHW
    n, c, h, w = x.shape
    d, need = _norm_plan(_native.OP_FWD, n, c, h, w, groups, _dtype_code(x, "x"), act, xl, yl, float(eps))
    _f32(gamma, "gamma", (c,), x.device)
    _f32(beta, "beta", (c,), x.device)
    _f32(mean, "mean", (n, groups), x.device)
    _f32(rstd, "rstd", (n, groups), x.device)
    given = (y, mean, rstd)
    on = _On(x.device, stream)
    with on as s:
        made = []
        if y is None:
            made.append(y := _like(x, yl))
        if mean is None:
            made.append(mean := torch.empty((n, groups), dtype=torch.float32, device=x.device))
        if rstd is None:
            made.append(rstd := torch.empty_like(mean))
        ws, nbytes = _workspace(workspace, need, x.device)
        st = lib.wtconv_group_norm_forward(d, _ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(mean),
                                           _ptr(rstd), _ptr(ws), nbytes, s)
        on.made(*made)
    _native.check(st, "wtconv_group_norm_forward")
    _written(*given)
    return y, mean, rstd


def wtconv_group_norm_backward(x, dy, groups, mean, rstd, gamma=None, beta=None, act="none", dx=None, dgamma=None,
                               dbeta=None, workspace=None, stream=None):
    """(dx, dgamma, dbeta) of the forward call whose x, mean, rstd, gamma, beta
    and act these are.  dy may lie in either layout; dx lies as x does.
    dgamma, dbeta: (C,) float32, also where gamma or beta is None."""
    lib = _native.load()
    _gpu_tensor(x, "x")
    _gpu_tensor(dy, "dy", x.device)
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise TypeError("dy must match x in shape and dtype")
    xl, yl = _layout_of(x, "x"), _layout_of(dy, "dy")
    if dx is not None:
        _gpu_tensor(dx, "dx", x.device)
        if dx.shape != x.shape or dx.dtype != x.dtype or (_layout_of(dx, "dx") != xl and not _one_layout(x)):
            raise TypeError("dx must match x in shape, dtype and layout")
    n, c, h, w = x.shape
    # eps is in rstd already
    d, need = _norm_plan(_native.OP_BWD, n, c, h, w, groups, _dtype_code(x, "x"), act, xl, yl, 1.0)
    _f32(gamma, "gamma", (c,), x.device)
    _f32(beta, "beta", (c,), x.device)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _gpu_tensor(t, name, x.device)
        _f32(t, name, (n, groups), x.device)
    _f32(dgamma, "dgamma", (c,), x.device)
    _f32(dbeta, "dbeta", (c,), x.device)
    given = (dx, dgamma, dbeta)
    on = _On(x.device, stream)
    with on as s:
        made = []
        if dx is None:
            made.append(dx := _like(x, xl))
        if dgamma is None:
            made.append(dgamma := torch.empty((c,), dtype=torch.float32, device=x.device))
        if dbeta is None:
            made.append(dbeta := torch.empty_like(dgamma))
        ws, nbytes = _workspace(workspace, need, x.device)
        st = lib.wtconv_group_norm_backward(d, _ptr(x), _ptr(dy), _ptr(gamma), _ptr(beta), _ptr(mean),
                                            _ptr(rstd), _ptr(dx), _ptr(dgamma), _ptr(dbeta), _ptr(ws), nbytes, s)
        on.made(*made)
    _native.check(st, "wtconv_group_norm_backward")
    _written(*given)
    return dx, dgamma, dbeta


# ---- Newton-Schulz and the Muon step -------------------------------------------

@functools.lru_cache(maxsize=512)
def _ortho_plan(batch, rows, cols, dtype, steps, eps):
    """The descriptor of these sizes (as ctypes takes it) and its workspace."""
    d = _native.OrthoDesc(batch, rows, cols, dtype, steps, eps)
    out = ctypes.c_size_t(0)
    _native.check(_native.load().wtconv_orthogonalize_workspace_size(ctypes.byref(d), ctypes.byref(out)),
                  "wtconv_orthogonalize_workspace_size")
    return ctypes.byref(d), out.value


def _ortho_of(t, name, steps, eps):
    _gpu_tensor(t, name)
    if t.dim() not in (2, 3):
        raise TypeError("%s must be a (rows, cols) or (batch, rows, cols) tensor" % name)
    if not t.is_contiguous():
        raise TypeError("%s must be contiguous" % name)
    b, r, c = t.shape if t.dim() == 3 else (1,) + tuple(t.shape)
    return _ortho_plan(b, r, c, _dtype_code(t, name), int(steps), float(eps))


def wtconv_orthogonalize_workspace_size(shape, dtype_code, steps=5) -> int:
    """Bytes of workspace of wtconv_orthogonalize and wtconv_muon_step for
    matrices of shape (rows, cols) or (batch, rows, cols) and a gradient of
    type dtype_code."""
    b, r, c = shape if len(shape) == 3 else (1,) + tuple(shape)
    return _ortho_plan(b, r, c, dtype_code, int(steps), 1e-7)[1]


def wtconv_orthogonalize(g, steps=5, eps=1e-7, out=None, workspace=None, stream=None):
    """The Newton-Schulz iteration on g: a (rows, cols) matrix or a (batch,
    rows, cols) stack of them, contiguous float32, float16 or bfloat16.
    Singular values go towards 1 (to about 0.7 .. 1.2 in five steps)."""
    lib = _native.load()
    d, need = _ortho_of(g, "g", steps, eps)
    if out is not None:
        _gpu_tensor(out, "out", g.device)
        if out.shape != g.shape or out.dtype != g.dtype or not out.is_contiguous():
            raise TypeError("out must match g in shape, dtype and layout")
    given = out
    on = _On(g.device, stream)
    with on as s:
        made = None
        if out is None:
            made = out = torch.empty_like(g)
        ws, nbytes = _workspace(workspace, need, g.device)
        st = lib.wtconv_orthogonalize(d, _ptr(g), _ptr(out), _ptr(ws), nbytes, s)
        on.made(made)
    _native.check(st, "wtconv_orthogonalize")
    _written(given)
    return out


def wtconv_muon_step(weight, grad, momentum, lr, mu=0.95, weight_decay=0.0, scale=1.0, nesterov=True, steps=5,
                     eps=1e-7, weight_out=None, momentum_out=None, workspace=None, stream=None):
    """(weight_out, momentum_out) of one Muon step: momentum_out = mu momentum +
    (1 - mu) grad; weight_out = (1 - lr weight_decay) weight - lr scale O, with O
    the orthogonalised mu momentum_out + (1 - mu) grad (nesterov) or
    momentum_out.  weight and momentum are float32 (rows, cols) or (batch,
    rows, cols); grad may be float32, float16 or bfloat16.  In place unless
    weight_out / momentum_out are given."""
    lib = _native.load()
    d, need = _ortho_of(grad, "grad", steps, eps)
    _gpu_tensor(weight, "weight", grad.device)
    _gpu_tensor(momentum, "momentum", grad.device)
    weight_out = weight if weight_out is None else weight_out
    momentum_out = momentum if momentum_out is None else momentum_out
    for t, name in ((weight, "weight"), (momentum, "momentum"), (weight_out, "weight_out"),
                    (momentum_out, "momentum_out")):
        _f32(t, name, grad.shape, grad.device)
    hyper = _native.MuonHyper(float(lr), float(mu), float(weight_decay), float(scale), int(bool(nesterov)))
    on = _On(grad.device, stream)
    with on as s:
        ws, nbytes = _workspace(workspace, need, grad.device)
        st = lib.wtconv_muon_step(d, ctypes.byref(hyper), _ptr(weight), _ptr(grad), _ptr(momentum),
                                  _ptr(weight_out), _ptr(momentum_out), _ptr(ws), nbytes, s)
    _native.check(st, "wtconv_muon_step")
    _written(weight_out, momentum_out)
    return weight_out, momentum_out
