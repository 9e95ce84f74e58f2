"""Binding of the operators of a block's half over the channels and of its
training step: the root-mean-square norm with the residual's addition, the gated
product, and the gradients' global norm and clipping.  Argument checks and
marshalling only, in the manner of the group norm's and Muon's binding (_train):
streams, devices, buffers and what counts as modified for autograd are as there.
"""
from __future__ import annotations

import array
import ctypes
import functools
import math

import torch

from . import _native
from ._train import _DTYPES, _F32, _On, _dtype_code, _f32, _gpu_tensor, _ptr, _workspace, _written


def _rows_of(t, name):
    """(rows, c) of a contiguous (..., c) tensor."""
    _gpu_tensor(t, name)
    if t.dim() < 1:
        raise TypeError("%s must be a (..., C) tensor" % name)
    if not t.is_contiguous():
        raise TypeError("%s must be contiguous" % name)
    c = t.shape[-1]
    return (t.numel() // c if c else 0), c


def _same(t, name, like, shape=None, dtype=None):
    dtype = like.dtype if dtype is None else dtype
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == (like.shape if shape is None else shape) and \
            t.device == like.device and t.is_contiguous():
        return
    _gpu_tensor(t, name, like.device)
    if t.shape != (like.shape if shape is None else shape) or t.dtype != dtype or not t.is_contiguous():
        raise TypeError("%s must be a contiguous %s tensor of shape %s" % (
            name, dtype, tuple(like.shape if shape is None else shape)))


# ---- root-mean-square norm -------------------------------------------------------

@functools.lru_cache(maxsize=512)
def _rms_plan(op, rows, c, dtype, eps):
    """The descriptor of these sizes (as ctypes takes it) and op's workspace."""
    d = _native.RmsDesc(rows, c, dtype, eps)
    out = ctypes.c_size_t(0)
    _native.check(_native.load().wtconv_rms_norm_workspace_size(ctypes.byref(d), op, ctypes.byref(out)),
                  "wtconv_rms_norm_workspace_size")
    return ctypes.byref(d), out.value


def wtconv_rms_norm_workspace_size(shape, dtype_code, op) -> int:
    """Bytes of workspace of the forward (OP_FWD) or backward (OP_BWD) call for
    activations of shape (..., C)."""
    return _rms_plan(op, math.prod(shape[:-1]), shape[-1], dtype_code, 1e-6)[1]


def wtconv_rms_norm_forward(x, residual=None, gamma=None, eps=1e-6, y=None, h=None, rstd=None, stream=None):
    """(y, h, rstd) of h = x + residual (rounded to their type), y = gamma h rstd,
    rstd = 1 / sqrt(mean of h^2 over the last dimension + eps).

    x, residual: contiguous (..., C) float32, float16 or bfloat16 tensors of one
    type and shape; without a residual h is x itself.  gamma: (C,) float32 or None.
    rstd: float32 of shape (...), for the backward call.  h may be given as x or
    residual (in place)."""
    lib = _native.load()
    rows, c = _rows_of(x, "x")
    d, _ = _rms_plan(_native.OP_FWD, rows, c, _dtype_code(x, "x"), float(eps))
    if residual is not None:
        _same(residual, "residual", x)
    elif h is not None and h is not x:
        raise TypeError("without a residual h is x itself")
    _f32(gamma, "gamma", (c,), x.device)
    if y is not None:
        _same(y, "y", x)
    if h is not None:
        _same(h, "h", x)
    _f32(rstd, "rstd", x.shape[:-1], x.device)
    given = (y, h if residual is not None else None, rstd)
    on = _On(x.device, stream)
    with on as s:
        made = []
        if y is None:
            made.append(y := torch.empty_like(x))
        if residual is None:
            h = x
        elif h is None:
            made.append(h := torch.empty_like(x))
        if rstd is None:
            made.append(rstd := torch.empty(x.shape[:-1], dtype=_F32, device=x.device))
        st = lib.wtconv_rms_norm_forward(d, _ptr(x), _ptr(residual), _ptr(gamma), _ptr(y), _ptr(h), _ptr(rstd), s)
        on.made(*made)
    _native.check(st, "wtconv_rms_norm_forward")
    _written(*given)
    return y, h, rstd


def wtconv_rms_norm_backward(h, dy, rstd, gamma=None, dh=None, dx=None, dgamma=None, workspace=None, stream=None):
    """(dx, dgamma) of the forward call whose h, rstd and gamma these are; dx is
    the residual's gradient too.  dy: the gradient of y; dh: the gradient that
    reaches h otherwise, or None.  dgamma: (C,) float32, also where gamma is None.
    dx may be given as dh (in place)."""
    lib = _native.load()
    rows, c = _rows_of(h, "h")
    # eps is in rstd already
    d, need = _rms_plan(_native.OP_BWD, rows, c, _dtype_code(h, "h"), 1.0)
    _same(dy, "dy", h)
    _gpu_tensor(rstd, "rstd", h.device)
    _f32(rstd, "rstd", h.shape[:-1], h.device)
    _f32(gamma, "gamma", (c,), h.device)
    if dh is not None:
        _same(dh, "dh", h)
    if dx is not None:
        _same(dx, "dx", h)
    _f32(dgamma, "dgamma", (c,), h.device)
    given = (dx, dgamma)
    on = _On(h.device, stream)
    with on as s:
        made = []
        if dx is None:
            made.append(dx := torch.empty_like(h))
        if dgamma is None:
            made.append(dgamma := torch.empty((c,), dtype=_F32, device=h.device))
        ws, nbytes = _workspace(workspace, need, h.device)
        st = lib.wtconv_rms_norm_backward(d, _ptr(h), _ptr(dy), _ptr(dh), _ptr(gamma), _ptr(rstd), _ptr(dx),
                                          _ptr(dgamma), _ptr(ws), nbytes, s)
        on.made(*made)
    _native.check(st, "wtconv_rms_norm_backward")
    _written(*given)
    return dx, dgamma


# ---- gated product ---------------------------------------------------------------

@functools.lru_cache(maxsize=512)
def _gated_plan(op, rows, c, f, dtype, act):
    """The descriptor of these sizes (as ctypes takes it) and op's workspace."""
    if act not in _native.ACTS:
        raise ValueError("act must be one of %s, got %r" % (", ".join(sorted(_native.ACTS)), act))
    d = _native.GatedDesc(rows, c, f, dtype, _native.ACTS[act])
    out = ctypes.c_size_t(0)
    _native.check(_native.load().wtconv_gated_workspace_size(ctypes.byref(d), op, ctypes.byref(out)),
                  "wtconv_gated_workspace_size")
    return ctypes.byref(d), out.value


def wtconv_gated_workspace_size(shape, f, dtype_code, op) -> int:
    """Bytes of workspace of the forward (OP_FWD) or backward (OP_BWD) call for x
    of shape (..., C) and f columns of each projection."""
    return _gated_plan(op, math.prod(shape[:-1]), shape[-1], f, dtype_code, "none")[1]


def _gated_of(op, x, w_gate, w_up, b_gate, b_up, act):
    rows, c = _rows_of(x, "x")
    _gpu_tensor(w_gate, "w_gate", x.device)
    if w_gate.dim() != 2 or w_gate.shape[1] != c:
        raise TypeError("w_gate must be a (F, C) tensor with C = %d" % c)
    f = w_gate.shape[0]
    d, need = _gated_plan(op, rows, c, f, _dtype_code(x, "x"), act)
    for t, name in ((w_gate, "w_gate"), (w_up, "w_up")):
        _same(t, name, x, (f, c))
    _f32(b_gate, "b_gate", (f,), x.device)
    _f32(b_up, "b_up", (f,), x.device)
    return d, need, f


def _factors(*tensors):
    """x and the weights, or copies that start on 16 bytes where the call asks for
    that: rows of 16-bit elements that 8 divides are read as they lie."""
    if tensors[0].dtype is _F32 or tensors[0].shape[-1] % 8:
        return tensors
    return [t if t.data_ptr() % 16 == 0 else t.clone() for t in tensors]


def wtconv_gated_forward(x, w_gate, w_up, b_gate=None, b_up=None, act="silu", h=None, workspace=None, stream=None):
    """h = act(x w_gate^T + b_gate) * (x w_up^T + b_up).

    x: contiguous (..., C) float32, float16 or bfloat16; w_gate, w_up: contiguous
    (F, C) of x's type; b_gate, b_up: (F,) float32 or None; h: (..., F) of x's type.
    act: "none", "relu", "silu" or "gelu" (erf)."""
    lib = _native.load()
    d, need, f = _gated_of(_native.OP_FWD, x, w_gate, w_up, b_gate, b_up, act)
    shape = x.shape[:-1] + (f,)
    if h is not None:
        _same(h, "h", x, shape)
    given = h
    on = _On(x.device, stream)
    with on as s:
        made = None
        if h is None:
            made = h = torch.empty(shape, dtype=x.dtype, device=x.device)
        ws, nbytes = _workspace(workspace, need, x.device)
        xa, ga, ua = _factors(x, w_gate, w_up)
        st = lib.wtconv_gated_forward(d, _ptr(xa), _ptr(ga), _ptr(ua), _ptr(b_gate), _ptr(b_up), _ptr(h), _ptr(ws),
                                      nbytes, s)
        on.made(made)
    _native.check(st, "wtconv_gated_forward")
    _written(given)
    return h


def wtconv_gated_backward(x, dh, w_gate, w_up, b_gate=None, b_up=None, act="silu", need=(True, True, True), dx=None,
                          dw_gate=None, dw_up=None, db_gate=None, db_up=None, workspace=None, stream=None,
                          dw_dtype=None):
    """(dx, dw_gate, dw_up, db_gate, db_up) of the forward call whose x, weights,
    biases and act these are; dh: the gradient of h.  db_gate, db_up: (F,) float32,
    also where a bias is None; the others have x's type, dw_gate and dw_up where
    dw_dtype is torch.float32 that one (their sums unrounded, for parameters that are
    kept in it).  The gradients of both projections are rounded to x's type before the
    products that dx and the weights' gradients are: in float16 they keep their digits
    between 2^-14 and 65504, as any float16 gradient.  need: whether dx, the weights'
    and the biases' gradients are wanted; the others come as None."""
    lib = _native.load()
    d, size, f = _gated_of(_native.OP_BWD, x, w_gate, w_up, b_gate, b_up, act)
    _same(dh, "dh", x, x.shape[:-1] + (f,))
    need_dx, need_dw, need_db = need
    if not (need_dx or need_dw or need_db):
        raise ValueError("need asks for none of the gradients")
    if dw_dtype is None:
        dw_dtype = x.dtype
    elif dw_dtype not in (x.dtype, _F32):
        raise ValueError("dw_dtype must be %s or float32, got %s" % (x.dtype, dw_dtype))
    for t, wanted, name in ((dx, need_dx, "dx"), (dw_gate, need_dw, "dw_gate"), (dw_up, need_dw, "dw_up"),
                            (db_gate, need_db, "db_gate"), (db_up, need_db, "db_up")):
        if t is not None and not wanted:
            raise ValueError("%s is given, but need does not ask for it" % name)
    for t, name, shape, dtype in ((dx, "dx", x.shape, x.dtype), (dw_gate, "dw_gate", w_gate.shape, dw_dtype),
                                  (dw_up, "dw_up", w_gate.shape, dw_dtype)):
        if t is not None:
            _same(t, name, x, shape, dtype)
    _f32(db_gate, "db_gate", (f,), x.device)
    _f32(db_up, "db_up", (f,), x.device)
    given = (dx, dw_gate, dw_up, db_gate, db_up)
    on = _On(x.device, stream)
    with on as s:
        made = []
        if dx is None and need_dx:
            made.append(dx := torch.empty_like(x))
        if dw_gate is None and need_dw:
            made.append(dw_gate := torch.empty_like(w_gate, dtype=dw_dtype))
        if dw_up is None and need_dw:
            made.append(dw_up := torch.empty_like(w_up, dtype=dw_dtype))
        if db_gate is None and need_db:
            made.append(db_gate := torch.empty((f,), dtype=_F32, device=x.device))
        if db_up is None and need_db:
            made.append(db_up := torch.empty((f,), dtype=_F32, device=x.device))
        ws, nbytes = _workspace(workspace, size, x.device)
        xa, ga, ua = _factors(x, w_gate, w_up)
        call = lib.wtconv_gated_backward if dw_dtype is x.dtype else lib.wtconv_gated_backward_f32_grads
        st = call(d, _ptr(xa), _ptr(dh), _ptr(ga), _ptr(ua), _ptr(b_gate), _ptr(b_up), _ptr(dx), _ptr(dw_gate),
                  _ptr(dw_up), _ptr(db_gate), _ptr(db_up), _ptr(ws), nbytes, s)
        on.made(*made)
    _native.check(st, "wtconv_gated_backward")
    _written(*given)
    return dx, dw_gate, dw_up, db_gate, db_up


# ---- gradient norm and clipping ----------------------------------------------------

@functools.lru_cache(maxsize=512)
def wtconv_grad_norm_workspace_size(count) -> int:
    """Bytes of workspace of wtconv_grad_norm and wtconv_clip_grad_norm for `count` tensors."""
    out = ctypes.c_size_t(0)
    _native.check(_native.load().wtconv_grad_norm_workspace_size(count, ctypes.byref(out)),
                  "wtconv_grad_norm_workspace_size")
    return out.value


def _table(grads, out, device):
    """The C entry point's table of tensors (_native.TensorEntry), as whole numbers of
    64 bits: a fifth of the time that a structure's fields take."""
    rows, index, codes, Tensor, apart = [], device.index, _DTYPES, torch.Tensor, out is not grads
    for i, g in enumerate(grads):
        # (a device's index and element counts: comparing devices and shapes takes half a microsecond)
        if not isinstance(g, Tensor) or g.get_device() != index or not g.is_contiguous():
            _gpu_tensor(g, "grads[%d]" % i, device)
            raise TypeError("grads[%d] must be contiguous" % i)
        code = codes.get(g.dtype)
        if code is None:
            _dtype_code(g, "grads[%d]" % i)
        at = to = g.data_ptr()
        n = g.numel()
        if apart:
            o = out[i]
            if not isinstance(o, Tensor) or o.dtype is not g.dtype or o.numel() != n or o.get_device() != index or \
                    not o.is_contiguous():
                raise TypeError("out[%d] must match grads[%d] in type, elements and device, and be contiguous" % (i, i))
            to = o.data_ptr()
        rows += (at, to, n, code)
    return array.array("Q", rows)


def _norm_call(grads, device, norm):
    """(list of grads, their device)."""
    grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    if grads:
        _gpu_tensor(grads[0], "grads[0]")
        if device is not None:
            asked = torch.device(device)  # without an index: any
            if asked != grads[0].device and (asked.type != "cuda" or asked.index is not None):
                raise TypeError("grads[0] lies on %s, not on %s" % (grads[0].device, device))
        device = grads[0].device
    else:
        device = torch.device("cuda" if device is None else device)
        if device.type != "cuda":
            raise TypeError("the norm of no tensors is asked for on %s, not on a GPU" % device)
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
    if norm is not None:
        _gpu_tensor(norm, "norm", device)
        _f32(norm, "norm", (), device)
    return grads, device


def wtconv_grad_norm(grads, norm=None, workspace=None, stream=None, device=None):
    """sqrt of the sum of the squares of all elements of `grads`, contiguous
    float32, float16 or bfloat16 tensors of any shapes on one device: a float32
    tensor of no dimensions on that device (no synchronisation; 0 for no tensors,
    on `device` or the current one)."""
    lib = _native.load()
    grads, device = _norm_call(grads, device, norm)
    table = _table(grads, grads, device)
    given = norm
    on = _On(device, stream)
    with on as s:
        made = None
        if norm is None:
            made = norm = torch.empty((), dtype=_F32, device=device)
        ws, nbytes = _workspace(workspace, wtconv_grad_norm_workspace_size(len(grads)), device)
        st = lib.wtconv_grad_norm(table.buffer_info()[0], len(grads), _ptr(norm), _ptr(ws), nbytes, s)
        on.made(made)
    _native.check(st, "wtconv_grad_norm")
    _written(given)
    return norm


def wtconv_clip_grad_norm(grads, max_norm, eps=1e-6, out=None, norm=None, workspace=None, stream=None, device=None):
    """(norm, out): the norm of wtconv_grad_norm, and every tensor times
    min(1, max_norm / (norm + eps)), in place or in the tensors of `out` (each of its
    gradient's type and number of elements).  max_norm and eps go by value into a
    captured graph."""
    lib = _native.load()
    grads, device = _norm_call(grads, device, norm)
    out = grads if out is None else [out] if isinstance(out, torch.Tensor) else list(out)
    if len(out) != len(grads):
        raise ValueError("out has %d tensors, grads has %d" % (len(out), len(grads)))
    table = _table(grads, out, device)
    given = norm
    on = _On(device, stream)
    with on as s:
        made = None
        if norm is None:
            made = norm = torch.empty((), dtype=_F32, device=device)
        ws, nbytes = _workspace(workspace, wtconv_grad_norm_workspace_size(len(grads)), device)
        st = lib.wtconv_clip_grad_norm(table.buffer_info()[0], len(grads), float(max_norm), float(eps), _ptr(norm),
                                       _ptr(ws), nbytes, s)
        on.made(made)
    _native.check(st, "wtconv_clip_grad_norm")
    _written(given, *out)
    return norm, out
