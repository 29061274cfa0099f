"""The dense layers of a per-Gaussian attribute head on torch tensors.

``linear_fwd`` / ``linear_bwd`` (``y = act(x w^T + bias) + residual``) and ``layernorm_fwd`` /
``layernorm_bwd`` check shapes, types, devices and strides, allocate what the caller did not hand in
and call the entry points of the same names in libgs.so (``native.gs_linear_fwd`` and so on), where
the formulas stand.  Matrices are 2-D CUDA tensors, float32 or bfloat16, whose rows may be any
distance apart (``stride(1) == 1``); the arrays of one call share one type.  Nothing synchronises with
the host, and nothing is kept between calls.

Work is enqueued on ``stream`` (the current torch stream when None), on which the tensors must be ready.
Outputs and scratch that a call allocates belong to that stream.
"""
from __future__ import annotations

from ctypes import addressof

import torch

from . import _native as N

_DTYPES = {torch.float32: N.GS_F32, torch.bfloat16: N.GS_BF16}
_ACTS = {"none": N.GS_ACT_NONE, "relu": N.GS_ACT_RELU, "gelu": N.GS_ACT_GELU, "silu": N.GS_ACT_SILU}


def _matrix(t, name, rows, cols, like):
    """Row stride of a matrix argument, checked against the call's shape, type and device."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must have shape [{rows}, {cols}], got {list(t.shape)}")
    if t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    if rows <= 1:
        return cols
    if s0 < cols:
        raise ValueError(f"{name} has overlapping rows (stride {s0} < {cols})")
    return s0


def _vector(t, name, n, like):
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n}, got {list(t.shape)}")
    if t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")


def _start(x, name):
    if x.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got {list(x.shape)}")
    if x.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor: there is no CPU path")
    return x.shape


class _On:
    """The stream of a call as a handle, with its device and stream made torch's current ones for the call's span."""

    def __init__(self, device, stream):
        self.guards = []
        if device.index != torch.cuda.current_device():
            self.guards.append(torch.cuda.device(device))
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        if stream is not None:
            self.guards.append(torch.cuda.stream(stream))
        self.index = device.index

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return _raw_stream(self.index)

    def __exit__(self, *e):
        for g in reversed(self.guards):
            g.__exit__(*e)


class _Here:
    """_On for the usual call: the current device and its current stream, nothing to enter."""

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *e):
        pass


_raw_stream = torch._C._cuda_getCurrentRawStream  # a handle without the Stream object around it
_current = torch._C._cuda_getDevice


def _on(device, stream):
    if stream is None and device.index == _current():
        return _Here(_raw_stream(device.index))
    return _On(device, stream)


def _scratch(n, device):
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


_entry = {}


def _call(name, *args):
    """A C entry point: its function looked up once, its status checked."""
    f = _entry.get(name)
    if f is None:
        f = _entry[name] = getattr(N.load(), name)
    status = f(*args)
    if status:
        N._check(status, name)


def _size(name, desc):
    f = _entry.get(name)
    if f is None:
        f = _entry[name] = getattr(N.load(), name)
    return f(desc)


def _at(t):
    return None if t is None else t.data_ptr()


def linear_fwd(x, w, bias=None, residual=None, act="none", keep_z=False, out=None, z=None, status=None, stream=None):
    """``(y, z)``: y = act(x w^T + bias) + residual, and z the sum before the activation (None unless
    ``keep_z`` or ``z`` asks for it).  x [rows, in], w [out, in], bias [out], residual [rows, out].
    ``out`` / ``z`` receive the results when given; ``out`` may be ``residual``.  ``status``: an int32
    CUDA tensor that is set to nonzero if a bounded wait on the device gave up."""
    rows, n_in = _start(x, "x")
    n_out = w.shape[0]
    d = N.LinearDesc()
    d.rows, d.in_features, d.out_features, d.dtype, d.act = rows, n_in, n_out, _DTYPES[x.dtype], _ACTS[act]
    d.ldx, d.ldw = _matrix(x, "x", rows, n_in, x), _matrix(w, "w", n_out, n_in, x)
    if bias is not None:
        _vector(bias, "bias", n_out, x)
    if residual is not None:
        d.ldr = _matrix(residual, "residual", rows, n_out, x)
    with _on(x.device, stream) as st:
        if out is None:
            out = torch.empty((rows, n_out), dtype=x.dtype, device=x.device)
            d.ldy = n_out
        else:
            d.ldy = _matrix(out, "out", rows, n_out, x)
        if z is not None:
            d.ldz = _matrix(z, "z", rows, n_out, x)
        elif keep_z:
            z = torch.empty((rows, n_out), dtype=x.dtype, device=x.device)
            d.ldz = n_out
        at = addressof(d)
        need = _size("gs_linear_fwd_workspace_size", at)
        ws = _scratch(need, x.device)
        _call("gs_linear_fwd", at, x.data_ptr(), w.data_ptr(), _at(bias), _at(residual), out.data_ptr(), _at(z), _at(ws), need,
              _at(status), st)
    return out, z


def linear_bwd(dy, x, w, z=None, act="none", bias=True, dx=None, dw=None, dbias=None, need_dx=True, need_dw=True,
               status=None, stream=None):
    """``(dx, dw, dbias)`` of ``linear_fwd`` for the output gradient dy (the residual's gradient is dy
    itself).  z is the forward's (``keep_z``), not needed with act "none".  ``bias=False``,
    ``need_dx=False`` and ``need_dw=False`` leave that output out (None).  ``dx`` / ``dw`` / ``dbias``
    receive the results (overwritten) when given."""
    rows, n_out = _start(dy, "dy")
    n_in = x.shape[1]
    d = N.LinearDesc()
    d.rows, d.in_features, d.out_features, d.dtype, d.act = rows, n_in, n_out, _DTYPES[dy.dtype], _ACTS[act]
    d.ldy, d.ldx = _matrix(dy, "dy", rows, n_out, dy), _matrix(x, "x", rows, n_in, dy)
    d.ldw = _matrix(w, "w", n_out, n_in, dy)
    if act == "none":
        z = None
    elif z is None:
        raise ValueError(f"z is needed for the gradient of {act}")
    else:
        d.ldz = _matrix(z, "z", rows, n_out, dy)
    with _on(dy.device, stream) as st:
        if dx is not None:
            d.lddx = _matrix(dx, "dx", rows, n_in, dy)
        elif need_dx:
            dx = torch.empty((rows, n_in), dtype=dy.dtype, device=dy.device)
            d.lddx = n_in
        if dw is not None:
            d.lddw = _matrix(dw, "dw", n_out, n_in, dy)
        elif need_dw:
            dw = torch.empty((n_out, n_in), dtype=dy.dtype, device=dy.device)
            d.lddw = n_in
        if dbias is not None:
            _vector(dbias, "dbias", n_out, dy)
        elif bias:
            dbias = torch.empty(n_out, dtype=dy.dtype, device=dy.device)
        at = addressof(d)
        need = _size("gs_linear_bwd_workspace_size", at)
        ws = _scratch(need, dy.device)
        _call("gs_linear_bwd", at, dy.data_ptr(), x.data_ptr(), w.data_ptr(), _at(z), _at(dx), _at(dw), _at(dbias), _at(ws), need,
              _at(status), st)
    return dx, dw, dbias


def layernorm_fwd(x, gamma, beta, eps=1e-5, out=None, stats=True, stream=None):
    """``(y, mean, rstd)``: y = (x - mean) rstd gamma + beta by rows; mean and rstd (float32 [rows], what
    the backward reads) are None with ``stats=False``.  ``out`` may be ``x``."""
    rows, n = _start(x, "x")
    d = N.LayerNormDesc()
    d.rows, d.width, d.dtype, d.eps = rows, n, _DTYPES[x.dtype], eps
    d.ldx = _matrix(x, "x", rows, n, x)
    _vector(gamma, "gamma", n, x)
    _vector(beta, "beta", n, x)
    with _on(x.device, stream) as st:
        if out is None:
            out = torch.empty((rows, n), dtype=x.dtype, device=x.device)
            d.ldy = n
        else:
            d.ldy = _matrix(out, "out", rows, n, x)
        mean = torch.empty(rows, dtype=torch.float32, device=x.device) if stats else None
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device) if stats else None
        _call("gs_layernorm_fwd", addressof(d), x.data_ptr(), gamma.data_ptr(), beta.data_ptr(), out.data_ptr(), _at(mean),
              _at(rstd), st)
    return out, mean, rstd


def layernorm_bwd(dy, x, gamma, mean, rstd, skip=None, dx=None, dgamma=None, dbeta=None, need_dx=True,
                  need_dparams=True, stream=None):
    """``(dx, dgamma, dbeta)`` of ``layernorm_fwd``; ``skip`` is a gradient added to dx (the residual
    path around the layer).  Outputs given are overwritten; ``dx`` may be ``dy`` or ``skip``."""
    rows, n = _start(dy, "dy")
    d = N.LayerNormDesc()
    d.rows, d.width, d.dtype = rows, n, _DTYPES[dy.dtype]
    d.lddy, d.ldx = _matrix(dy, "dy", rows, n, dy), _matrix(x, "x", rows, n, dy)
    _vector(gamma, "gamma", n, dy)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t.dtype != torch.float32 or t.device != dy.device or tuple(t.shape) != (rows,) or (rows > 1 and t.stride(0) != 1):
            raise ValueError(f"{name} must be a contiguous float32 vector of {rows} on {dy.device}")
    if skip is not None:
        d.ldskip = _matrix(skip, "skip", rows, n, dy)
    with _on(dy.device, stream) as st:
        if dx is not None:
            d.lddx = _matrix(dx, "dx", rows, n, dy)
        elif need_dx:
            dx = torch.empty((rows, n), dtype=dy.dtype, device=dy.device)
            d.lddx = n
        if dgamma is not None:
            _vector(dgamma, "dgamma", n, dy)
        elif need_dparams:
            dgamma = torch.empty(n, dtype=dy.dtype, device=dy.device)
        if dbeta is not None:
            _vector(dbeta, "dbeta", n, dy)
        elif need_dparams:
            dbeta = torch.empty(n, dtype=dy.dtype, device=dy.device)
        at = addressof(d)
        need = _size("gs_layernorm_bwd_workspace_size", at) if dgamma is not None or dbeta is not None else 0
        ws = _scratch(need, dy.device)
        _call("gs_layernorm_bwd", at, dy.data_ptr(), x.data_ptr(), gamma.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _at(skip),
              _at(dx), _at(dgamma), _at(dbeta), _at(ws), need, st)
    return dx, dgamma, dbeta
