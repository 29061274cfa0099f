"""The dense layers of a per-Gaussian attribute head on torch tensors.

``linear_fwd`` / ``linear_bwd`` (``y = act(x w^T + bias) + residual``) and ``layernorm_fwd`` /
``layernorm_bwd`` check shapes, types, devices and strides (``ValueError``), allocate what the caller did not
hand in and call the entry points of the same names in libgs.so (``native.gs_linear_fwd`` and so on, which take
addresses), where the formulas stand.  Matrices are 2-D CUDA tensors, float32 or bfloat16, whose rows may be any
distance apart (``stride(1) == 1``); the arrays of one call share one type.  Nothing synchronises with
the host, and nothing is kept between calls.

Work is enqueued on ``stream`` (a ``torch.cuda.Stream``, a handle, or None: the current torch stream), on which
the tensors must be ready.  Outputs and scratch that a call allocates belong to that stream.  ``status`` is an
int32 CUDA tensor that is set to nonzero if a bounded wait on the device gave up, and is never cleared: without it
such a call's invalid outputs go unnoticed.  An output that a call is handed must not overlap its inputs or another
output, but for the cases named below.

Autograd does not see these calls: outputs never require a gradient, whatever the inputs do.  The backward functions
are called by the program, as ``head.py`` does.
"""
from __future__ import annotations

from . import _native as N

_ACTS = {"none": N.GS_ACT_NONE, "relu": N.GS_ACT_RELU, "gelu": N.GS_ACT_GELU, "silu": N.GS_ACT_SILU}
_binding = None


def _load():
    """The module _dense (raises if it was not built)."""
    global _binding
    if _binding is None:
        import torch  # noqa: F401  (its libraries come first)
        N.load()
        from . import _dense
        _binding = _dense
    return _binding


def _act(act):
    try:
        return _ACTS[act]
    except (KeyError, TypeError):
        raise ValueError(f"act must be one of {', '.join(_ACTS)}, got {act!r}") from None


def _handle(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def _matrix(t, name, rows, cols, like):
    """Row stride of a matrix argument, checked against the call's shape, type and device."""
    return _load().check_matrix(t, name, rows, cols, like)


def _vector(t, name, n, like):
    _load().check_vector(t, name, n, like)


def linear_fwd(x, w, bias=None, residual=None, act="none", keep_z=False, out=None, z=None, status=None, stream=None):
    """``(y, z)``: y = act(x w^T + bias) + residual, and z the sum before the activation (None unless
    ``keep_z`` or ``z`` asks for it).  x [rows, in], w [out, in], bias [out], residual [rows, out].
    ``out`` / ``z`` receive the results when given; ``out`` may be ``residual``."""
    return (_binding or _load()).linear_fwd(x, w, bias, residual, _act(act), keep_z, out, z, status, _handle(stream))


def linear_bwd(dy, x, w, z=None, act="none", bias=True, dx=None, dw=None, dbias=None, need_dx=True, need_dw=True,
               status=None, stream=None):
    """``(dx, dw, dbias)`` of ``linear_fwd`` for the output gradient dy (the residual's gradient is dy
    itself).  z is the forward's (``keep_z``), not needed with act "none".  ``bias=False``,
    ``need_dx=False`` and ``need_dw=False`` leave that output out (None).  ``dx`` / ``dw`` / ``dbias``
    receive the results (overwritten) when given."""
    return (_binding or _load()).linear_bwd(dy, x, w, z, _act(act), bias, dx, dw, dbias, need_dx, need_dw, status,
                                            _handle(stream))


def layernorm_fwd(x, gamma, beta, eps=1e-5, out=None, stats=True, stream=None):
    """``(y, mean, rstd)``: y = (x - mean) rstd gamma + beta by rows; mean and rstd (float32 [rows], what
    the backward reads) are None with ``stats=False``.  ``out`` may be ``x``."""
    return (_binding or _load()).layernorm_fwd(x, gamma, beta, eps, out, stats, _handle(stream))


def layernorm_bwd(dy, x, gamma, mean, rstd, skip=None, dx=None, dgamma=None, dbeta=None, need_dx=True,
                  need_dparams=True, stream=None):
    """``(dx, dgamma, dbeta)`` of ``layernorm_fwd``; ``skip`` is a gradient added to dx (the residual
    path around the layer).  Outputs given are overwritten; ``dx`` may be ``dy`` or ``skip``."""
    return (_binding or _load()).layernorm_bwd(dy, x, gamma, mean, rstd, skip, dx, dgamma, dbeta, need_dx, need_dparams,
                                               _handle(stream))
