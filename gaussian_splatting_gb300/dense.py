"""The dense layers of a per-Gaussian attribute head on torch tensors.

``linear_fwd`` / ``linear_bwd`` (``y = act(x w^T + bias) + residual``), ``layernorm_fwd`` / ``layernorm_bwd``,
``groupnorm_fwd`` / ``groupnorm_bwd`` (channels-last feature maps, with an activation), ``embedding_fwd`` /
``embedding_bwd`` (learned codes) and ``adamw`` (the update of all of a network's tensors) check shapes, types, devices
and strides (``ValueError``), allocate what the caller did not hand in and call the entry points of the same names in libgs.so (``native.gs_linear_fwd`` and so on, which take
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


def embedding_fwd(table, idx, scale=1.0, out=None, stream=None):
    """y [rows, width]: ``scale`` times the rows of ``table`` [n, width] that ``idx`` (int32 or int64 [rows], contiguous)
    names; zeros where an index is not in 0..n-1 (no code)."""
    return (_binding or _load()).embedding_fwd(table, idx, scale, out, _handle(stream))


def embedding_bwd(dy, idx, n, scale=1.0, dtable=None, stream=None):
    """dtable [n, width] of ``embedding_fwd`` for the output gradient dy [rows, width]: ``scale`` times the sum of the
    rows of each code, zeros for a code without rows.  ``dtable`` receives it (overwritten) when given."""
    return (_binding or _load()).embedding_bwd(dy, idx, n, scale, dtable, _handle(stream))


def groupnorm_fwd(x, gamma, beta, groups, samples=1, act="none", eps=1e-5, out=None, stats=True, stream=None):
    """``(y, mean, rstd)``: y = act((x - mean) rstd gamma + beta) with mean and rstd over a map's rows and a group's
    channels.  x [samples * rows, channels] holds ``samples`` maps of equally many rows (a batch of channels-last images:
    ``images.permute(0, 2, 3, 1).reshape(-1, channels)``), its channels ``groups`` groups of neighbours.  mean and rstd
    (float32 [samples, groups], what the backward reads) are None with ``stats=False``.  ``out`` may be ``x``, which the
    backward then lacks."""
    return (_binding or _load()).groupnorm_fwd(x, gamma, beta, groups, samples, _act(act), eps, out, stats, _handle(stream))


def groupnorm_bwd(dy, x, gamma, beta, mean, rstd, act="none", skip=None, dx=None, dgamma=None, dbeta=None, need_dx=True,
                  need_dparams=True, stream=None):
    """``(dx, dgamma, dbeta)`` of ``groupnorm_fwd``; maps and groups are those of ``mean`` [samples, groups].  ``skip`` is
    a gradient added to dx (the residual path around the layer).  Outputs given are overwritten; ``dx`` may be ``dy`` or
    ``skip``."""
    return (_binding or _load()).groupnorm_bwd(dy, x, gamma, beta, mean, rstd, _act(act), skip, dx, dgamma, dbeta, need_dx,
                                               need_dparams, _handle(stream))


def adamw_state(params, bits=32):
    """``(exp_avg, exp_avg_sq, scales)`` for ``adamw``, all zero: a float32 tensor like each of ``params``, or with
    ``bits=8`` a float8_e4m3fn one and, in ``scales``, the two lists of its float32 scales (None with 32 bits)."""
    import torch
    if bits not in (8, 32):
        raise ValueError(f"bits must be 32 or 8, got {bits!r}")
    params = list(params)

    def zeros():
        # (zeroed as bytes: not every operation takes the 8-bit type)
        return [torch.zeros(p.shape, dtype=torch.float32, device=p.device) if bits == 32 else
                torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(torch.float8_e4m3fn) for p in params]

    def scale():
        return [torch.zeros((p.numel() + 255) // 256, dtype=torch.float32, device=p.device) for p in params]

    return zeros(), zeros(), None if bits == 32 else (scale(), scale())


def adamw(params, grads, exp_avg, exp_avg_sq, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, scales=None,
          copies=None, seed=0, counts=None, stream=None):
    """One AdamW step, number ``step`` (from 1), over all tensors of the list ``params`` (float32), in place, from ``grads``
    (float32 or bfloat16, all alike).  ``lr`` and ``weight_decay`` are numbers, or sequences of one for each tensor.

    The moments (``adamw_state`` makes them) are float32, or with ``scales`` float8_e4m3fn: ``exp_avg_sq`` then holds the
    root of the second moment, and each 256 neighbouring values of a tensor share a scale.  They are rounded at random, by
    ``seed`` and ``step`` alone: the same call gives the same bits.  (So does a captured one each time it is replayed, with the
    same bias corrections: ``step`` and ``lr`` are taken when it is captured.)  A value without gradients in a run whose
    scales stay keeps a small rest of its moments, which ``gs.h`` states; 32-bit ones fade to zero.  ``copies`` (bfloat16, like ``params``) receive the
    updated parameters, for layers that compute in bfloat16.  With ``counts`` (int64 [records, 2], as
    ``AttributeHead.status`` or ``StepResult.status``) the step is skipped on the device where any record's second
    entry is not zero.  Tensors are contiguous; none may overlap another, but for gradients among
    themselves."""
    (_binding or _load()).adamw(params, grads, exp_avg, exp_avg_sq, step, lr, betas[0], betas[1], eps, weight_decay, scales,
                                copies, seed, counts, _handle(stream))
