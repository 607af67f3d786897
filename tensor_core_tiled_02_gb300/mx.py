"""The norm between layers and microscaled operands on torch tensors
(``include/mx_ops.h``).

``rms_norm`` adds the residual, normalises and scales; ``rms_norm_mx`` writes the
result as ``mx_linear`` reads it: blocks of 32 values in 8 bits ("e4m3") or 4
("e2m1") that share a power-of-two scale (the OCP formats MXFP8 and MXFP4).
``mx_quantize`` brings weights and activations into that form, ``mx_dequantize``
back.  The rest is as in ``layers.py``: rows may be strided, calls are
asynchronous on ``stream`` (default: torch's current stream of the tensors'
device), nothing records an autograd graph, ``ValueError`` for tensors a call
cannot take, ``GemmError`` for a status of the library.

A microscaled matrix is ``Mx(data, scale, cols, format)``; any tuple of these four
will do as an operand.  ``data`` is uint8 [rows, blocks * 32 or 16 bytes], the last
block filled up with zeros; ``scale`` is uint8 [rows / 128, blocks / 4, 32, 4, 4]
(rounded up): the block's exponent plus 127 at [row // 128, block // 4, row % 32,
row // 32 % 4, block % 4], 255 for a block of NaN.
"""
from __future__ import annotations

from typing import NamedTuple

from .layers import _act, _call

FORMATS = {"e4m3": 0, "e2m1": 1}


class Mx(NamedTuple):
    """A matrix [rows, cols] in microscaled blocks along its rows."""

    data: object
    scale: object
    cols: int
    format: str


_new = tuple.__new__  # an Mx of four values, without its constructor's steps


def _format(format):
    code = FORMATS.get(format) if isinstance(format, str) else None
    if code is None:
        raise ValueError(f"format must be one of {sorted(FORMATS)}, got {format!r}")
    return code


def _mx(a, name):
    if not isinstance(a, tuple) or len(a) != 4:
        raise ValueError(f"{name} must be an Mx: (data, scale, cols, format)")
    return a


_DTYPES = {None: 1}  # and torch's two, once torch is there


def _dtype(dtype):
    try:
        return _DTYPES[dtype]
    except (KeyError, TypeError):
        import torch

        _DTYPES.update({torch.float16: 0, torch.bfloat16: 1})
        if dtype is torch.float16 or dtype is torch.bfloat16:
            return _DTYPES[dtype]
        raise ValueError(f"dtype must be torch.float16 or torch.bfloat16, got {dtype!r}") from None


def rms_norm(x, weight, residual=None, eps=1e-6, save=False, out=None, h_out=None, stream=None):
    """y = h * rstd * weight, h = x + residual, rstd = 1 / sqrt(mean(h**2) + eps) of each row.

    x [tokens, dim], weight [dim] of x's type (16-byte aligned).  Returns y; with ``residual``
    (y, h), h rounded to x's type, which the norm is taken of; with ``save`` (y, h, rstd) for
    ``rms_norm_backward``, h being x where there is no residual and rstd fp32 [tokens].
    ``h_out`` takes h and may be x or the residual itself.
    """
    y, h, rstd = _call("rms_norm", stream, x, x, weight, residual, eps, None, bool(save), out, h_out)
    if out is not None:
        y = out
    if h_out is not None:
        h = h_out
    if save:
        return y, (x if h is None else h), rstd
    return y if residual is None else (y, h)


def rms_norm_mx(x, weight, format="e4m3", residual=None, eps=1e-6, h_out=None, stream=None):
    """``rms_norm`` with y as an ``Mx`` of ``format``, rounded once: y, or with ``residual`` (y, h)."""
    data, scale, h, _, dim = _call("rms_norm", stream, x, x, weight, residual, eps, _format(format), False, None, h_out)
    y = _new(Mx, (data, scale, dim, format))
    return y if residual is None else (y, h if h_out is None else h_out)


def rms_norm_backward(dy, h, weight, rstd, dh=None, out=None, stream=None):
    """Gradients of ``rms_norm``: (dx, dweight), from what ``rms_norm(..., save=True)`` returned.

    dx is the gradient of x and of the residual alike; ``dh`` is the gradient that reaches h
    by another way (the residual stream) and is added to it.  ``out`` takes dx and may be dy
    or dh itself.
    """
    dx, dweight = _call("rms_norm_backward", stream, h, dy, h, weight, rstd, dh, out)
    return (dx if out is None else out), dweight


def mx_quantize(x, format="e2m1", transpose=False, stream=None):
    """x [rows, cols] (fp16 or bf16) as an ``Mx``; with ``transpose`` x.T, [cols, rows].

    A block's scale is the power of two at or below its largest magnitude, less the format's
    largest exponent; values are rounded to nearest even and end at the format's largest (a
    block's peak between 6 and 8 scales in e2m1 becomes 6).  A weight [in, out] as ``linear``
    takes it becomes ``mx_linear``'s by ``transpose``, blocks along ``in``.
    """
    data, scale, cols = _call("mx_quantize", stream, x, x, _format(format), bool(transpose))
    return _new(Mx, (data, scale, cols, format))


def mx_dequantize(a, dtype=None, stream=None):
    """The values of an ``Mx`` as fp16 or bf16 (the default), which hold them exactly if
    ``mx_quantize`` made them of that type."""
    data, scale, cols, format = _mx(a, "a")
    return _call("mx_dequantize", stream, data, data, scale, cols, _format(format), _dtype(dtype))


def mx_linear(x, w, bias=None, act=None, residual=None, dtype=None, out=None, stream=None):
    """y = act(x @ w.T + bias) + residual, x [tokens, k] and w [n, k] each an ``Mx`` of one format.

    ``dtype`` (bf16 by default, or fp16) is that of y, ``bias`` [n] and ``residual`` [tokens, n];
    ``act`` as in ``linear``; ``out`` may be the residual itself.  Products and sums are fp32's.

    The gradients straight through the rounding are products of the same kind, of operands
    quantised along the other axis: for y = x @ w with w [k, n]
    ``dx = mx_linear(mx_quantize(dy), mx_quantize(w))`` and
    ``dw = mx_linear(mx_quantize(x, transpose=True), mx_quantize(dy, transpose=True))``.
    """
    data, scale, cols, format = _mx(x, "x")
    w_data, w_scale, w_cols, w_format = _mx(w, "w")
    if cols != w_cols or format != w_format:
        raise ValueError(f"x is [.., {cols}] {format}, w [.., {w_cols}] {w_format}")
    return _call("mx_linear", stream, data, data, scale, w_data, w_scale, cols, _format(format), bias, _act(act), residual,
                 _dtype(dtype), out)
