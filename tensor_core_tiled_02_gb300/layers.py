"""Python binding of the layer operators (``include/layer_ops.h``).

Argument marshalling only, as for ``matmul``: tensors in, tensors out, every
step in the CUDA library.  Activations are [tokens, features], weights [in,
out] as ``matmul`` takes them, the vocabulary's weight [vocabulary, features].
Operands are fp16 or bf16, of one type per call; rows may be strided (a view
of wider rows) as long as a row's entries are contiguous, row strides are
multiples of 8 and addresses multiples of 16 bytes.

Calls are asynchronous on ``stream`` (default: torch's current stream of the
tensors' device).  Outputs and workspaces that a call allocates belong to that
stream; tensors handed in must be ready on it, and live until it has passed.
The calls do not record an autograd graph: each forward pass has its
``_backward``.  ``ValueError`` for tensors a call cannot take, ``GemmError``
for a status of the library.
"""
from __future__ import annotations

import array
import ctypes
import struct

import tensor_core_tiled_02_gb300 as _tc

ACTS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
REDUCTIONS = {"none": 0, "mean": 1, "sum": 2}
# d of one piece of the vocabulary (linear_cross_entropy_backward) takes about this much
LOSS_PIECE_BYTES = 256 << 20

_torch = None
_dtypes = None


def _lazy():
    global _torch, _dtypes
    if _torch is None:
        import torch

        _dtypes = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
        _torch = torch
    return _torch


class _Call:
    """The device and stream of one call."""

    def __init__(self, tensor, stream):
        torch = _torch
        self.device = tensor.device
        self.stream = None
        if stream is None:
            self.handle = torch.cuda.current_stream(self.device).cuda_stream
        elif hasattr(stream, "cuda_stream"):
            self.handle = stream.cuda_stream
            self.stream = stream
        else:
            self.handle = int(stream)
            self.stream = torch.cuda.ExternalStream(self.handle, device=self.device) if self.handle else (
                torch.cuda.default_stream(self.device))

    def empty(self, shape, dtype):
        """Memory that belongs to the call's stream."""
        if self.stream is None:
            return _torch.empty(shape, dtype=dtype, device=self.device)
        with _torch.cuda.stream(self.stream):
            return _torch.empty(shape, dtype=dtype, device=self.device)

    def matrix(self, rows, cols, dtype):
        """A matrix whose row stride the library takes: a multiple of 8."""
        if cols % 8 == 0:
            return self.empty((rows, cols), dtype)
        return self.empty((rows, (cols + 7) // 8 * 8), dtype)[:, :cols]

    def run(self, name, args, *more):
        fn = getattr(_tc.load_library(), name)
        if _torch.cuda.current_device() == self.device.index:
            rc = fn(args, *more)
        else:
            with _torch.cuda.device(self.device):
                rc = fn(args, *more)
        if rc != 0:
            raise _tc.GemmError(rc, name)


def _check(name, t, rows, cols, dtype, device):
    """A [rows, cols] CUDA matrix of `dtype`; its row stride."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{name} must be [{rows}, {cols}], got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return _stride(name, t)


def _stride(name, t):
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 7) // 8 * 8


def _operand(name, t):
    """The operand that fixes a call's type and device."""
    if t.dim() != 2 or _dtypes.get(t.dtype, 2) == 2:
        raise ValueError(f"{name} must be a 2-D fp16 or bf16 tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return _stride(name, t)


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(k for k in ACTS if k)}, got {act!r}")
    return ACTS[act]


def _size(name, args, *more):
    n = ctypes.c_size_t(0)
    rc = getattr(_tc.load_library(), name)(args, *more, ctypes.byref(n))
    if rc != 0:
        raise _tc.GemmError(rc, name)
    return n.value


def linear(x, w, bias=None, act=None, residual=None, save_preact=False, out=None, stream=None):
    """y = act(x @ w + bias) + residual, x [tokens, k], w [k, n].

    ``act``: None, "relu", "silu", "gelu" (erf) or "gelu_tanh"; ``bias`` [n] and
    ``residual`` [tokens, n] of x's type.  ``out`` may be the residual itself.
    With ``save_preact`` returns (y, x @ w + bias), the latter for ``linear_backward``.
    """
    torch = _lazy()
    code = _act(act)
    ldx = _operand("x", x)
    dt, dev = x.dtype, x.device
    tokens, k = x.shape
    if w.dim() != 2:
        raise ValueError("w must be 2-D")
    n = w.shape[1]
    ldw = _check("w", w, k, n, dt, dev)
    if bias is not None and (bias.dtype != dt or bias.shape != (n,) or bias.device != dev or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous {dt} [{n}] tensor on {dev}")
    ldr = _check("residual", residual, tokens, n, dt, dev) if residual is not None else 0
    call = _Call(x, stream)
    y = out if out is not None else call.matrix(tokens, n, dt)
    ldy = _check("out", y, tokens, n, dt, dev)
    pre = call.matrix(tokens, n, dt) if save_preact else None
    if tokens and k and n:
        call.run("linear_forward", struct.pack(
            "16q", x.data_ptr(), w.data_ptr(), bias.data_ptr() if bias is not None else 0,
            residual.data_ptr() if residual is not None else 0, y.data_ptr(), pre.data_ptr() if save_preact else 0,
            ldx, ldw, ldr, ldy, _stride("preact", pre) if save_preact else 0, tokens, k, n, _dtypes[dt], code),
            call.handle)
    elif tokens and n:
        raise ValueError("x and w must have k >= 1")
    return (y, pre) if save_preact else y


def linear_backward(dy, x, w, act=None, preact=None, bias=False, stream=None):
    """Gradients of ``linear``: (dx, dw, dbias), dbias None unless ``bias``.

    ``preact`` is what ``linear(..., save_preact=True)`` returned; it may be None
    when ``act`` is.  The residual's gradient is ``dy`` itself.
    """
    torch = _lazy()
    code = _act(act)
    ldx = _operand("x", x)
    dt, dev = x.dtype, x.device
    tokens, k = x.shape
    if w.dim() != 2 or w.shape[1] < 1 or k < 1:
        raise ValueError("w must be 2-D and not empty")
    n = w.shape[1]
    ldw = _check("w", w, k, n, dt, dev)
    lddy = _check("dy", dy, tokens, n, dt, dev)
    if code and preact is None:
        raise ValueError("preact is needed for the slope of the activation")
    ldp = _check("preact", preact, tokens, n, dt, dev) if code else 0
    call = _Call(x, stream)
    dx, dw = call.matrix(tokens, k, dt), call.matrix(k, n, dt)
    dbias = call.empty((n,), dt) if bias else None

    def pack(ws, nbytes):
        return struct.pack("20q", dy.data_ptr(), x.data_ptr(), w.data_ptr(), preact.data_ptr() if code else 0,
                           dx.data_ptr(), dw.data_ptr(), dbias.data_ptr() if bias else 0, ws, lddy, ldx, ldw, ldp,
                           _stride("dx", dx), _stride("dw", dw), tokens, k, n, _dtypes[dt], code, nbytes)

    nbytes = _size("linear_backward_workspace", pack(0, 0))
    ws = call.empty((nbytes,), torch.uint8) if nbytes else None
    call.run("linear_backward", pack(ws.data_ptr() if nbytes else 0, nbytes), call.handle)
    return dx, dw, dbias


def gated_ffn(x, w_gate, w_up, w_down, act="silu", residual=None, save=False, out=None, stream=None):
    """y = (act(x @ w_gate) * (x @ w_up)) @ w_down + residual.

    x [tokens, dim], w_gate and w_up [dim, ffn], w_down [ffn, dim_out].  ``out`` may be
    the residual itself.  With ``save`` returns (y, gate, up, hidden): x @ w_gate,
    x @ w_up and act(gate) * up, which ``gated_ffn_backward`` reads.
    """
    _lazy()
    code = _act(act)
    ldx = _operand("x", x)
    dt, dev = x.dtype, x.device
    tokens, dim = x.shape
    if w_gate.dim() != 2 or w_down.dim() != 2 or not (dim and w_gate.shape[1] and w_down.shape[1]):
        raise ValueError("the weights must be 2-D and not empty")
    ffn, dim_out = w_gate.shape[1], w_down.shape[1]
    ldg, ldu = _check("w_gate", w_gate, dim, ffn, dt, dev), _check("w_up", w_up, dim, ffn, dt, dev)
    ldd = _check("w_down", w_down, ffn, dim_out, dt, dev)
    ldr = _check("residual", residual, tokens, dim_out, dt, dev) if residual is not None else 0
    call = _Call(x, stream)
    y = out if out is not None else call.matrix(tokens, dim_out, dt)
    ldy = _check("out", y, tokens, dim_out, dt, dev)
    hidden = call.matrix(tokens, ffn, dt)
    gate, up = (call.matrix(tokens, ffn, dt), call.matrix(tokens, ffn, dt)) if save else (None, None)
    ldh = _stride("hidden", hidden)
    call.run("gated_ffn_forward", struct.pack(
        "24q", x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
        residual.data_ptr() if residual is not None else 0, y.data_ptr(), hidden.data_ptr(),
        gate.data_ptr() if save else 0, up.data_ptr() if save else 0, ldx, ldg, ldu, ldd, ldr, ldy, ldh, ldh, ldh,
        tokens, dim, ffn, dim_out, _dtypes[dt], code), call.handle)
    return (y, gate, up, hidden) if save else y


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, gate, up, hidden, act="silu", stream=None):
    """Gradients of ``gated_ffn``: (dx, dw_gate, dw_up, dw_down), from what
    ``gated_ffn(..., save=True)`` returned.  The residual's gradient is ``dy`` itself."""
    torch = _lazy()
    code = _act(act)
    ldx = _operand("x", x)
    dt, dev = x.dtype, x.device
    tokens, dim = x.shape
    if w_gate.dim() != 2 or w_down.dim() != 2 or not (dim and w_gate.shape[1] and w_down.shape[1]):
        raise ValueError("the weights must be 2-D and not empty")
    ffn, dim_out = w_gate.shape[1], w_down.shape[1]
    lds = [_check("dy", dy, tokens, dim_out, dt, dev), ldx, _check("w_gate", w_gate, dim, ffn, dt, dev),
           _check("w_up", w_up, dim, ffn, dt, dev), _check("w_down", w_down, ffn, dim_out, dt, dev),
           _check("gate", gate, tokens, ffn, dt, dev), _check("up", up, tokens, ffn, dt, dev),
           _check("hidden", hidden, tokens, ffn, dt, dev)]
    call = _Call(x, stream)
    grads = (call.matrix(tokens, dim, dt), call.matrix(dim, ffn, dt), call.matrix(dim, ffn, dt),
             call.matrix(ffn, dim_out, dt))
    ptrs = [t.data_ptr() for t in (dy, x, w_gate, w_up, w_down, gate, up, hidden) + grads]
    rest = lds + [_stride("gradient", g) for g in grads] + [tokens, dim, ffn, dim_out, _dtypes[dt], code]

    def pack(ws, nbytes):
        return struct.pack("32q", *ptrs, ws, *rest, nbytes)

    nbytes = _size("gated_ffn_backward_workspace", pack(0, 0))
    ws = call.empty((nbytes,), torch.uint8) if nbytes else None
    call.run("gated_ffn_backward", pack(ws.data_ptr() if nbytes else 0, nbytes), call.handle)
    return grads


def _loss_operands(h, w, target, reduction):
    torch = _lazy()
    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)}, got {reduction!r}")
    ldh = _operand("h", h)
    tokens, dim = h.shape
    if w.dim() != 2 or w.shape[0] < 1 or dim < 1:
        raise ValueError("w must be [vocabulary, features] and not empty")
    ldw = _check("w", w, w.shape[0], dim, h.dtype, h.device)
    if target.dtype != torch.int64 or target.shape != (tokens,) or target.device != h.device or not target.is_contiguous():
        raise ValueError(f"target must be a contiguous int64 [{tokens}] tensor on {h.device}")
    return ldh, ldw, tokens, dim, w.shape[0]


def linear_cross_entropy(h, w, target, ignore_index=-100, reduction="mean", stream=None):
    """The cross entropy of the logits h @ w.T against ``target``: (loss, lse), fp32.

    h [tokens, dim], w [vocabulary, dim], target [tokens] int64.  ``loss`` is one value
    ("mean": over the targets that count, 0 when none does; "sum") or [tokens] ("none", 0
    where the target is ``ignore_index``); ``lse`` [tokens] is the logits' log-sum-exp,
    which the backward pass reads.  The logits never reach memory.
    """
    torch = _lazy()
    ldh, ldw, tokens, dim, vocab = _loss_operands(h, w, target, reduction)
    call = _Call(h, stream)
    loss = call.empty((tokens,) if reduction == "none" else (), torch.float32)
    lse = call.empty((tokens,), torch.float32)

    def pack(ws, nbytes):
        return struct.pack("15q", h.data_ptr(), w.data_ptr(), target.data_ptr(), loss.data_ptr(), lse.data_ptr(), ws,
                           ldh, ldw, tokens, dim, vocab, _dtypes[h.dtype], ignore_index, REDUCTIONS[reduction], nbytes)

    nbytes = _size("linear_cross_entropy_workspace", pack(0, 0))
    ws = call.empty((nbytes,), torch.uint8) if nbytes else None
    call.run("linear_cross_entropy", pack(ws.data_ptr() if nbytes else 0, nbytes), call.handle)
    return loss, lse


def linear_cross_entropy_backward(grad_loss, h, w, target, lse, ignore_index=-100, reduction="mean", piece=None,
                                  stream=None):
    """Gradients of ``linear_cross_entropy``: (dh, dw).

    ``grad_loss`` is the loss's gradient, fp32 on the device: one value, or [tokens]
    for reduction "none".  The logits are computed again, ``piece`` words of the
    vocabulary at a time (a multiple of 256; by default what fits LOSS_PIECE_BYTES).
    h has to be finite in ignored rows too: their weight in dw is 0, not absent.
    """
    torch = _lazy()
    ldh, ldw, tokens, dim, vocab = _loss_operands(h, w, target, reduction)
    dev = h.device
    each = reduction == "none"
    if grad_loss.dtype != torch.float32 or grad_loss.device != dev or grad_loss.numel() != (tokens if each else 1) or (
            not grad_loss.is_contiguous()):
        raise ValueError(f"grad_loss must be fp32 on {dev}, {'[tokens]' if each else 'one value'}")
    if lse.dtype != torch.float32 or lse.shape != (tokens,) or lse.device != dev or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous fp32 [{tokens}] tensor on {dev}")
    if piece is None:
        piece = max(256, LOSS_PIECE_BYTES // (2 * max(tokens, 1)) // 256 * 256)
    call = _Call(h, stream)
    dh, dw = call.matrix(tokens, dim, h.dtype), call.matrix(vocab, dim, h.dtype)

    def pack(ws, nbytes):
        return struct.pack("19q", h.data_ptr(), w.data_ptr(), target.data_ptr(), lse.data_ptr(), grad_loss.data_ptr(),
                           dh.data_ptr(), dw.data_ptr(), ws, ldh, ldw, _stride("dh", dh), _stride("dw", dw), tokens,
                           dim, vocab, _dtypes[h.dtype], ignore_index, REDUCTIONS[reduction], nbytes)

    nbytes = _size("linear_cross_entropy_backward_workspace", pack(0, 0), int(piece))
    ws = call.empty((nbytes,), torch.uint8) if nbytes else None
    call.run("linear_cross_entropy_backward", pack(ws.data_ptr() if nbytes else 0, nbytes), call.handle)
    return dh, dw


def clip_grad_norm(grads, max_norm, out=None, eps=1e-6, stream=None):
    """Scales gradients by min(1, max_norm / (norm + eps)), norm their global 2-norm.

    ``grads``: dense CUDA tensors, fp16, bf16 or fp32, of any shapes, types mixed.  In
    place, or into ``out`` (tensors of the same sizes and types).  Returns the norm
    before clipping: one fp32 value on the device, nothing waits for it.
    """
    torch = _lazy()
    grads = list(grads)
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError(f"{len(grads)} gradients, but {len(outs)} outputs")
    if not grads:
        raise ValueError("no gradients")
    dev = grads[0].device
    codes = []
    for g, o in zip(grads, outs):
        code = _dtypes.get(g.dtype)
        if code is None or not g.is_cuda or g.device != dev or not g.is_contiguous():
            raise ValueError("gradients must be dense fp16, bf16 or fp32 tensors on one CUDA device")
        if o is not g and (o.dtype != g.dtype or o.shape != g.shape or o.device != dev or not o.is_contiguous()):
            raise ValueError("out must match the gradients")
        codes.append(code)
    call = _Call(grads[0], stream)
    norm = call.empty((), torch.float32)
    src = array.array("q", [g.data_ptr() for g in grads])
    dst = src if out is None else array.array("q", [o.data_ptr() for o in outs])
    count = array.array("q", [g.numel() for g in grads])
    kinds = array.array("i", codes)
    nbytes = _size("grad_clip_workspace", len(grads))
    ws = call.empty((nbytes,), torch.uint8)
    call.run("grad_clip", struct.pack("7q2dq", src.buffer_info()[0], dst.buffer_info()[0], count.buffer_info()[0],
                                      kinds.buffer_info()[0], norm.data_ptr(), ws.data_ptr(), len(grads), max_norm, eps,
                                      nbytes), call.handle)
    return norm
