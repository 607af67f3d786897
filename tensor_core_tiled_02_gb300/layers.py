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
import operator
import struct

import tensor_core_tiled_02_gb300 as _tc

ACTS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
REDUCTIONS = {"none": 0, "mean": 1, "sum": 2}
# d of one piece of the vocabulary (linear_cross_entropy_backward) takes about this much
LOSS_PIECE_BYTES = 512 << 20
_NO_WORKSPACE = bytes(16)
_DTYPE = operator.attrgetter("dtype")

# torch and what is asked of it on every call, looked up once (importing this module does not import torch)
_torch = None
_dtypes = None
_raw_stream = None


def _lazy():
    global _torch, _dtypes, _raw_stream
    if _torch is None:
        import torch

        _dtypes = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
        # the current stream's handle without building a Stream object, where torch offers it
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _torch = torch
    return _torch


def _side_stream(stream, index):
    """(handle, torch stream) of a stream the caller names."""
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream, stream
    handle = int(stream)
    return handle, (_torch.cuda.ExternalStream(handle, device=index) if handle else _torch.cuda.default_stream(index))


class _Call:
    """The device and stream of one call."""

    __slots__ = ("device", "index", "handle", "stream")

    def __init__(self, tensor, stream):
        self.device = tensor.device
        self.index = tensor.get_device()
        self.stream = None
        if stream is None:
            self.handle = _raw_stream(self.index)
        else:
            self.handle, self.stream = _side_stream(stream, self.index)

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

    def run(self, name, args):
        fn = getattr(_tc.load_library(), name)
        if _torch.cuda.current_device() == self.index:
            rc = fn(args, self.handle)
        else:
            with _torch.cuda.device(self.device):
                rc = fn(args, self.handle)
        if rc != 0:
            raise _tc.GemmError(rc, name)

    def run_with_workspace(self, name, args, *more):
        """`args` lacks its last two fields, the workspace and its size."""
        n = ctypes.c_size_t(0)
        size = name + "_workspace"
        rc = getattr(_tc.load_library(), size)(args + _NO_WORKSPACE, *more, ctypes.byref(n))
        if rc != 0:
            raise _tc.GemmError(rc, size)
        nbytes = n.value
        if nbytes == 0:
            return self.run(name, args + _NO_WORKSPACE)
        ws = self.empty((nbytes,), _torch.uint8)
        self.run(name, args + struct.pack("2q", ws.data_ptr(), nbytes))


def _check(name, t, rows, cols, dtype, index):
    """A [rows, cols] matrix of `dtype` on device `index`; its row stride."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on CUDA device {index}")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return ld if rows > 1 else (cols + 7) // 8 * 8


def _operand(name, t):
    """The operand that fixes a call's type and device: rows, columns, row stride."""
    if t.dim() != 2 or _dtypes.get(t.dtype, 2) == 2:
        raise ValueError(f"{name} must be a 2-D fp16 or bf16 tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return rows, cols, ld if rows > 1 else (cols + 7) // 8 * 8


def _vector(name, t, n, dtype, index):
    if t.dtype is not dtype or t.shape != (n,) or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} [{n}] tensor on CUDA device {index}")
    return t.data_ptr()


def _act(act):
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(k for k in ACTS if k)}, got {act!r}")
    return code


def _pitch(cols):
    return (cols + 7) // 8 * 8


def linear(x, w, bias=None, act=None, residual=None, save_preact=False, out=None, stream=None):
    """y = act(x @ w + bias) + residual, x [tokens, k], w [k, n].

    ``act``: None, "relu", "silu", "gelu" (erf) or "gelu_tanh"; ``bias`` [n] and
    ``residual`` [tokens, n] of x's type.  ``out`` may be the residual itself.
    With ``save_preact`` returns (y, x @ w + bias), the latter for ``linear_backward``.
    """
    torch = _lazy()
    code = _act(act)
    tokens, k, ldx = _operand("x", x)
    dt, dev = x.dtype, x.get_device()
    if w.dim() != 2 or w.shape[1] < 1 or k < 1:
        raise ValueError("w must be 2-D and not empty")
    n = w.shape[1]
    ldw = _check("w", w, k, n, dt, dev)
    pbias = _vector("bias", bias, n, dt, dev) if bias is not None else 0
    ldr = _check("residual", residual, tokens, n, dt, dev) if residual is not None else 0
    call = _Call(x, stream)
    y = out if out is not None else call.matrix(tokens, n, dt)
    ldy = _check("out", y, tokens, n, dt, dev) if out is not None else _pitch(n)
    pre = call.matrix(tokens, n, dt) if save_preact else None
    call.run("linear_forward", struct.pack(
        "16q", x.data_ptr(), w.data_ptr(), pbias, residual.data_ptr() if residual is not None else 0, y.data_ptr(),
        pre.data_ptr() if save_preact else 0, ldx, ldw, ldr, ldy, _pitch(n), tokens, k, n, _dtypes[dt], code))
    return (y, pre) if save_preact else y


def linear_backward(dy, x, w, act=None, preact=None, bias=False, stream=None):
    """Gradients of ``linear``: (dx, dw, dbias), dbias None unless ``bias``.

    ``preact`` is what ``linear(..., save_preact=True)`` returned; it may be None
    when ``act`` is.  The residual's gradient is ``dy`` itself.
    """
    torch = _lazy()
    code = _act(act)
    tokens, k, ldx = _operand("x", x)
    dt, dev = x.dtype, x.get_device()
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

    call.run_with_workspace("linear_backward", struct.pack(
        "18q", dy.data_ptr(), x.data_ptr(), w.data_ptr(), preact.data_ptr() if code else 0, dx.data_ptr(), dw.data_ptr(),
        dbias.data_ptr() if bias else 0, lddy, ldx, ldw, ldp, _pitch(k), _pitch(n), tokens, k, n, _dtypes[dt], code))
    return dx, dw, dbias


def gated_ffn(x, w_gate, w_up, w_down, act="silu", residual=None, save=False, out=None, stream=None):
    """y = (act(x @ w_gate) * (x @ w_up)) @ w_down + residual.

    x [tokens, dim], w_gate and w_up [dim, ffn], w_down [ffn, dim_out].  ``out`` may be
    the residual itself.  With ``save`` returns (y, gate, up, hidden): x @ w_gate,
    x @ w_up and act(gate) * up, which ``gated_ffn_backward`` reads.
    """
    _lazy()
    code = _act(act)
    tokens, dim, ldx = _operand("x", x)
    dt, dev = x.dtype, x.get_device()
    if w_gate.dim() != 2 or w_down.dim() != 2 or not (dim and w_gate.shape[1] and w_down.shape[1]):
        raise ValueError("the weights must be 2-D and not empty")
    ffn, dim_out = w_gate.shape[1], w_down.shape[1]
    ldg, ldu = _check("w_gate", w_gate, dim, ffn, dt, dev), _check("w_up", w_up, dim, ffn, dt, dev)
    ldd = _check("w_down", w_down, ffn, dim_out, dt, dev)
    ldr = _check("residual", residual, tokens, dim_out, dt, dev) if residual is not None else 0
    call = _Call(x, stream)
    y = out if out is not None else call.matrix(tokens, dim_out, dt)
    ldy = _check("out", y, tokens, dim_out, dt, dev) if out is not None else _pitch(dim_out)
    hidden = call.matrix(tokens, ffn, dt)
    gate, up = (call.matrix(tokens, ffn, dt), call.matrix(tokens, ffn, dt)) if save else (None, None)
    ldh = _pitch(ffn)
    call.run("gated_ffn_forward", struct.pack(
        "24q", x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
        residual.data_ptr() if residual is not None else 0, y.data_ptr(), hidden.data_ptr(),
        gate.data_ptr() if save else 0, up.data_ptr() if save else 0, ldx, ldg, ldu, ldd, ldr, ldy, ldh, ldh, ldh,
        tokens, dim, ffn, dim_out, _dtypes[dt], code))
    return (y, gate, up, hidden) if save else y


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, gate, up, hidden, act="silu", stream=None):
    """Gradients of ``gated_ffn``: (dx, dw_gate, dw_up, dw_down), from what
    ``gated_ffn(..., save=True)`` returned.  The residual's gradient is ``dy`` itself."""
    torch = _lazy()
    code = _act(act)
    tokens, dim, ldx = _operand("x", x)
    dt, dev = x.dtype, x.get_device()
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
    call.run_with_workspace("gated_ffn_backward", struct.pack(
        "30q", *[t.data_ptr() for t in (dy, x, w_gate, w_up, w_down, gate, up, hidden) + grads], *lds,
        _pitch(dim), _pitch(ffn), _pitch(ffn), _pitch(dim_out), tokens, dim, ffn, dim_out, _dtypes[dt], code))
    return grads


def _loss_operands(h, w, target, reduction):
    torch = _lazy()
    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)}, got {reduction!r}")
    tokens, dim, ldh = _operand("h", h)
    if w.dim() != 2 or w.shape[0] < 1 or dim < 1:
        raise ValueError("w must be [vocabulary, features] and not empty")
    dev, vocab = h.get_device(), w.shape[0]
    ldw = _check("w", w, vocab, dim, h.dtype, dev)
    return ldh, ldw, tokens, dim, vocab, _vector("target", target, tokens, torch.int64, dev)


def linear_cross_entropy(h, w, target, ignore_index=-100, reduction="mean", stream=None):
    """The cross entropy of the logits h @ w.T against ``target``: (loss, lse), fp32.

    h [tokens, dim], w [vocabulary, dim], target [tokens] int64.  ``loss`` is one value
    ("mean": over the targets that count, 0 when none does; "sum") or [tokens] ("none", 0
    where the target is ``ignore_index``); ``lse`` [tokens] is the logits' log-sum-exp,
    which the backward pass reads.  The logits never reach memory.
    """
    torch = _lazy()
    ldh, ldw, tokens, dim, vocab, ptarget = _loss_operands(h, w, target, reduction)
    call = _Call(h, stream)
    loss = call.empty((tokens,) if reduction == "none" else (), torch.float32)
    lse = call.empty((tokens,), torch.float32)

    call.run_with_workspace("linear_cross_entropy", struct.pack(
        "13q", h.data_ptr(), w.data_ptr(), ptarget, loss.data_ptr(), lse.data_ptr(), ldh, ldw, tokens, dim, vocab,
        _dtypes[h.dtype], ignore_index, REDUCTIONS[reduction]))
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
    ldh, ldw, tokens, dim, vocab, ptarget = _loss_operands(h, w, target, reduction)
    dev = h.get_device()
    each = reduction == "none"
    if grad_loss.dtype is not torch.float32 or grad_loss.get_device() != dev or not grad_loss.is_contiguous() or (
            grad_loss.numel() != (tokens if each else 1)):
        raise ValueError(f"grad_loss must be fp32 on CUDA device {dev}, {'[tokens]' if each else 'one value'}")
    plse = _vector("lse", lse, tokens, torch.float32, dev)
    if piece is None:
        piece = max(256, LOSS_PIECE_BYTES // (2 * max(tokens, 1)) // 256 * 256)
    call = _Call(h, stream)
    dh, dw = call.matrix(tokens, dim, h.dtype), call.matrix(vocab, dim, h.dtype)

    call.run_with_workspace("linear_cross_entropy_backward", struct.pack(
        "17q", h.data_ptr(), w.data_ptr(), ptarget, plse, grad_loss.data_ptr(), dh.data_ptr(), dw.data_ptr(), ldh, ldw,
        _pitch(dim), _pitch(dim), tokens, dim, vocab, _dtypes[h.dtype], ignore_index, REDUCTIONS[reduction]), int(piece))
    return dh, dw


def clip_grad_norm(grads, max_norm, out=None, eps=1e-6, stream=None):
    """Scales gradients by min(1, max_norm / (norm + eps)), norm their global 2-norm.

    ``grads``: dense CUDA tensors, fp16, bf16 or fp32, of any shapes, types mixed.  In
    place, or into ``out`` (tensors of the same sizes and types).  Returns the norm
    before clipping: one fp32 value on the device, nothing waits for it.
    """
    torch = _lazy()
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    # hundreds of tensors are common: each question is put to all of them in one sweep
    tensor = torch.Tensor
    call = _Call(grads[0], stream)
    out = grads if out is None else list(out)
    kinds, counts = list(map(_DTYPE, grads)), list(map(tensor.numel, grads))
    for name, ts in (("gradients", grads),) if out is grads else (("gradients", grads), ("out", out)):
        if set(map(tensor.get_device, ts)) != {call.index} or call.index < 0 or not all(map(tensor.is_contiguous, ts)):
            raise ValueError(f"{name} must be dense tensors on one CUDA device")
    if out is not grads and (list(map(_DTYPE, out)) != kinds or list(map(tensor.numel, out)) != counts):
        raise ValueError("out must have the gradients' sizes and types")
    try:
        codes = array.array("i", [_dtypes[k] for k in kinds])
    except KeyError as e:
        raise ValueError(f"gradients must be fp16, bf16 or fp32, got {e.args[0]}") from None
    src = array.array("q", list(map(tensor.data_ptr, grads)))
    dst = src if out is grads else array.array("q", list(map(tensor.data_ptr, out)))
    counts = array.array("q", counts)
    norm = call.empty((), torch.float32)
    n = ctypes.c_size_t(0)
    rc = _tc.load_library().grad_clip_workspace(len(grads), ctypes.byref(n))
    if rc != 0:
        raise _tc.GemmError(rc, "grad_clip_workspace")
    ws = call.empty((n.value,), torch.uint8)
    call.run("grad_clip", struct.pack("7q2dq", src.buffer_info()[0], dst.buffer_info()[0], counts.buffer_info()[0],
                                      codes.buffer_info()[0], norm.data_ptr(), ws.data_ptr(), len(grads), max_norm, eps,
                                      n.value))
    return norm
