"""The layer operators on torch tensors (``include/layer_ops.h``).

Tensors in, tensors out, every step in the CUDA library; the argument checks
and the marshalling are native too (``csrc/layer_binding.cpp``, built with the
library).  Activations are [tokens, features], weights [in, out] as ``matmul``
takes them, the vocabulary's weight [vocabulary, features].  Operands are fp16
or bf16, of one type per call; rows may be strided (a view of wider rows) as
long as a row's entries are contiguous, row strides are multiples of 8 and
addresses multiples of 16 bytes.

Calls are asynchronous on ``stream`` (default: torch's current stream of the
tensors' device).  Outputs and workspaces that a call allocates belong to that
stream; tensors handed in must be ready on it, and live until it has passed.
The calls do not record an autograd graph: each forward pass has its
``_backward``, and a tensor that requires a gradient is warned of unless gradients
are off.  Tensors written in place or through ``out`` change their version.  ``ValueError`` for tensors a call cannot take, ``GemmError``
for a status of the library.
"""
from __future__ import annotations

import ctypes
import importlib
import operator
import threading

import tensor_core_tiled_02_gb300 as _tc

ACTS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
REDUCTIONS = {"none": 0, "mean": 1, "sum": 2}
# d of one piece of the vocabulary (linear_cross_entropy_backward) takes at most about this much
LOSS_PIECE_BYTES = 512 << 20

# the library's entry points, in the order the binding takes them
_ENTRIES = ("linear_forward", "linear_backward", "linear_backward_workspace", "gated_ffn_forward", "gated_ffn_backward",
            "gated_ffn_backward_workspace", "linear_cross_entropy", "linear_cross_entropy_workspace",
            "linear_cross_entropy_backward", "linear_cross_entropy_backward_workspace", "grad_clip",
            "grad_clip_workspace")
_lock = threading.Lock()
_bound = None


def _native():
    """The binding, loaded and bound to the library on first use.  Raises if either is not built."""
    global _bound
    if _bound is None:
        with _lock:
            if _bound is None:
                import torch  # noqa: F401  (its libraries first: the binding is linked against them)

                lib = _tc.load_library()
                try:
                    mod = importlib.import_module("tensor_core_tiled_02_gb300._layers")
                except ImportError as e:
                    raise RuntimeError("the layer operators' binding is missing or was built for another torch: "
                                       "build it with `python -m tensor_core_tiled_02_gb300.build`") from e
                mod.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in _ENTRIES))
                _bound = mod
    return _bound


def _on(stream, tensor):
    """The torch stream context of a stream the caller names (a stream or a handle)."""
    import torch

    if not isinstance(tensor, torch.Tensor) or not tensor.is_cuda:
        raise ValueError("every tensor must be a CUDA tensor")
    if not hasattr(stream, "cuda_stream"):
        try:
            handle = operator.index(stream)
        except TypeError:
            raise ValueError(f"stream must be a stream or its handle, got {stream!r}") from None
        stream = (torch.cuda.ExternalStream(handle, device=tensor.device) if handle
                  else torch.cuda.default_stream(tensor.device))
    if stream.device != tensor.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {tensor.device}")
    return torch.cuda.stream(stream)


def _call(name, stream, tensor, *args):
    fn = getattr(_bound or _native(), name)
    if stream is None:
        r = fn(*args)
    else:
        with _on(stream, tensor):
            r = fn(*args)
    if type(r) is int:
        raise _tc.GemmError(r, name)
    return r


def _act(act):
    code = ACTS.get(act) if act is None or isinstance(act, str) else None
    if code is None:
        raise ValueError(f"act must be one of {sorted(k for k in ACTS if k)}, got {act!r}")
    return code


def _reduction(reduction):
    code = REDUCTIONS.get(reduction) if isinstance(reduction, str) else None
    if code is None:
        raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)}, got {reduction!r}")
    return code


def linear(x, w, bias=None, act=None, residual=None, save_preact=False, out=None, stream=None):
    """y = act(x @ w + bias) + residual, x [tokens, k], w [k, n].

    ``act``: None, "relu", "silu", "gelu" (erf) or "gelu_tanh"; ``bias`` [n] and
    ``residual`` [tokens, n] of x's type.  ``out`` may be the residual itself.
    With ``save_preact`` returns (y, x @ w + bias), the latter for ``linear_backward``.
    """
    return _call("linear", stream, x, x, w, bias, _act(act), residual, bool(save_preact), out)


def linear_backward(dy, x, w, act=None, preact=None, bias=False, stream=None):
    """Gradients of ``linear``: (dx, dw, dbias), dbias None unless ``bias``.

    ``preact`` is what ``linear(..., save_preact=True)`` returned; it may be None
    when ``act`` is.  The residual's gradient is ``dy`` itself.
    """
    return _call("linear_backward", stream, x, dy, x, w, _act(act), preact, bool(bias))


def gated_ffn(x, w_gate, w_up, w_down, act="silu", residual=None, save=False, out=None, stream=None):
    """y = (act(x @ w_gate) * (x @ w_up)) @ w_down + residual.

    x [tokens, dim], w_gate and w_up [dim, ffn], w_down [ffn, dim_out].  ``out`` may be
    the residual itself.  With ``save`` returns (y, gate, up, hidden): x @ w_gate,
    x @ w_up and act(gate) * up, which ``gated_ffn_backward`` reads.  The second product
    takes hidden rounded to x's type: in fp16 above 65504 it is infinite, kept or not.
    """
    return _call("gated_ffn", stream, x, x, w_gate, w_up, w_down, _act(act), residual, bool(save), out)


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, gate, up, hidden, act="silu", stream=None):
    """Gradients of ``gated_ffn``: (dx, dw_gate, dw_up, dw_down), from what
    ``gated_ffn(..., save=True)`` returned.  The residual's gradient is ``dy`` itself."""
    return _call("gated_ffn_backward", stream, x, dy, x, w_gate, w_up, w_down, gate, up, hidden, _act(act))


def linear_cross_entropy(h, w, target, ignore_index=-100, reduction="mean", stream=None):
    """The cross entropy of the logits h @ w.T against ``target``: (loss, lse), fp32.

    h [tokens, dim], w [vocabulary, dim], target [tokens] int64.  ``loss`` is one value
    ("mean": over the targets that count, 0 when none does; "sum") or [tokens] ("none", 0
    where the target is ``ignore_index``); ``lse`` [tokens] is the logits' log-sum-exp,
    which the backward pass reads.  The logits never reach memory.
    """
    return _call("linear_cross_entropy", stream, h, h, w, target, ignore_index, _reduction(reduction))


def linear_cross_entropy_backward(grad_loss, h, w, target, lse, ignore_index=-100, reduction="mean", piece=None,
                                  stream=None):
    """Gradients of ``linear_cross_entropy``: (dh, dw).

    ``grad_loss`` is the loss's gradient, fp32 on the device: one value, or [tokens]
    for reduction "none".  The logits are computed again, ``piece`` words of the
    vocabulary at a time (a multiple of 256; by default what fits LOSS_PIECE_BYTES).
    In fp16 with reduction "none" every row of dh keeps its own precision, however far the
    rows' gradients lie apart, at twice the memory for a piece.
    h has to be finite in ignored rows too: their weight in dw is 0, not absent.
    """
    if piece is None:
        import torch

        if not isinstance(h, torch.Tensor) or h.dim() != 2:
            raise ValueError("h must be a 2-D fp16 or bf16 tensor")
        copies = 2 if reduction == "none" and h.dtype == torch.float16 else 1
        piece = max(256, LOSS_PIECE_BYTES // (2 * copies * max(h.shape[0], 1)) // 256 * 256)
    return _call("linear_cross_entropy_backward", stream, h, grad_loss, h, w, target, lse, ignore_index,
                 _reduction(reduction), piece)


def clip_grad_norm(grads, max_norm, out=None, eps=1e-6, stream=None):
    """Scales gradients by min(1, max_norm / (norm + eps)), norm their global 2-norm.

    ``grads``: dense CUDA tensors, fp16, bf16 or fp32, of any shapes, types mixed.  In
    place, or into ``out`` (tensors of the same sizes and types).  Returns the norm
    before clipping: one fp32 value on the device, nothing waits for it.  Squares are
    summed in fp32: a norm above 1e19 comes out infinite and scales by 0.
    """
    try:
        grads, out = list(grads), None if out is None else list(out)
    except TypeError:
        raise ValueError("gradients and out must be lists of tensors") from None
    return _call("clip_grad_norm", stream, grads[0] if grads else None, grads, max_norm, out, eps)
