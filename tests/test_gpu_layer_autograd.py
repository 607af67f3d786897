"""What autograd sees of the layer operators, which it does not run."""
import pytest

import tensor_core_tiled_02_gb300 as tc

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16 = torch.bfloat16


def ones(*shape):
    return torch.ones(*shape, device="cuda", dtype=BF16)


def writers():
    """(what, the tensor it writes, the call)"""
    y, g, a, b = ones(8, 64), ones(8, 64), ones(100), ones(50)
    x, w = ones(8, 64), ones(64, 64)
    return [("linear", y, lambda: tc.linear(x, w, out=y)), ("residual", y, lambda: tc.linear(x, w, residual=y, out=y)),
            ("gated", g, lambda: tc.gated_ffn(x, w, w, w, out=g)), ("clip", a, lambda: tc.clip_grad_norm([b, a], 1.0)),
            ("clip out", b, lambda: tc.clip_grad_norm([ones(50)], 1.0, out=[b]))]


@pytest.mark.parametrize("i", range(5))
def test_written_tensors_change_version(i):
    _, t, call = writers()[i]
    before = t._version
    call()
    assert t._version > before
    # a value saved for a backward pass and then overwritten is noticed
    leaf = torch.ones_like(t, requires_grad=True)
    kept = leaf * 2
    loss = (kept * kept).float().sum()
    alias = kept.detach()
    if t.dim() == 2:
        tc.linear(ones(8, 64), ones(64, 64), out=alias)
    else:
        tc.clip_grad_norm([alias], 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inputs_and_refused_calls_do_not():
    x, w, y = ones(8, 64), ones(64, 64), ones(8, 64)
    tc.linear(x, w)
    tc.linear_backward(y, x, w)
    with pytest.raises(tc.GemmError):
        tc.linear(x, w, out=w[:8])
    with pytest.raises(ValueError):
        tc.linear(x, w, out=ones(9, 64))
    g, out = ones(100), ones(100)
    tc.clip_grad_norm([g], 1.0, out=[out])
    assert [t._version for t in (x, w, y, g)] == [0] * 4


def test_inference_tensors():
    with torch.inference_mode():
        x, w, y = ones(8, 64), ones(64, 64), ones(8, 64)
        tc.linear(x, w, out=y)
        tc.clip_grad_norm([y], 1.0)
    tc.linear(x, w, out=y)
    assert (y == 64).all()
