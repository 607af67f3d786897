"""What autograd sees of the layer operators, which it does not run."""
import warnings

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


def test_operands_that_require_gradients():
    """The call goes through and says that it records no graph; silent where gradients are off."""
    x, w = ones(8, 64), ones(64, 64).requires_grad_(True)
    y = ones(8, 64)
    h, target = ones(8, 64).requires_grad_(True), torch.zeros(8, dtype=torch.int64, device="cuda")
    for call in (lambda: tc.linear(x, w, out=y), lambda: tc.gated_ffn(x, w, w, w), lambda: tc.linear_backward(x, x, w),
                 lambda: tc.linear_cross_entropy(h, x, target)):
        with pytest.warns(UserWarning, match="records no autograd graph"):
            out = call()
        assert not any(t.requires_grad for t in (out if isinstance(out, tuple) else (out,)) if t is not None)
        with warnings.catch_warnings(), torch.no_grad():
            warnings.simplefilter("error")
            call()
    # turned into an error, it leaves the output alone
    y.zero_()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(UserWarning):
            tc.linear(x, w, out=y)
        tc.linear(x, w.detach())
    assert torch.count_nonzero(y) == 0
