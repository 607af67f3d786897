"""Arguments of the layer operators that no tensor has but a caller of the C ABI can
pass: refused on the host, before any CUDA call.  No compute call is made here."""
import pytest

import tensor_core_tiled_02_gb300 as tc
from test_layer_abi import ALIAS, ALIGN, DIM, GATED, LINEAR, LINEAR_GRAD, LOSS, LOSS_GRAD, P, built  # noqa: F401  (built: a fixture)


@pytest.fixture(scope="module")
def lib(built):  # noqa: F811
    return tc.load_library()


# a row stride whose bytes pass 64 bits: 2^62 elements of 2 bytes are -2^63
@pytest.mark.parametrize("ld", [1 << 39, 1 << 62, (1 << 62) + 128, (1 << 63) - 8], ids=hex)
@pytest.mark.parametrize("args,entry,names", [
    (LINEAR, "linear_forward", ("ldx", "ldw", "ldr", "ldy", "ldp")),
    (LINEAR_GRAD, "linear_backward", ("lddy", "ldx", "ldw", "ldp", "lddx", "lddw")),
    (GATED, "gated_ffn_forward", ("ldx", "ldg", "ldu", "ldd", "ldr", "ldy", "ldh", "ld_gate", "ld_up")),
    (LOSS, "linear_cross_entropy", ("ldh", "ldw")),
    (LOSS_GRAD, "linear_cross_entropy_backward", ("ldh", "ldw", "lddh", "lddw"))], ids=lambda a: a if isinstance(a, str) else "")
def test_row_strides_that_overflow(lib, args, entry, names, ld):
    there = {"linear_forward": dict(residual=P[3], preact=P[4]),
             "gated_ffn_forward": dict(residual=P[6], gate=P[7], up=P[8])}.get(entry, {})
    for name in names:
        assert args.call(getattr(lib, entry), None, **there, **{name: ld}) == DIM, name


def side(**changes):
    return LINEAR.call(tc.load_library().linear_forward, None, **changes)


@pytest.mark.parametrize("changes", [
    dict(y=P[0] + 126, ldx=256, ldy=256),                           # one element of x's rows: and no multiple of 16 bytes
    dict(y=P[0] + 112, ldx=256, ldy=256),                           # x's last eight columns
    dict(y=P[0] + 272, ldx=256, ldy=256),                           # past the stride, into x's next row
    dict(y=P[0] + 512 + 272, ldx=256, ldy=256),                     # the same a row on
    dict(y=P[0] - 512 * 4 + 272, ldx=256, ldy=256),                 # the same before x
    dict(y=P[0] + 128, ldx=256, ldy=264),                           # another stride
    dict(y=P[2], residual=P[2] + 512 * 3, ldy=256, ldr=256),        # rows of the residual
    dict(y=P[2], preact=P[2] + 240, ldy=256, ldp=256)], ids=str)
def test_overlapping_column_ranges(lib, changes):
    assert side(**changes) in ((ALIGN,) if changes.get("y") == P[0] + 126 else (ALIAS,))


def test_refusals_before_the_binding_sees_the_tensors():
    """A stream to enter and a piece to choose are looked up on the tensors first: what is not a
    tensor, has no rows or is no list of any is refused all the same."""
    torch = pytest.importorskip("torch")
    x, t = torch.zeros(8, 64, dtype=torch.float16), torch.zeros(8, dtype=torch.int64)
    for call in (lambda: tc.linear([1.0], x, stream=3), lambda: tc.linear(None, x, stream=0), lambda: tc.linear(x, x, stream="no"),
                 lambda: tc.clip_grad_norm([], 1.0, stream=3), lambda: tc.clip_grad_norm([None], 1.0, stream=0),
                 lambda: tc.clip_grad_norm(None, 1.0), lambda: tc.clip_grad_norm([x], 1.0, out=3),
                 lambda: tc.linear_cross_entropy_backward(x, None, x, t, x),
                 lambda: tc.linear_cross_entropy_backward(x, torch.zeros((), dtype=torch.float16), x, t, x),
                 lambda: tc.linear_cross_entropy_backward(x, x, x, t, x, piece=2.5),
                 lambda: tc.linear(x, x, act=[]), lambda: tc.linear_cross_entropy(x, x, t, reduction=["mean"])):
        with pytest.raises(ValueError):
            call()
