"""Arguments of the layer operators that no tensor has but a caller of the C ABI can
pass: refused on the host, before any CUDA call.  No compute call is made here."""
import pytest

import tensor_core_tiled_02_gb300 as tc
from test_layer_abi import DIM, GATED, LINEAR, LINEAR_GRAD, LOSS, LOSS_GRAD, P, built  # noqa: F401  (built: a fixture)


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
