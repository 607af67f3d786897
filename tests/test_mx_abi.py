"""The norm's and the microscaled operands' C ABI and binding on the CPU: arguments are refused
before any CUDA call, workspaces are sized on the host.  No compute call is made here."""
import ctypes
import struct

import pytest

import tensor_core_tiled_02_gb300 as tc
from test_layer_abi import ALIAS, ALIGN, CONFIG, DIM, DTYPE, NULL, OK, WORKSPACE, Args, P, built  # noqa: F401  (built: a fixture)

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib(built):  # noqa: F811
    return tc.load_library()


class WithEps(Args):
    def call(self, fn, *more, **changes):
        f = {**self, **changes}
        return fn(struct.pack(f"{len(f) - 1}qd", *f.values()), *more)


NORM = WithEps(x=P[0], residual=P[1], weight=P[2], h=P[3], y=P[4], data=0, scale=0, rstd=P[5], ldx=64, ldr=64, ldh=64, ldy=64, ldd=64,
               tokens=32, dim=64, dtype=1, format=0, eps=1e-6)
NORM_GRAD = Args(dy=P[0], h=P[1], weight=P[2], dh=P[3], rstd=P[4], dx=P[5], dweight=P[6], lddy=64, ldh=64, lddh=64, lddx=64, tokens=32,
                 dim=64, dtype=0, workspace=P[7], workspace_bytes=1 << 20)
QUANT = Args(x=P[0], data=P[1], scale=P[2], ldx=64, ldd=64, rows=32, cols=64, dtype=0, format=0, transpose=0)
VALUES = Args(data=P[0], scale=P[1], x=P[2], ldd=64, ldx=64, rows=32, cols=64, dtype=0, format=0)
LINEAR = Args(x=P[0], x_scale=P[1], w=P[2], w_scale=P[3], bias=0, residual=0, y=P[4], ldx=64, ldw=64, ldr=128, ldy=128, tokens=32, k=64,
              n=128, dtype=0, act=0, format=0)


@pytest.mark.parametrize("changes,code", [
    (dict(dtype=2), DTYPE), (dict(tokens=-1), DIM), (dict(dim=0), DIM), (dict(dim=2**31 - 1), DIM), (dict(eps=-1e-9), CONFIG),
    (dict(eps=float("nan")), CONFIG), (dict(x=0), NULL), (dict(weight=0), NULL), (dict(h=0), NULL), (dict(residual=0), NULL),
    (dict(y=0), NULL), (dict(data=P[6]), NULL), (dict(scale=P[6]), NULL), (dict(data=P[6], scale=P[7], format=2), CONFIG),
    (dict(x=P[0] + 8), ALIGN), (dict(ldh=68), ALIGN), (dict(ldx=56), DIM), (dict(weight=P[2] + 2), ALIGN), (dict(rstd=P[5] + 2), ALIGN),
    (dict(data=P[6] + 8, scale=P[7]), ALIGN), (dict(data=P[6], scale=P[7] + 8), ALIGN), (dict(data=P[6], scale=P[7], ldd=72), ALIGN),
    (dict(data=P[6], scale=P[7], ldd=48), DIM),
    (dict(y=P[0]), ALIAS), (dict(y=P[3]), ALIAS), (dict(h=P[0] + 16), ALIAS), (dict(h=P[0], ldh=72), ALIAS), (dict(h=P[1], ldh=72), ALIAS),
    (dict(rstd=P[4] + 64), ALIAS), (dict(data=P[4], scale=P[7]), ALIAS), (dict(data=P[6], scale=P[6] + 512), ALIAS),
    (dict(h=P[2] - 64), ALIAS), (dict(ldx=1 << 62), DIM), (dict(ldr=(1 << 63) - 8), DIM)], ids=str)
def test_norm_refusals(lib, changes, code):
    assert NORM.call(lib.rms_norm_forward, None, **changes) == code


@pytest.mark.parametrize("changes,code", [
    (dict(dtype=3), DTYPE), (dict(tokens=-1), DIM), (dict(dim=0), DIM), (dict(dy=0), NULL), (dict(h=0), NULL), (dict(weight=0), NULL),
    (dict(rstd=0), NULL), (dict(workspace=0), NULL), (dict(workspace=P[7] + 64), ALIGN), (dict(workspace_bytes=64), WORKSPACE),
    (dict(dx=P[1]), ALIAS), (dict(dx=P[0], lddx=72), ALIAS), (dict(dx=P[3] + 16), ALIAS), (dict(dweight=P[2]), ALIAS),
    (dict(dweight=P[5] + 64), ALIAS), (dict(workspace=P[5]), ALIAS), (dict(lddx=60), DIM), (dict(lddy=68), ALIGN),
    (dict(dweight=P[6] + 1), ALIGN), (dict(rstd=P[4] + 1), ALIGN), (dict(weight=P[2] + 8), ALIGN)], ids=str)
def test_norm_backward_refusals(lib, changes, code):
    assert NORM_GRAD.call(lib.rms_norm_backward, None, **changes) == code


def test_norm_backward_workspace(lib):
    fn = lib.rms_norm_backward_workspace
    pad = lambda n: (n + 255) // 256 * 256  # noqa: E731
    assert NORM_GRAD.size(fn, dweight=0) == (OK, 0)
    sizes = [NORM_GRAD.size(fn, tokens=t) for t in (0, 1, 32, 1 << 20, 1 << 30)]
    assert sizes[0] == (OK, 0) and all(rc == OK and n % 256 == 0 for rc, n in sizes)
    assert sizes[1][1] >= pad(64 * 4) and sizes[3] == sizes[4]  # a bounded number of partial sums
    assert NORM_GRAD.size(fn, dtype=2)[0] == DTYPE and NORM_GRAD.size(fn, dim=0)[0] == DIM and fn(None, None) == NULL


@pytest.mark.parametrize("changes,code", [
    (dict(dtype=2), DTYPE), (dict(format=2), CONFIG), (dict(transpose=2), CONFIG), (dict(rows=-1), DIM), (dict(cols=1 << 31), DIM),
    (dict(x=0), NULL), (dict(data=0), NULL), (dict(scale=0), NULL), (dict(ldx=60), DIM), (dict(ldx=68), ALIGN), (dict(ldd=48), DIM),
    (dict(ldd=72), ALIGN), (dict(data=P[1] + 8), ALIGN), (dict(scale=P[2] + 4), ALIGN), (dict(data=P[0]), ALIAS), (dict(scale=P[0] + 64), ALIAS),
    (dict(scale=P[1] + 1024), ALIAS), (dict(transpose=1, ldd=16), DIM), (dict(ldd=1 << 62), DIM)], ids=str)
def test_quantize_refusals(lib, changes, code):
    assert QUANT.call(lib.mx_quantize, None, **changes) == code


@pytest.mark.parametrize("changes,code", [
    (dict(dtype=2), DTYPE), (dict(format=-1), CONFIG), (dict(rows=1 << 31), DIM), (dict(x=0), NULL), (dict(data=0), NULL), (dict(scale=0), NULL),
    (dict(ldx=60), DIM), (dict(ldd=32), DIM), (dict(x=P[2] + 2), ALIGN), (dict(x=P[0]), ALIAS), (dict(x=P[1]), ALIAS)], ids=str)
def test_dequantize_refusals(lib, changes, code):
    assert VALUES.call(lib.mx_dequantize, None, **changes) == code


@pytest.mark.parametrize("changes,code", [
    (dict(dtype=2), DTYPE), (dict(act=5), CONFIG), (dict(format=2), CONFIG), (dict(tokens=-1), DIM), (dict(k=0), DIM), (dict(n=0), DIM),
    (dict(n=2**31 - 1), DIM), (dict(x=0), NULL), (dict(x_scale=0), NULL), (dict(w=0), NULL), (dict(w_scale=0), NULL), (dict(y=0), NULL),
    (dict(x=P[0] + 8), ALIGN), (dict(ldx=72), ALIGN), (dict(ldw=48), DIM), (dict(x_scale=P[1] + 8), ALIGN), (dict(ldy=120), DIM),
    (dict(bias=P[5] + 1), ALIGN), (dict(y=P[0]), ALIAS), (dict(y=P[1]), ALIAS), (dict(y=P[3]), ALIAS), (dict(bias=P[4]), ALIAS),
    (dict(residual=P[4] + 16), ALIAS), (dict(residual=P[4], ldr=136), ALIAS), (dict(ldw=1 << 62), DIM), (dict(ldy=1 << 62), DIM)], ids=str)
def test_linear_refusals(lib, changes, code):
    assert LINEAR.call(lib.mx_linear, None, **changes) == code


def test_nothing_to_do(lib):
    for fn in (lib.rms_norm_forward, lib.rms_norm_backward, lib.mx_quantize, lib.mx_dequantize, lib.mx_linear):
        assert fn(None, None) == NULL
    assert NORM.call(lib.rms_norm_forward, None, tokens=0, x=0, y=0) == OK
    assert NORM_GRAD.call(lib.rms_norm_backward, None, dx=0, dweight=0) == OK
    assert QUANT.call(lib.mx_quantize, None, rows=0, x=0) == OK and QUANT.call(lib.mx_quantize, None, cols=0, data=0) == OK
    assert VALUES.call(lib.mx_dequantize, None, rows=0, x=0) == OK
    assert LINEAR.call(lib.mx_linear, None, tokens=0, x=0, y=0) == OK


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(8, 64, dtype=torch.float16), torch.ones(64, dtype=torch.float16)
    data, scale = torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8)
    m = tc.Mx(data, scale, 64, "e4m3")
    for call in (lambda: tc.rms_norm(x, w), lambda: tc.rms_norm_mx(x, w), lambda: tc.rms_norm_backward(x, x, w, w), lambda: tc.mx_quantize(x),
                 lambda: tc.mx_dequantize(m), lambda: tc.mx_linear(m, m), lambda: tc.mx_linear(x, m), lambda: tc.mx_linear(m, m, dtype="bf16"),
                 lambda: tc.mx_linear(m, m._replace(cols=32)), lambda: tc.mx_linear(m, m._replace(format="e2m1")), lambda: tc.mx_quantize(x, "int8"),
                 lambda: tc.mx_quantize(x, []), lambda: tc.rms_norm(None, w, stream=3), lambda: tc.mx_dequantize(None),
                 lambda: tc.mx_linear(m._replace(format=None), m._replace(format=None)), lambda: tc.rms_norm([1.0], w)):
        with pytest.raises(ValueError):
            call()
    assert ctypes.sizeof(ctypes.c_void_p) == 8
