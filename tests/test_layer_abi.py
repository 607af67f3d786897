"""The layer operators' C ABI and binding on the CPU: arguments are refused
before any CUDA call, workspaces are sized on the host, host tensors never
reach a kernel.  No compute call is made here."""
import ctypes
import struct

import pytest

import tensor_core_tiled_02_gb300 as tc
from tensor_core_tiled_02_gb300 import build as tcbuild

torch = pytest.importorskip("torch")

OK, NULL, DIM, DTYPE, ALIGN, ALIAS, CONFIG, WORKSPACE = 0, -1, -2, -3, -4, -5, -6, -12
P = [1 << 30, 2 << 30, 3 << 30, 4 << 30, 5 << 30, 6 << 30, 7 << 30, 8 << 30, 9 << 30]  # far apart, aligned


@pytest.fixture(scope="module", autouse=True)
def built():
    if tcbuild.needs_build():
        tcbuild.build()
    if tcbuild.binding_needs_build():
        tcbuild.build_binding()


@pytest.fixture(scope="module")
def lib():
    return tc.load_library()


class Args(dict):
    """Fields of an argument structure, in order, all 8 bytes."""

    def call(self, fn, *more, **changes):
        f = {**self, **changes}
        return fn(struct.pack(f"{len(f)}q", *f.values()), *more)

    def size(self, fn, *more, **changes):
        n = ctypes.c_size_t(12345)
        rc = self.call(fn, *more, ctypes.byref(n), **changes)
        return rc, n.value


LINEAR = Args(x=P[0], w=P[1], bias=0, residual=0, y=P[2], preact=0, ldx=64, ldw=128, ldr=128, ldy=128, ldp=128, tokens=32,
              k=64, n=128, dtype=0, act=0)
LINEAR_GRAD = Args(dy=P[0], x=P[1], w=P[2], preact=P[3], dx=P[4], dw=P[5], dbias=P[6], lddy=128, ldx=64, ldw=128, ldp=128,
                   lddx=64, lddw=128, tokens=32, k=64, n=128, dtype=1, act=2, workspace=P[7], workspace_bytes=1 << 24)
GATED = Args(x=P[0], w_gate=P[1], w_up=P[2], w_down=P[3], residual=0, y=P[4], hidden=P[5], gate=0, up=0, ldx=64, ldg=128,
             ldu=128, ldd=64, ldr=64, ldy=64, ldh=128, ld_gate=128, ld_up=128, tokens=32, dim=64, ffn=128, dim_out=64,
             dtype=0, act=2)
LOSS = Args(h=P[0], w=P[1], target=P[2], loss=P[3], lse=P[4], ldh=64, ldw=64, tokens=32, dim=64, vocab=999, dtype=0,
            ignore=-100, reduction=1, workspace=P[5], workspace_bytes=1 << 24)
LOSS_GRAD = Args(h=P[0], w=P[1], target=P[2], lse=P[3], grad=P[4], dh=P[5], dw=P[6], ldh=64, ldw=64, lddh=64, lddw=64,
                 tokens=32, dim=64, vocab=999, dtype=0, ignore=-100, reduction=1, workspace=P[7], workspace_bytes=1 << 24)


@pytest.mark.parametrize("changes,code", [
    (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE), (dict(act=5), CONFIG), (dict(act=-1), CONFIG),
    (dict(tokens=-1), DIM), (dict(k=0), DIM), (dict(n=0), DIM), (dict(n=2**31 - 1), DIM), (dict(tokens=2**31), DIM),
    (dict(x=0), NULL), (dict(w=0), NULL), (dict(y=0), NULL),
    (dict(x=P[0] + 8), ALIGN), (dict(ldx=68), ALIGN), (dict(ldw=132), ALIGN), (dict(ldy=130), ALIGN), (dict(bias=P[4] + 1), ALIGN),
    (dict(ldx=56), DIM), (dict(ldw=120), DIM),
    (dict(y=P[0]), ALIAS), (dict(y=P[1] + 256), ALIAS), (dict(residual=P[2] + 16), ALIAS), (dict(preact=P[2]), ALIAS),
    (dict(residual=P[2], ldr=136), ALIAS),          # in place, but rows elsewhere
    (dict(residual=P[3], preact=P[3]), ALIAS), (dict(preact=P[3] + 2), ALIGN)], ids=str)
def test_linear_refusals(lib, changes, code):
    assert LINEAR.call(lib.linear_forward, None, **changes) == code


def test_nothing_to_do(lib):
    assert lib.linear_forward(None, None) == NULL
    # no tokens: nothing is read or written, and no device is asked
    assert LINEAR.call(lib.linear_forward, None, tokens=0, x=0, y=0) == OK
    assert GATED.call(lib.gated_ffn_forward, None, tokens=0, x=0, y=0, hidden=0) == OK
    assert LINEAR_GRAD.call(lib.linear_backward, None, dx=0, dw=0, dbias=0) == OK
    assert LOSS_GRAD.call(lib.linear_cross_entropy_backward, None, dh=0, dw=0) == OK
    assert LOSS.call(lib.linear_cross_entropy, None, tokens=0, reduction=0, loss=0, lse=0) == OK


@pytest.mark.parametrize("changes,code", [
    (dict(dy=0), NULL), (dict(preact=0), NULL), (dict(w=0), NULL), (dict(x=0), NULL), (dict(workspace=0), NULL),
    (dict(workspace=P[7] + 128), ALIGN), (dict(workspace_bytes=100), WORKSPACE), (dict(workspace_bytes=-1), WORKSPACE),
    (dict(workspace=P[0]), ALIAS), (dict(dx=P[5]), ALIAS), (dict(dw=P[1]), ALIAS), (dict(dbias=P[5] + 64), ALIAS),
    (dict(lddw=64), DIM), (dict(lddx=60), DIM), (dict(dbias=P[6] + 1), ALIGN)], ids=str)
def test_linear_backward_refusals(lib, changes, code):
    assert LINEAR_GRAD.call(lib.linear_backward, None, **changes) == code


def test_linear_backward_workspace(lib):
    fn = lib.linear_backward_workspace
    pad = lambda n: (n + 255) // 256 * 256  # noqa: E731
    slope, sums = pad(32 * 128 * 2), pad(1 * 128 * 4)   # dpre; one block of 64 rows of column sums
    assert LINEAR_GRAD.size(fn) == (OK, slope + sums)
    assert LINEAR_GRAD.size(fn, dbias=0) == (OK, slope)
    assert LINEAR_GRAD.size(fn, act=0) == (OK, sums)       # dy is dpre
    assert LINEAR_GRAD.size(fn, act=0, dbias=0) == (OK, 0)
    assert LINEAR_GRAD.size(fn, dx=0, dw=0) == (OK, sums)
    assert LINEAR_GRAD.size(fn, dtype=2)[0] == DTYPE and fn(None, None) == NULL
    # sizes whose products pass 32 bits
    assert LINEAR_GRAD.size(fn, tokens=1 << 20, n=1 << 16, ldp=1 << 16, dbias=0) == (OK, 1 << 37)


@pytest.mark.parametrize("changes,code", [
    (dict(hidden=0), NULL), (dict(gate=P[6]), NULL), (dict(w_up=0), NULL), (dict(ffn=0), DIM), (dict(dim_out=0), DIM),
    (dict(ldd=56), DIM), (dict(ldh=130), ALIGN), (dict(hidden=P[4]), ALIAS), (dict(hidden=P[3] + 1024), ALIAS),
    (dict(gate=P[6], up=P[6]), ALIAS), (dict(y=P[0]), ALIAS), (dict(dtype=3), DTYPE), (dict(act=9), CONFIG)], ids=str)
def test_gated_refusals(lib, changes, code):
    assert GATED.call(lib.gated_ffn_forward, None, **changes) == code


@pytest.mark.parametrize("changes,code", [
    (dict(target=0), NULL), (dict(lse=0), NULL), (dict(loss=0), NULL), (dict(h=0), NULL), (dict(target=P[2] + 4), ALIGN),
    (dict(loss=P[3] + 2), ALIGN), (dict(vocab=0), DIM), (dict(reduction=3), CONFIG), (dict(dtype=2), DTYPE),
    (dict(workspace_bytes=64), WORKSPACE), (dict(lse=P[3]), ALIAS), (dict(workspace=P[1]), ALIAS)], ids=str)
def test_loss_refusals(lib, changes, code):
    assert LOSS.call(lib.linear_cross_entropy, None, **changes) == code


@pytest.mark.parametrize("changes,code", [
    (dict(grad=0), NULL), (dict(lse=0), NULL), (dict(workspace=0), NULL), (dict(workspace=P[7] + 16), ALIGN),
    (dict(workspace_bytes=4096), WORKSPACE), (dict(dw=P[1]), ALIAS), (dict(dh=P[0]), ALIAS), (dict(dw=P[5] + 1024), ALIAS),
    (dict(lddw=60), DIM), (dict(vocab=-1), DIM)], ids=str)
def test_loss_backward_refusals(lib, changes, code):
    assert LOSS_GRAD.call(lib.linear_cross_entropy_backward, None, **changes) == code


def test_loss_backward_workspace(lib):
    fn = lib.linear_cross_entropy_backward_workspace
    whole = LOSS_GRAD.size(fn, 1024)
    assert whole[0] == OK and LOSS_GRAD.size(fn, 1 << 20) == whole      # a piece is at most the vocabulary
    small = LOSS_GRAD.size(fn, 256)
    assert small[0] == OK and small[1] < whole[1] + 32 * 64 * 4
    for piece in (0, 100, 255, 300):
        assert LOSS_GRAD.size(fn, piece)[0] == DIM
    assert LOSS_GRAD.size(fn, 256, tokens=0) == (OK, 0)


def clip_args(src, dst, count, dtype, ws=P[8], ws_bytes=1 << 20, max_norm=1.0, eps=1e-6, norm=P[7]):
    n = len(src)
    keep = ((ctypes.c_longlong * n)(*src), (ctypes.c_longlong * n)(*dst), (ctypes.c_longlong * n)(*count),
            (ctypes.c_int * n)(*dtype))
    return keep, struct.pack("7q2dq", *(ctypes.addressof(k) for k in keep), norm, ws, n, max_norm, eps, ws_bytes)


@pytest.mark.parametrize("change,code", [
    (dict(count=[-1, 5]), DIM), (dict(dtype=[0, 3]), DTYPE), (dict(src=[0, P[1]]), NULL), (dict(src=[P[0] + 1, P[1]]), ALIGN),
    (dict(dst=[P[2], P[3] + 2]), ALIGN), (dict(dst=[P[0] + 2, P[3]]), ALIAS), (dict(ws=0), NULL), (dict(ws_bytes=8), WORKSPACE),
    (dict(max_norm=-1.0), CONFIG), (dict(max_norm=float("nan")), CONFIG), (dict(eps=-1e-6), CONFIG), (dict(norm=P[7] + 1), ALIGN)],
    ids=str)
def test_clip_refusals(lib, change, code):
    base = dict(src=[P[0], P[1]], dst=[P[2], P[3]], count=[100, 5], dtype=[0, 2])
    keep, args = clip_args(**{**base, **change})
    assert lib.grad_clip(args, None) == code


def test_clip_workspace(lib):
    n = ctypes.c_size_t(0)
    sizes = []
    for tensors in (0, 1, 48, 49, 1000, 1001):
        assert lib.grad_clip_workspace(tensors, ctypes.byref(n)) == OK
        sizes.append(n.value)
    assert sizes[0] == sizes[4] > 0 and sizes[5] == 2 * sizes[4]
    assert lib.grad_clip_workspace(-1, ctypes.byref(n)) == DIM and lib.grad_clip_workspace(1, None) == NULL


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(8, 64, dtype=torch.float16), torch.zeros(64, 128, dtype=torch.float16)
    t = torch.zeros(8, dtype=torch.int64)
    for call in (lambda: tc.linear(x, w), lambda: tc.linear_backward(x, x, w), lambda: tc.gated_ffn(x, w, w, w.T),
                 lambda: tc.gated_ffn_backward(x, x, w, w, w.T, x, x, x), lambda: tc.linear_cross_entropy(x, x, t),
                 lambda: tc.linear_cross_entropy_backward(x, x, x, t, x), lambda: tc.clip_grad_norm([x], 1.0),
                 lambda: tc.clip_grad_norm([], 1.0), lambda: tc.linear(x, w, act="softplus"), lambda: tc.linear([1.0], w),
                 lambda: tc.linear_cross_entropy(x, x, t, reduction="max"), lambda: tc.linear(x, w, stream=3)):
        with pytest.raises(ValueError):
            call()
