"""What lies behind an output's last column stays as it is: outputs as views of wider
rows whose width is no multiple of 8, through the torch binding and the C ABI."""
import ctypes
import struct

import pytest

import tensor_core_tiled_02_gb300 as tc
from layer_ref import V, check

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DT = torch.bfloat16
GUARD = 3.0


@pytest.fixture(autouse=True)
def _status():
    yield
    rc, site = tc.gemm_f16_device_status(reset=True)
    assert rc == 0, f"a device wait gave up (site {site})"


def draw(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pitch = (shape[-1] + 7) // 8 * 8
    return (torch.randn(*shape[:-1], pitch, generator=g, device="cuda") * scale).to(DT)[..., :shape[-1]]


def guarded(rows, cols):
    """[rows, cols] in rows of up to 15 entries more, all of them GUARD."""
    buf = torch.full((rows, (cols + 7) // 8 * 8 + 8), GUARD, device="cuda", dtype=DT)
    return buf, buf[:, :cols]


def kept(buf, cols):
    return bool((buf[:, cols:] == GUARD).all())


WIDTHS = [1, 5, 7, 8, 9, 123, 257, 1031]


@pytest.mark.parametrize("tokens", [1, 40, 300, 2500])
@pytest.mark.parametrize("n", WIDTHS)
def test_forward(tokens, n):
    for k in (72, 4096):  # the latter split along K where the tiles are few
        if k == 4096 and tokens != 300:
            continue
        x, w, r = draw(1, tokens, k), draw(2, k, n, scale=k ** -0.5), draw(3, tokens, n)
        want = V(x) @ V(w)
        buf, out = guarded(tokens, n)
        tc.linear(x, w, out=out)
        check(out, want, DT, 1.0, "y")
        assert kept(buf, n), "y"
        out.copy_(r)
        tc.linear(x, w, residual=out, out=out)
        check(out, want + V(r), DT, 1.0, "in place")
        assert kept(buf, n), "in place"
        # the block's second product
        buf, out = guarded(tokens, n)
        tc.gated_ffn(x, draw(4, k, 64, scale=k ** -0.5), draw(5, k, 64, scale=k ** -0.5), draw(6, 64, n, scale=0.125), out=out)
        assert kept(buf, n), "gated"


def call(name, fmt, *fields):
    torch.cuda.synchronize()
    rc = getattr(tc.load_library(), name)(struct.pack(fmt, *fields), None)
    torch.cuda.synchronize()
    assert rc == 0, (name, rc)


@pytest.mark.parametrize("tokens", [5, 300, 2500])
@pytest.mark.parametrize("n", WIDTHS)
def test_kept_for_the_backward_pass(tokens, n):
    """preact, hidden, gate and up, which only the C ABI lets a caller place."""
    k = 72
    x, w, u = draw(1, tokens, k), draw(2, k, n, scale=k ** -0.5), draw(3, k, n, scale=k ** -0.5)
    d = draw(4, n, 64, scale=0.1)
    (by, y), (bp, pre) = guarded(tokens, n), guarded(tokens, n)
    call("linear_forward", "16q", x.data_ptr(), w.data_ptr(), 0, 0, y.data_ptr(), pre.data_ptr(), x.stride(0), w.stride(0), 0,
         y.stride(0), pre.stride(0), tokens, k, n, 1, 2)
    py, ppre = tc.linear(x, w, act="silu", save_preact=True)
    assert torch.equal(y, py) and torch.equal(pre, ppre) and kept(by, n) and kept(bp, n)
    (bh, h), (bg, g), (bu, up) = guarded(tokens, n), guarded(tokens, n), guarded(tokens, n)
    out = torch.empty(tokens, 64, device="cuda", dtype=DT)
    call("gated_ffn_forward", "24q", x.data_ptr(), w.data_ptr(), u.data_ptr(), d.data_ptr(), 0, out.data_ptr(), h.data_ptr(),
         g.data_ptr(), up.data_ptr(), x.stride(0), w.stride(0), u.stride(0), d.stride(0), 0, 64, h.stride(0), g.stride(0),
         up.stride(0), tokens, k, n, 64, 1, 2)
    py, pg, pu, ph = tc.gated_ffn(x, w, u, d, save=True)
    assert all(torch.equal(a, b) for a, b in ((out, py), (g, pg), (up, pu), (h, ph)))
    assert kept(bh, n) and kept(bg, n) and kept(bu, n)


@pytest.mark.parametrize("tokens", [5, 300, 2500])
@pytest.mark.parametrize("k,n", [(1, 64), (64, 5), (123, 257), (1031, 9), (72, 1031)])
def test_gradients(tokens, k, n):
    x, w, dy = draw(1, tokens, k), draw(2, k, n, scale=k ** -0.5), draw(3, tokens, n)
    (bx, dx), (bw, dw) = guarded(tokens, k), guarded(k, n)
    call("linear_backward", "20q", dy.data_ptr(), x.data_ptr(), w.data_ptr(), 0, dx.data_ptr(), dw.data_ptr(), 0, dy.stride(0),
         x.stride(0), w.stride(0), 0, dx.stride(0), dw.stride(0), tokens, k, n, 1, 0, 0, 0)
    px, pw, _ = tc.linear_backward(dy, x, w)
    assert torch.equal(dx, px) and torch.equal(dw, pw) and kept(bx, k) and kept(bw, n)
    # the loss's: h [tokens, k], w [n, k], over one piece and over several
    wt, target = draw(4, 600, k), torch.arange(tokens, device="cuda") % 600
    _, lse = tc.linear_cross_entropy(x, wt, target)
    one = torch.ones(1, device="cuda")
    for piece in (256, 768):
        (bh, dh), (bw, dw) = guarded(tokens, k), guarded(600, k)
        f = [x.data_ptr(), wt.data_ptr(), target.data_ptr(), lse.data_ptr(), one.data_ptr(), dh.data_ptr(), dw.data_ptr(),
             x.stride(0), wt.stride(0), dh.stride(0), dw.stride(0), tokens, k, 600, 1, -100, 1, 0, 0]
        size = ctypes.c_size_t()
        assert tc.load_library().linear_cross_entropy_backward_workspace(struct.pack("19q", *f), piece, ctypes.byref(size)) == 0
        ws = torch.empty(size.value, device="cuda", dtype=torch.uint8)
        call("linear_cross_entropy_backward", "19q", *f[:-2], ws.data_ptr(), size.value)
        ph, pw = tc.linear_cross_entropy_backward(one[0], x, wt, target, lse, piece=piece)
        assert torch.equal(dh, ph) and torch.equal(dw, pw) and kept(bh, k) and kept(bw, k)
