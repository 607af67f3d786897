"""The norm with the residual's addition, its microscaled output and its gradients, against
64 bits.

Bounds, in units of 2^-24 of the magnitude at hand (one fp32 rounding each).  A thread adds
at most c values one after the other and 10 more in two trees: squares, all of one sign, are
off by c + 10.  rstd halves that and adds three roundings (division, sum, root, the last two
weighing half and one).  h w is exact (two 16-bit significands), so y has one rounding more.
The gradient's mean is off by (c + 10 + 2) of the mean of magnitudes, and five products and
sums follow; dweight adds the rows of one block (of at least 152, or fewer for long rows), then
the blocks' sums (24 at most one after the other and 5 in a tree), terms of two roundings
each.  c: eight columns to each of 8 vectors, or of a thread's share of a long row.
"""
import math

import pytest

import mx_ref
import tensor_core_tiled_02_gb300 as tc
from layer_ref import V, check

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F16, BF16 = torch.float16, torch.bfloat16
EPS = 1e-5
ULP = 2.0 ** -24


@pytest.fixture(autouse=True)
def _status():
    yield
    rc, site = tc.gemm_f16_device_status(reset=True)
    assert rc == 0, f"a device wait gave up (site {site})"


def draw(seed, rows, cols, dt=BF16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, (cols + 7) // 8 * 8, generator=g, device="cuda") * scale
    return x.to(dt)[:, :cols]


def vector(seed, n, dt=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1 + 0.3 * torch.randn(n, generator=g, device="cuda")).to(dt)


def chain(dim):
    return max(64, 8 * math.ceil(dim / 8192))


def normed(h, w, eps=EPS):
    """(y, rstd) with their bounds."""
    h64 = h.double()
    rstd = (h64.pow(2).mean(1, keepdim=True) + eps).rsqrt()
    off = ((chain(h.shape[1]) + 10) / 2 + 3) * ULP
    y = h64 * w.double() * rstd
    return V(y, (off + ULP) * 1.01 * y.abs() + 2.0 ** -149), V(rstd, off * rstd)


SHAPES = [(1, 1), (1, 8), (3, 5), (1, 4096), (2, 257), (7, 1003), (33, 256), (130, 2048), (517, 1003), (400, 520), (1000, 4096), (64, 8192),
          (5, 16392), (400, 16400), (3, 65536), (2, 65544), (2, 140001)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dt", [F16, BF16], ids=str)
def test_forward(shape, dt):
    t, d = shape
    x, r, w = draw(1, t, d, dt), draw(2, t, d, dt, 2.0), vector(3, d, dt)
    want, rstd = normed(x, w)
    check(tc.rms_norm(x, w, eps=EPS), want, dt, 1.0, "y")
    y, h, s = tc.rms_norm(x, w, eps=EPS, save=True)
    check(y, want, dt, 1.0, "saved y")
    assert h is x and s.dtype == torch.float32 and ((s.double()[:, None] - rstd.v).abs() <= rstd.e).all()
    y, h = tc.rms_norm(x, w, residual=r, eps=EPS)
    assert torch.equal(h, (x.float() + r.float()).to(dt))
    want, _ = normed(h, w)
    check(y, want, dt, 1.0, "with residual")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_forward_mx(shape, fmt):
    """Each value is what some y within its bound rounds to, under a scale that some such
    largest magnitude has."""
    t, d = shape
    x, r, w = draw(4, t, d), draw(5, t, d, scale=2.0), vector(6, d)
    m, h = tc.rms_norm_mx(x, w, format=fmt, residual=r, eps=EPS)
    assert torch.equal(h, (x.float() + r.float()).to(BF16)) and m.cols == d and m.format == fmt
    want, _ = normed(h, w)
    byte, behind = mx_ref.scale_bytes(m, t)
    assert not behind.any()
    lo, hi = want.v.abs() - want.e, want.v.abs() + want.e
    low, high = (mx_ref.exponents(mx_ref.blocks(v.clamp(min=0)), fmt) for v in (lo, hi))
    assert ((byte == low) | (byte == high)).all()
    s = torch.repeat_interleave(mx_ref.pow2(byte - 127), 32, 1)[:, :d]
    table = torch.tensor(mx_ref.TABLE[fmt], dtype=torch.float64, device="cuda")
    got = mx_ref.values(m) / s
    a, b = (table[mx_ref.nearest(v.clamp(min=0) / s, fmt)] for v in (lo, hi))
    assert ((got.abs() >= a) & (got.abs() <= b)).all()
    assert ((got == 0) | (torch.sign(got) == torch.sign(want.v))).all()
    filled = mx_ref.values((m.data, m.scale, -(-d // 32) * 32, fmt))[:, d:]
    assert not filled.any()
    only = tc.rms_norm_mx(h, w, format=fmt, eps=EPS)
    assert torch.equal(only.data, m.data) and torch.equal(mx_ref.scale_bytes(only, t)[0], byte)


def gradients(dy, h, w, rstd, dh):
    """The formula in 64 bits with its bounds; rstd as saved."""
    dim = h.shape[1]
    g, h, w, r = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    gw, c = g * w, chain(dim)
    mean, size = (gw * h).mean(1, keepdim=True), (gw * h).abs().mean(1, keepdim=True)
    dx = r * gw - h * r ** 3 * mean
    e = ULP * (3 * (r * gw).abs() + h.abs() * r ** 3 * (c + 12 + 5) * size)
    if dh is not None:
        dx = dx + dh.double()
        e = e + ULP * dh.double().abs()
    e = e + 2 * ULP * dx.abs()
    dw, mag = (g * h * r).sum(0, keepdim=True), (g * h * r).abs().sum(0, keepdim=True)
    blocks = 152 if dim <= 16384 else max(8, 608 // math.ceil(dim / 2048))
    rows = math.ceil(len(h) / min(len(h), blocks))
    return V(dx, 1.01 * e), V(dw, 1.01 * ULP * (rows + 24 + 5 + 3) * mag)


@pytest.mark.parametrize("shape", SHAPES + [(5000, 264)], ids=str)
@pytest.mark.parametrize("dt", [F16, BF16], ids=str)
def test_backward(shape, dt):
    t, d = shape
    h, dy, dh, w = draw(7, t, d, dt, 2.0), draw(8, t, d, dt, 0.1), draw(9, t, d, dt, 0.1), vector(10, d, dt)
    _, _, rstd = tc.rms_norm(h, w, eps=EPS, save=True)
    for extra in (None, dh):
        dx, dw = tc.rms_norm_backward(dy, h, w, rstd, dh=extra)
        wx, ww = gradients(dy, h, w, rstd, extra)
        check(dx, wx, dt, 1.0, "dx")
        assert dw.dtype == dt and tuple(dw.shape) == (d,)
        check(dw[None], ww, dt, 1.0, "dweight")
    for over in (0, 1):  # in place: dx over dy, over dh
        args = [draw(8, t, d, dt, 0.1), draw(9, t, d, dt, 0.1)]
        out, again = tc.rms_norm_backward(args[0], h, w, rstd, dh=args[1], out=args[over])
        assert out is args[over] and torch.equal(out, dx) and torch.equal(again, dw)


def test_formula_is_the_gradient():
    """The formula above against automatic differentiation of the definition."""
    h = draw(11, 9, 77).double().requires_grad_()
    w = vector(12, 77).double().requires_grad_()
    dy = draw(13, 9, 77)
    rstd = (h.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
    dx, dw = torch.autograd.grad(h * rstd * w, (h, w), dy.double())
    g, r, hd, wd = dy.double(), rstd.detach(), h.detach(), w.detach()
    assert torch.allclose(dx, r * g * wd - hd * r ** 3 * (g * wd * hd).mean(1, keepdim=True), rtol=1e-12, atol=1e-14)
    assert torch.allclose(dw, (g * hd * r).sum(0), rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("residual", [False, True])
def test_gradient_against_differences(residual):
    """Along a random direction: the loss sum(y c) at h + t d less that at h - t d, over the
    steps as fp16 holds them.  y's own rounding, 2^-12 of it at most, spreads evenly, so its
    sum over n values stays within 6 / sqrt(3) sqrt(sum (y c)^2) 2^-12 on each side; the third
    order is (t |d| / |h|)^2 of the change."""
    t, d = 64, 512
    x, w, c = draw(14, t, d, F16), vector(15, d, F16), draw(16, t, d, F16)
    r = draw(17, t, d, F16) if residual else None
    _, h, rstd = tc.rms_norm(x, w, residual=r, eps=EPS, save=True)
    dx, dw = tc.rms_norm_backward(c, h, w, rstd)
    step = 0.125
    delta = draw(18, t, d, F16).float() * step
    plus, minus = (h.float() + delta).to(F16), (h.float() - delta).to(F16)
    yp, ym = (tc.rms_norm(v, w, eps=EPS).double() * c.double() for v in (plus, minus))
    got = (yp - ym).sum().item()
    want = (dx.double() * (plus.double() - minus.double())).sum().item()
    noise = 2 * 3.5 * 2.0 ** -12 * yp.norm().item()
    change = (dx.double() * (plus.double() - minus.double())).norm().item()
    assert abs(got - want) <= noise + 6 * step ** 2 * change
    # and along the weight, in which y is linear
    dw_step = (0.25 * torch.randn(d, generator=torch.Generator().manual_seed(19))).cuda()
    wp, wm = (w.float() + dw_step).to(F16), (w.float() - dw_step).to(F16)
    yp, ym = (tc.rms_norm(h, v, eps=EPS).double() * c.double() for v in (wp, wm))
    got, want = (yp - ym).sum().item(), (dw.double() * (wp.double() - wm.double())).sum().item()
    rounding = 2.0 ** -11 * (dw.double() * (wp.double() - wm.double())).abs().sum().item()
    assert abs(got - want) <= 2 * 3.5 * 2.0 ** -12 * yp.norm().item() + rounding


@pytest.mark.parametrize("shape", [(3, 40), (40, 4096), (700, 1000)], ids=str)
def test_in_place_and_views(shape):
    t, d = shape
    w = vector(20, d)
    x, r = draw(21, t, d), draw(22, t, d)
    y, h = tc.rms_norm(x, w, residual=r, eps=EPS)
    for which in (0, 1):  # h over the residual, over x
        a = [x.clone(), r.clone()]
        y2, h2 = tc.rms_norm(a[0], w, residual=a[1], eps=EPS, h_out=a[1 - which])
        assert h2 is a[1 - which] and torch.equal(h2, h) and torch.equal(y2, y)
    wide = torch.full((t, 2 * ((d + 7) // 8 * 8) + 16), 3.0, dtype=BF16, device="cuda")
    at = (d + 7) // 8 * 8 + 8
    wide[:, :d] = x
    y3, h3 = tc.rms_norm(wide[:, :d], w, residual=r, eps=EPS, out=wide[:, at:at + d])
    assert torch.equal(wide[:, at:at + d], y) and (wide[:, d:at] == 3).all() and (wide[:, at + d:] == 3).all()
    dy = draw(23, t, d)
    _, _, rstd = tc.rms_norm(h, w, eps=EPS, save=True)
    dx, dw = tc.rms_norm_backward(dy, h, w, rstd)
    wide[:] = 3.0
    tc.rms_norm_backward(dy, h, w, rstd, out=wide[:, 8:8 + d])
    assert torch.equal(wide[:, 8:8 + d], dx) and (wide[:, :8] == 3).all() and (wide[:, 8 + d:] == 3).all()


@pytest.mark.parametrize("dim", [16392, 40007])
def test_long_rows_in_place(dim):
    """h over the residual, over x; the longer rows are read twice."""
    w, x, r = vector(24, dim), draw(25, 3, dim), draw(26, 3, dim)
    y, h = tc.rms_norm(x, w, residual=r, eps=EPS)
    for which in (0, 1):
        a = [draw(25, 3, dim), draw(26, 3, dim)]
        y2, h2 = tc.rms_norm(a[0], w, residual=a[1], eps=EPS, h_out=a[1 - which])
        assert h2 is a[1 - which] and torch.equal(h2, h) and torch.equal(y2, y)


@pytest.mark.parametrize("dim", [64, 1003, 4096])
def test_special_rows(dim):
    x, w = draw(24, 9, dim), vector(25, dim)
    x[1], x[2, dim // 2], x[3, 0] = 0.0, float("nan"), float("inf")
    x[4], x[5] = 1e-30, 1e30           # squares below and above fp32's range
    y, _, rstd = tc.rms_norm(x, w, eps=EPS, save=True)
    assert not y[1].any() and y[2].isnan().all()
    assert rstd[3] == 0 and y[3, 0].isnan() and not y[3, 1:].any()
    assert rstd[5] == 0 and not y[5].any()
    want, _ = normed(x[[0, 1, 4, 6, 7, 8]], w)
    check(y[[0, 1, 4, 6, 7, 8]], want, BF16, 1.0, "the other rows")
    assert tc.rms_norm(x, w, eps=0.0)[1].isnan().all()   # 0 / 0
    m = tc.rms_norm_mx(x, w, format="e4m3", eps=EPS)
    v = mx_ref.values(m)
    assert v[2].isnan().all() and v[3, :32].isnan().all() and not v[3, 32:].any() and not v[1].any() and v[[0, 4, 6]].isfinite().all()


def test_no_tokens():
    x, w = torch.zeros(0, 72, dtype=F16, device="cuda"), vector(26, 72, F16)
    y, h, rstd = tc.rms_norm(x, w, residual=x, save=True)
    assert tuple(y.shape) == tuple(h.shape) == (0, 72) and tuple(rstd.shape) == (0,)
    dx, dw = tc.rms_norm_backward(x, x, w, rstd)
    assert tuple(dx.shape) == (0, 72) and not dw.any()
    assert tuple(tc.rms_norm_mx(x, w).data.shape) == (0, 96)


@pytest.mark.parametrize("tokens", [1, 300, 3000])
def test_same_bits_on_another_stream_and_in_a_graph(tokens):
    d = 1032
    x, r, w, dy = draw(27, tokens, d), draw(28, tokens, d), vector(29, d), draw(30, tokens, d)

    def both(stream=None):
        y, h, rstd = tc.rms_norm(x, w, residual=r, save=True, stream=stream)
        return (y, h, rstd, *tc.rms_norm_backward(dy, h, w, rstd, dh=dy, stream=stream))

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(on_side, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = both()
    for seed in (31, 32):
        x.copy_(draw(seed, tokens, d))
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(held, both()))


def test_written_tensors_change_version():
    x, r, w = draw(33, 4, 64), draw(34, 4, 64), vector(35, 64)
    out = torch.empty_like(x)
    before = [t._version for t in (x, r, w, out)]
    tc.rms_norm(x, w, residual=r, h_out=r, out=out)
    assert [t._version - b for t, b in zip((x, r, w, out), before)] == [0, 1, 0, 1]


def test_refusals():
    x, w = draw(36, 8, 64), vector(37, 64)
    rstd = torch.ones(8, device="cuda")
    for call in (lambda: tc.rms_norm(x, w.float()), lambda: tc.rms_norm(x, w[:32]), lambda: tc.rms_norm(x.float(), w),
                 lambda: tc.rms_norm(x[0], w), lambda: tc.rms_norm(x, w, residual=x[:4]), lambda: tc.rms_norm(x, w, h_out=x.clone()),
                 lambda: tc.rms_norm(x, w, out=x.half()), lambda: tc.rms_norm(x.cpu(), w), lambda: tc.rms_norm(x, w.cpu()),
                 lambda: tc.rms_norm(x, w, eps="small"), lambda: tc.rms_norm_mx(x, w, format="fp8"), lambda: tc.rms_norm(x.T, w[:8]),
                 lambda: tc.rms_norm_backward(x, x, w, rstd[:4]), lambda: tc.rms_norm_backward(x, x, w, rstd.double()),
                 lambda: tc.rms_norm_backward(x[:4], x, w, rstd), lambda: tc.rms_norm_backward(x, x, w, rstd, dh=x.half())):
        with pytest.raises(ValueError):
            call()
    wide = draw(38, 9, 128)
    for call, code in ((lambda: tc.rms_norm(x, w, eps=-1.0), -6), (lambda: tc.rms_norm(x, w, eps=float("nan")), -6),
                       (lambda: tc.rms_norm(x, w, out=x), -5), (lambda: tc.rms_norm(torch.zeros(8, 60, dtype=BF16, device="cuda"), w[:60]), -4),
                       (lambda: tc.rms_norm(wide[:8, 64:], w, residual=x, h_out=wide[1:, 64:]), -5),
                       (lambda: tc.rms_norm(x, vector(1, 80)[1:65]), -4), (lambda: tc.rms_norm_backward(x, x.clone(), w, rstd, out=w.expand(8, 64)), -2),
                       (lambda: (lambda h: tc.rms_norm_backward(x, h, w, rstd, out=h))(x.clone()), -5)):
        with pytest.raises(tc.GemmError) as e:
            call()
        assert e.value.code == code
