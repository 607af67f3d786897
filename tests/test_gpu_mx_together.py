"""The norm, the quantisation and the microscaled linear layer as a program uses them: in a
row, captured, from several threads, on matrices past 2^31 entries, and when a wait runs out."""
import struct
import threading
import warnings

import pytest

import layer_ref
import mx_ref
import tensor_core_tiled_02_gb300 as tc
from layer_ref import V, check

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16 = torch.bfloat16
EPS = 1e-5


@pytest.fixture(autouse=True)
def _status():
    yield
    rc, site = tc.gemm_f16_device_status(reset=True)
    assert rc == 0, f"a device wait gave up (site {site})"


def draw(seed, rows, cols, scale=1.0, dt=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, (cols + 7) // 8 * 8, generator=g, device="cuda") * scale).to(dt)[:, :cols]


def vector(seed, n, dt=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1 + 0.3 * torch.randn(n, generator=g, device="cuda")).to(dt)


@pytest.mark.parametrize("tokens", [1, 150, 1500])
def test_block_and_its_gradients(tokens):
    """h = x + r, out = h + ffn(norm(h)): forward and back through the package's calls, against
    automatic differentiation of the same in 64 bits."""
    d, f = 264, 520
    x, r, w = draw(1, tokens, d), draw(2, tokens, d), vector(3, d)
    wg, wu, wd = draw(4, d, f, d ** -0.5), draw(5, d, f, d ** -0.5), draw(6, f, d, f ** -0.5)
    dout = draw(7, tokens, d, 0.1)
    y, h, rstd = tc.rms_norm(x, w, residual=r, eps=EPS, save=True)
    out, gate, up, hidden = tc.gated_ffn(y, wg, wu, wd, residual=h, save=True)
    dy, dwg, dwu, dwd = tc.gated_ffn_backward(dout, y, wg, wu, wd, gate, up, hidden)
    dx, dw = tc.rms_norm_backward(dy, h, w, rstd, dh=dout)

    leaves = [t.double().requires_grad_() for t in (h, w, wg, wu, wd)]
    h64, w64, g64, u64, d64 = leaves
    n64 = h64 * (h64.pow(2).mean(1, keepdim=True) + EPS).rsqrt() * w64
    want = layer_ref.act64("silu", n64 @ g64) * (n64 @ u64) @ d64 + h64
    exact = torch.autograd.grad(want, leaves, dout.double())
    # some six roundings to bf16 on the way (u / sqrt 3 each): sqrt(6 / 3) u of a norm, four times that
    room = 4 * 2 ** 0.5 * layer_ref.U[BF16]
    for name, a, b in [("out", out, want), *zip(("dx", "dw", "dw_gate", "dw_up", "dw_down"), (dx, dw, dwg, dwu, dwd), exact)]:
        off = (a.double() - b).norm().item()
        assert off <= room * b.norm().item(), (name, off / b.norm().item())


def serving(x, r, w, wq1, wq2, fmt):
    """norm -> product with activation -> quantise -> product onto the stream."""
    a, h = tc.rms_norm_mx(x, w, format=fmt, residual=r, eps=EPS)
    hidden = tc.mx_linear(a, wq1, act="gelu_tanh")
    return a, h, hidden, tc.mx_linear(tc.mx_quantize(hidden, fmt), wq2, residual=h)


@pytest.mark.parametrize("tokens", [1, 40, 300, 1100])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_serving_block(tokens, fmt):
    d, f = 520, 1288
    x, r, w = draw(8, tokens, d), draw(9, tokens, d), vector(10, d)
    wq1, wq2 = tc.mx_quantize(draw(11, d, f, d ** -0.5), fmt, transpose=True), tc.mx_quantize(draw(12, f, d, f ** -0.5), fmt, transpose=True)
    a, h, hidden, out = serving(x, r, w, wq1, wq2, fmt)
    check(hidden, (V(mx_ref.values(a)) @ V(mx_ref.values(wq1)).T).act("gelu_tanh"), BF16, 1.0, "hidden")
    q, _ = mx_ref.quantize(hidden, fmt)
    check(out, V(q) @ V(mx_ref.values(wq2)).T + V(h), BF16, 1.0, "out")
    # captured twice, the graphs replayed in turn on new inputs
    graphs = []
    for _ in range(2):
        xs, rs = x.clone(), r.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = serving(xs, rs, w, wq1, wq2, fmt)
        graphs.append((g, xs, rs, res[3]))
    for seed in (13, 14):
        for i, (g, xs, rs, _) in enumerate(graphs):
            xs.copy_(draw(seed + 10 * i, tokens, d))
            g.replay()
        for g, xs, rs, got in graphs:
            assert torch.equal(got, serving(xs, rs, w, wq1, wq2, fmt)[3])


def test_many_launches_in_a_row():
    """Norms whose blocks fill the GPU before and behind products on CTA pairs, a few times over:
    the products held to 64 bits, and the same bits each time."""
    tokens, d, n = 2000, 4096, 4096
    x, r, w = draw(15, tokens, d), draw(16, tokens, d), vector(17, d)
    wq = tc.mx_quantize(draw(18, n, d, d ** -0.5), "e4m3")
    got = []
    for _ in range(4):
        a, h = tc.rms_norm_mx(x, w, residual=r, eps=EPS)
        got.append(tc.mx_linear(a, wq))
    check(got[0], V(mx_ref.values(a)) @ V(mx_ref.values(wq)).T, BF16, 1.0, "y")
    assert all(torch.equal(y, got[0]) for y in got[1:])


def test_many_launches_beside_the_layer_operators():
    """The same with products in 16 bits between the norms, and quantising behind them."""
    tokens, d = 2000, 2048
    x, r, w, wl = draw(90, tokens, d), draw(91, tokens, d), vector(92, d), draw(93, d, d, d ** -0.5)
    got = []
    for _ in range(4):
        y, h = tc.rms_norm(x, w, residual=r, eps=EPS)
        z = tc.linear(y, wl)
        m = tc.mx_quantize(z, "e4m3")
        got.append((z, m.data, tc.linear(z, wl, residual=h)))
    first = got[0]
    check(first[0], V(y) @ V(wl), BF16, 1.0, "z")
    assert torch.equal(mx_ref.values(m), mx_ref.quantize(first[0], "e4m3")[0])
    check(first[2], V(first[0]) @ V(wl) + V(h), BF16, 1.0, "on the stream")
    assert all(torch.equal(a, b) for more in got[1:] for a, b in zip(more, first))


def test_more_than_2_31_entries():
    rows, cols = 66000, 33000
    at = [0, 1, 2**31 // cols - 1, 2**31 // cols, 2**31 // cols + 1, 65535, 65999]
    # the product's output
    x, w = tc.mx_quantize(draw(19, rows, 64)), tc.mx_quantize(draw(20, cols, 64, 0.125))
    y = tc.mx_linear(x, w, act="relu")
    held = mx_ref.values(x)[at]
    check(y[at], (V(held) @ V(mx_ref.values(w)).T).act("relu"), BF16, 1.0, "y")
    # that output held, along rows and columns, and back
    for fmt in ("e4m3", "e2m1"):
        m = tc.mx_quantize(y, fmt)
        back = tc.mx_dequantize(m)
        want, _ = mx_ref.quantize(y[at], fmt)
        assert torch.equal(back[at].double(), want)
        del m, back
    m = tc.mx_quantize(y, "e2m1", transpose=True)
    back = tc.mx_dequantize(m)
    cat = [0, 1, 2**31 // rows - 1, 2**31 // rows, 2**31 // rows + 1, 32999]
    want, _ = mx_ref.quantize(y[:, cat].T, "e2m1")
    assert torch.equal(back[cat].double(), want)
    del m, back
    # the norm and its gradients
    weight = vector(21, cols)
    n, h, rstd = tc.rms_norm(y, weight, eps=EPS, save=True)
    r64 = (y[at].double().pow(2).mean(1, keepdim=True) + EPS).rsqrt()
    want = y[at].double() * weight.double() * r64
    check(n[at], V(want, 2.0 ** -18 * want.abs()), BF16, 1.0, "norm")
    dx, _ = tc.rms_norm_backward(n, y, weight, rstd)
    g = n[at].double() * weight.double()
    mean = (g * y[at].double()).mean(1, keepdim=True)
    exact = r64 * g - y[at].double() * r64 ** 3 * mean
    room = 2.0 ** -17 * ((r64 * g).abs() + (y[at].double() * r64 ** 3 * (g * y[at].double()).abs().mean(1, keepdim=True)).abs())
    check(dx[at], V(exact, room), BF16, 1.0, "dx")


@pytest.mark.parametrize("tokens,residual", [(3, False), (1100, False), (1100, True)])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_wait_that_runs_out_is_reported(tokens, residual, fmt):
    """With no loads issued the MMA warp's bounded wait runs out; the context stays usable."""
    x, w, r = tc.mx_quantize(draw(22, tokens, 512), fmt), tc.mx_quantize(draw(23, 3000, 512), fmt), draw(24, tokens, 3000)
    try:
        tc.gemm_f16_set_config(inject_stall=1, wait_limit=2_000_000)
        tc.mx_linear(x, w, residual=r if residual else None)
        torch.cuda.synchronize()
        rc, site = tc.gemm_f16_device_status(reset=True)
        assert rc == -11 and site == 2
    finally:
        tc.gemm_f16_set_config()
    check(tc.mx_linear(x, w, residual=r), V(mx_ref.values(x)) @ V(mx_ref.values(w)).T + V(r), BF16, 1.0, "after")


def test_calls_from_several_threads():
    """Six host threads, each on a stream of its own, call into different kernels at once."""
    jobs = []
    for i, (t, k, n, fmt) in enumerate([(1, 512, 1024, "e2m1"), (64, 256, 520, "e4m3"), (300, 1024, 264, "e2m1"), (512, 2048, 2048, "e4m3"),
                                        (2000, 264, 776, "e4m3"), (150, 136, 2048, "e2m1")]):
        x, w, s = draw(30 + i, t, k), draw(40 + i, n, k, k ** -0.5), vector(50 + i, k)
        m = tc.rms_norm_mx(x, s, format=fmt, eps=EPS)
        wq = tc.mx_quantize(w, fmt)
        jobs.append((x, s, w, fmt, V(mx_ref.values(m)) @ V(mx_ref.values(wq)).T))
    torch.cuda.synchronize()
    got, errors = [None] * len(jobs), []

    def work(i):
        try:
            side = torch.cuda.Stream()
            x, s, w, fmt, _ = jobs[i]
            with torch.cuda.stream(side):
                for _ in range(5):
                    got[i] = tc.mx_linear(tc.rms_norm_mx(x, s, format=fmt, eps=EPS), tc.mx_quantize(w, fmt))
            side.synchronize()
        except Exception as e:  # noqa: BLE001  (reported below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for y, job in zip(got, jobs):
        check(y, job[4], BF16, 1.0, "thread")


def test_operands_that_require_gradients_and_versions():
    x, w = draw(60, 8, 64), vector(61, 64).requires_grad_()
    for call in (lambda: tc.rms_norm(x, w), lambda: tc.rms_norm_mx(x, w), lambda: tc.mx_quantize(draw(1, 8, 64).requires_grad_())):
        with pytest.warns(UserWarning, match="records no autograd graph"):
            call()
        with warnings.catch_warnings(), torch.no_grad():
            warnings.simplefilter("error")
            call()
    w = w.detach()
    m = tc.mx_quantize(draw(62, 16, 64))
    a, y, dx = tc.mx_quantize(x), draw(63, 8, 16), draw(64, 8, 64)
    _, _, rstd = tc.rms_norm(x, w, save=True)
    before = [t._version for t in (x, w, a.data, m.data, y, dx)]
    tc.mx_linear(a, m, residual=y, out=y)
    tc.rms_norm_backward(x, x, w, rstd, out=dx)
    assert [t._version - b for t, b in zip((x, w, a.data, m.data, y, dx), before)] == [0, 0, 0, 0, 1, 1]
    with torch.inference_mode():
        z = draw(65, 8, 16)
        tc.mx_linear(a, m, out=z)
    tc.mx_linear(a, m, out=z)


@pytest.mark.parametrize("tokens", [1, 5, 200])
@pytest.mark.parametrize("dim", [33, 264, 1003])
def test_norm_places_both_forms(tokens, dim):
    """y in 16 bits and held at once, rows of the held one apart, through the C ABI."""
    x, w = draw(70, tokens, dim), vector(71, dim)
    pitch, width = x.stride(0) if tokens > 1 else (dim + 7) // 8 * 8, -(-dim // 32) * 32
    y = torch.full((tokens, pitch + 8), 3.0, dtype=BF16, device="cuda")
    data = torch.full((tokens, width + 32), 0xA5, dtype=torch.uint8, device="cuda")
    tiles = -(-tokens // 128) * -(-dim // 128) * 512
    scale = torch.full((tiles + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    rc = tc.load_library().rms_norm_forward(struct.pack("17qd", x.data_ptr(), 0, w.data_ptr(), 0, y.data_ptr(), data.data_ptr(), scale.data_ptr(),
                                                        0, pitch, 0, 0, pitch + 8, width + 32, tokens, dim, 1, 0, EPS), None)
    torch.cuda.synchronize()
    assert rc == 0
    m = tc.rms_norm_mx(x, w, format="e4m3", eps=EPS)
    assert torch.equal(y[:, :dim], tc.rms_norm(x, w, eps=EPS)) and (y[:, dim:] == 3).all()
    assert torch.equal(data[:, :width], m.data) and (data[:, width:] == 0xA5).all() and (scale[tiles:] == 0xA5).all()


def test_gradients_one_by_one():
    """dx without dweight and dweight without dx, which only the C ABI asks for."""
    for tokens, dim in ((5, 40), (300, 4096), (40, 16400)):
        h, dy, w = draw(80, tokens, dim), draw(81, tokens, dim), vector(82, dim)
        _, _, rstd = tc.rms_norm(h, w, eps=EPS, save=True)
        dx, dw = tc.rms_norm_backward(dy, h, w, rstd)
        ox, ow = torch.empty_like(h), torch.empty_like(w)
        ws = torch.empty(700 * dim * 4 // 256 * 256 + 256, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for px, pw in ((ox.data_ptr(), 0), (0, ow.data_ptr())):
            rc = tc.load_library().rms_norm_backward(struct.pack("16q", dy.data_ptr(), h.data_ptr(), w.data_ptr(), 0, rstd.data_ptr(), px, pw, dim,
                                                                 dim, 0, dim, tokens, dim, 1, ws.data_ptr(), ws.numel()), None)
            assert rc == 0
        torch.cuda.synchronize()
        assert torch.equal(ox, dx) and torch.equal(ow, dw)
