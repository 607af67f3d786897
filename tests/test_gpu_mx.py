"""Microscaled operands: quantisation bit for bit, the linear layer on them against 64 bits
with the bound of layer_ref.py (held values are exact, so only the products' sums and the
epilogue round)."""
import struct

import pytest

import mx_ref
import tensor_core_tiled_02_gb300 as tc
from layer_ref import V, check

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F16, BF16 = torch.float16, torch.bfloat16
FORMATS = ["e2m1", "e4m3"]


@pytest.fixture(autouse=True)
def _status():
    yield
    rc, site = tc.gemm_f16_device_status(reset=True)
    assert rc == 0, f"a device wait gave up (site {site})"


def draw(seed, rows, cols, dt=BF16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, (cols + 7) // 8 * 8, generator=g, device="cuda") * scale
    x *= torch.exp(torch.randn(x.shape[1], generator=g, device="cuda"))  # columns of many sizes
    return x.to(dt)[:, :cols]


def check_held(m, x, fmt):
    """m is x [rows, cols] held in the format, to the bit."""
    rows, cols = x.shape
    width = -(-cols // 32) * (32 if fmt == "e4m3" else 16)
    assert m.cols == cols and m.format == fmt and tuple(m.data.shape) == (rows, width)
    want, byte = mx_ref.quantize(x, fmt)
    got, behind = mx_ref.scale_bytes(m, rows)
    assert torch.equal(got, byte) and not behind.any()
    assert torch.equal(torch.nan_to_num(mx_ref.values(m), nan=1e300), torch.nan_to_num(want, nan=1e300))
    whole = mx_ref.values((m.data, m.scale, -(-cols // 32) * 32, fmt))[:, cols:]
    assert not torch.nan_to_num(whole).any(), "the last block is filled up with zeros"


SHAPES = [(1, 1), (1, 31), (1, 32), (3, 33), (32, 64), (33, 65), (127, 129), (128, 128), (130, 257), (5, 4096), (300, 1000), (257, 24)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", [F16, BF16], ids=str)
def test_quantize(shape, fmt, dt):
    x = draw(1, *shape, dt)
    check_held(tc.mx_quantize(x, fmt), x, fmt)
    check_held(tc.mx_quantize(x, fmt, transpose=True), x.T, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", [F16, BF16], ids=str)
def test_quantize_every_value(fmt, dt):
    """Every 16-bit value, NaN and infinities among them, in blocks of neighbours and in blocks
    of one exponent's range each."""
    bits = torch.arange(-32768, 32768, device="cuda", dtype=torch.int32).to(torch.int16).view(dt)
    for x in (bits.view(-1, 256), bits.view(256, 256).T.contiguous(), bits.view(-1, 8)):
        check_held(tc.mx_quantize(x, fmt), x, fmt)
        check_held(tc.mx_quantize(x, fmt, transpose=True), x.T, fmt)
        back = tc.mx_dequantize(tc.mx_quantize(x, fmt), dtype=dt)
        want, _ = mx_ref.quantize(x, fmt)
        assert torch.equal(torch.nan_to_num(back.double(), nan=1e300), torch.nan_to_num(want, nan=1e300))


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_ties(fmt):
    """Values half way between two of the format's, under a scale that a larger one fixes."""
    t = torch.tensor(mx_ref.TABLE[fmt], dtype=torch.float64, device="cuda")
    half = (t[1:] + t[:-1]) / 2
    half = half[half >= 2.0 ** -8]  # in bf16's precision
    half = torch.cat((half, -half))
    half = torch.nn.functional.pad(half, (0, -len(half) % 31)).view(-1, 31)
    x = torch.cat((torch.full_like(half[:, :1], t[-1]), half), 1).to(BF16)
    assert torch.equal(x.double()[:, 1:], half)
    check_held(tc.mx_quantize(x, fmt), x, fmt)
    check_held(tc.mx_quantize(x.T.contiguous()[:, : len(x) // 8 * 8 or None], fmt, transpose=True) if len(x) % 8 == 0 else
               tc.mx_quantize(x, fmt), x, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", [F16, BF16], ids=str)
def test_dequantize(fmt, dt):
    for rows, cols in SHAPES:
        m = tc.mx_quantize(draw(2, rows, cols, dt), fmt)
        assert torch.equal(tc.mx_dequantize(m, dtype=dt).double(), mx_ref.values(m))
    # every code under every scale
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(256, 1)
    cols = 256 if fmt == "e4m3" else 512
    byte = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None].repeat(1, cols // 32)
    scale = byte.view(-1, 4, 32, cols // 128, 4).permute(0, 3, 2, 1, 4).contiguous()
    m = (codes, scale, cols, fmt)
    got = tc.mx_dequantize(m, dtype=dt)
    want = mx_ref.values(m).float().to(dt)
    assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(want, nan=7.0)) and torch.equal(got.isnan(), want.isnan())


def test_quantize_views():
    """Rows of wider ones; nothing behind a row's bytes is written."""
    buf = draw(3, 70, 512)
    x = buf[2:68, 64:64 + 200]
    for fmt in FORMATS:
        check_held(tc.mx_quantize(x, fmt), x, fmt)
        check_held(tc.mx_quantize(x, fmt, transpose=True), x.T, fmt)
        width = 7 * (32 if fmt == "e4m3" else 16)
        for transpose, rows, w in ((0, 66, width), (1, 200, 3 * (32 if fmt == "e4m3" else 16))):
            data = torch.full((rows, w + 48), 0xA5, dtype=torch.uint8, device="cuda")
            tiles = -(-rows // 128) * (2 if not transpose else 1) * 512
            scale = torch.full((tiles + 64,), 0xA5, dtype=torch.uint8, device="cuda")
            torch.cuda.synchronize()
            rc = tc.load_library().mx_quantize(struct.pack("10q", x.data_ptr(), data.data_ptr(), scale.data_ptr(), 512, w + 48, 66, 200,
                                                           1, 0 if fmt == "e4m3" else 1, transpose), None)
            torch.cuda.synchronize()
            assert rc == 0
            want = tc.mx_quantize(x, fmt, transpose=bool(transpose))
            assert torch.equal(data[:, :w], want.data) and (data[:, w:] == 0xA5).all() and (scale[tiles:] == 0xA5).all()


# ---- the linear layer -----------------------------------------------------------------------

# tokens, k, n
PRODUCTS = [(1, 1, 1), (1, 32, 8), (1, 33, 5), (2, 64, 130), (3, 100, 7), (1, 4096, 512), (8, 1000, 300), (16, 96, 128), (17, 129, 257),
            (33, 2048, 200), (64, 512, 1000), (100, 640, 129), (128, 256, 256), (129, 4000, 131), (200, 1504, 640), (300, 72, 1031),
            (513, 2080, 520), (1000, 352, 1200), (2500, 224, 264), (4096, 128, 2048), (1, 16384, 136), (700, 8200, 264), (1300, 4200, 136), (2100, 2080, 72)]


def product(x, w):
    return V(mx_ref.values(x)) @ V(mx_ref.values(w)).T


@pytest.mark.parametrize("shape", PRODUCTS, ids=str)
@pytest.mark.parametrize("fmt", FORMATS)
def test_linear(shape, fmt):
    t, k, n = shape
    x, w = mx_ref.hold(draw(4, t, k), fmt), mx_ref.hold(draw(5, n, k, scale=k ** -0.5), fmt)
    want = product(x, w)
    for dt in (BF16, F16):
        check(tc.mx_linear(x, w, dtype=dt), want, dt, 1.0, "y")
    bias, r = draw(6, 1, n)[0].contiguous(), draw(7, t, n)
    check(tc.mx_linear(x, w, bias=bias, act="silu", residual=r), (want + V(bias[None])).act("silu") + V(r), BF16, 1.0, "epilogue")


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dt", [F16, BF16], ids=str)
@pytest.mark.parametrize("tokens", [3, 150, 1100])
def test_linear_epilogue(act, dt, tokens):
    k, n = 320, 520
    x, w = tc.mx_quantize(draw(8, tokens, k, dt, 0.3), "e4m3"), tc.mx_quantize(draw(9, n, k, dt, k ** -0.5), "e4m3")
    bias, r = draw(10, 1, n, dt)[0].contiguous(), draw(11, tokens, n, dt)
    want = (product(x, w) + V(bias[None])).act(act) + V(r)
    check(tc.mx_linear(x, w, bias=bias, act=act, residual=r, dtype=dt), want, dt, 1.0, act)
    out = r.clone()
    assert tc.mx_linear(x, w, bias=bias, act=act, residual=out, dtype=dt, out=out) is out
    check(out, want, dt, 1.0, "in place")


@pytest.mark.parametrize("tokens", [1, 5, 40, 300, 2500])
@pytest.mark.parametrize("n", [1, 7, 9, 123, 257, 1031])
def test_linear_behind_the_last_column(tokens, n):
    for k in (64, 2048):
        x, w = tc.mx_quantize(draw(12, tokens, k)), tc.mx_quantize(draw(13, n, k, scale=k ** -0.5))
        buf = torch.full((tokens, (n + 7) // 8 * 8 + 8), 3.0, dtype=BF16, device="cuda")
        tc.mx_linear(x, w, out=buf[:, :n])
        check(buf[:, :n], product(x, w), BF16, 1.0, "y")
        assert (buf[:, n:] == 3).all()


@pytest.mark.parametrize("tokens", [1, 6, 150, 1300])
@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_special_values(tokens, fmt):
    """A NaN block makes its row (or column) NaN and no other; the ends of the scales' range."""
    k, n = 416, 300
    xs, ws = draw(14, tokens, k), draw(15, n, k, scale=k ** -0.5)
    xs[tokens // 2, 70], ws[123, 415] = float("nan"), float("inf")
    x, w = tc.mx_quantize(xs, fmt), tc.mx_quantize(ws, fmt)
    y = tc.mx_linear(x, w)
    bad = torch.zeros(tokens, n, dtype=torch.bool, device="cuda")
    bad[tokens // 2], bad[:, 123] = True, True
    assert torch.equal(y.isnan(), bad)
    xs[tokens // 2, 70], ws[123, 415] = 0.0, 0.0
    # 2^-100 and 2^100, exact factors
    x, w = tc.mx_quantize(xs, fmt), tc.mx_quantize(ws, fmt)
    small = (x.data, torch.where(x.scale > 0, x.scale - 100, x.scale), k, fmt)
    large = (w.data, torch.where(w.scale > 0, w.scale + 100, w.scale), k, fmt)
    assert mx_ref.scale_bytes(x, tokens)[0].min() > 100 and mx_ref.scale_bytes(w, n)[0].max() < 155
    assert torch.equal(tc.mx_linear(small, large), tc.mx_linear(x, w))
    # all zero, and largest times largest: infinite
    zero = tc.mx_quantize(torch.zeros_like(xs), fmt)
    assert not tc.mx_linear(zero, w).any()
    most = (x.data, torch.full_like(x.scale, 254), k, fmt)
    top = (torch.full_like(w.data, 0x77 if fmt == "e2m1" else 0x7E), torch.full_like(w.scale, 254), k, fmt)
    ones = (torch.full_like(x.data, 0x77 if fmt == "e2m1" else 0x7E), most[1], k, fmt)
    assert (tc.mx_linear(ones, top) == float("inf")).all()


def test_linear_strided_operands():
    k, n, t = 256, 264, 140
    x, w = tc.mx_quantize(draw(16, t, k)), tc.mx_quantize(draw(17, n, k))
    buf = torch.zeros(t, 400, dtype=torch.uint8, device="cuda")
    buf[:, 32:32 + 128] = x.data
    view = (buf[:, 32:32 + 128], x.scale, k, "e2m1")
    assert torch.equal(tc.mx_linear(view, w), tc.mx_linear(x, w))
    assert torch.equal(tc.mx_dequantize(view), tc.mx_dequantize(x))


def test_no_tokens():
    w = tc.mx_quantize(draw(18, 64, 96))
    x = tc.mx_quantize(torch.zeros(0, 96, dtype=BF16, device="cuda"))
    assert tuple(x.data.shape) == (0, 48) and tuple(tc.mx_linear(x, w).shape) == (0, 64)
    assert tuple(tc.mx_dequantize(x).shape) == (0, 96)
    assert tuple(tc.mx_quantize(torch.zeros(96, 0, dtype=BF16, device="cuda"), transpose=True).data.shape) == (0, 48)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [100, 1000])
def test_gradients_straight_through(fmt, tokens):
    """dx and dw of y = x w as products of the same kind, operands quantised along the other axis."""
    k, n = 200, 328
    x, w, dy = draw(19, tokens, k, scale=0.5), draw(20, k, n, scale=k ** -0.5), draw(21, tokens, n, scale=0.1)
    q = lambda t: V(mx_ref.quantize(t, fmt)[0])  # noqa: E731
    check(tc.mx_linear(tc.mx_quantize(x, fmt), tc.mx_quantize(w, fmt, transpose=True)), q(x) @ q(w.T).T, BF16, 1.0, "y")
    check(tc.mx_linear(tc.mx_quantize(dy, fmt), tc.mx_quantize(w, fmt)), q(dy) @ q(w).T, BF16, 1.0, "dx")
    check(tc.mx_linear(tc.mx_quantize(x, fmt, transpose=True), tc.mx_quantize(dy, fmt, transpose=True)), q(x.T) @ q(dy.T).T, BF16, 1.0,
          "dw")


@pytest.mark.parametrize("tokens", [1, 9, 260, 1200])
def test_same_bits_on_another_stream_and_in_a_graph(tokens):
    k, n = 1056, 1304
    x, w = draw(22, tokens, k), tc.mx_quantize(draw(23, n, k))
    want = tc.mx_linear(tc.mx_quantize(x), w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = tc.mx_linear(tc.mx_quantize(x, stream=side), w, stream=side)
    side.synchronize()
    assert torch.equal(on_side, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = tc.mx_linear(tc.mx_quantize(x), w)
    for seed in (24, 25):
        x.copy_(draw(seed, tokens, k))
        g.replay()
        assert torch.equal(y, tc.mx_linear(tc.mx_quantize(x), w))


def test_refusals():
    x, w = tc.mx_quantize(draw(26, 8, 64)), tc.mx_quantize(draw(27, 16, 64))
    wide = tc.mx_quantize(draw(28, 16, 96))
    for call in (lambda: tc.mx_linear(x, wide), lambda: tc.mx_linear(x, tc.mx_quantize(draw(27, 16, 64), "e4m3")),
                 lambda: tc.mx_linear(x.data, w), lambda: tc.mx_linear(x, w, dtype=torch.float32), lambda: tc.mx_linear(x, w, act="softplus"),
                 lambda: tc.mx_linear((x.data[:, :16], x.scale, 64, "e2m1"), w), lambda: tc.mx_linear((x.data, x.scale[..., :2], 64, "e2m1"), w),
                 lambda: tc.mx_linear((x.data.float(), x.scale, 64, "e2m1"), w), lambda: tc.mx_linear(x, w, bias=draw(1, 1, 16, F16)[0]),
                 lambda: tc.mx_linear(x, w, residual=draw(1, 8, 24)), lambda: tc.mx_linear(x, w, out=draw(1, 9, 16)),
                 lambda: tc.mx_linear((x.data.cpu(), x.scale, 64, "e2m1"), w), lambda: tc.mx_linear((x.data, x.scale.cpu(), 64, "e2m1"), w),
                 lambda: tc.mx_linear((x.data, x.scale, -1, "e2m1"), w), lambda: tc.mx_linear((x.data, x.scale, "64", "e2m1"), w),
                 lambda: tc.mx_quantize(draw(1, 8, 64), "e5m2"), lambda: tc.mx_quantize(draw(1, 8, 64).float()),
                 lambda: tc.mx_quantize(draw(1, 8, 64).T), lambda: tc.mx_dequantize(x, dtype=torch.float32), lambda: tc.mx_dequantize(x[:2])):
        with pytest.raises(ValueError):
            call()
    for call, code in ((lambda: tc.mx_quantize(torch.zeros(8, 60, dtype=BF16, device="cuda")), -4),
                       (lambda: tc.mx_linear((torch.zeros(8, 40, dtype=torch.uint8, device="cuda")[:, :32], x.scale, 64, "e2m1"), w), -4),
                       (lambda: tc.mx_linear(x, w, out=x.data.view(BF16)), -5)):
        with pytest.raises(tc.GemmError) as e:
            call()
        assert e.value.code == code
