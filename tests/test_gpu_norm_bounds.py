"""The norm and its gradients against 64 bits with bounds from the kernels' own division of the work.

In units of 2^-24 of the magnitude at hand (one fp32 rounding each).  Forward, a thread adds the
squares of c columns one after the other: eight to each of its one, two or four vectors (rows beyond
32768 columns: its share of the row); then ten more in two trees.  The same back, with two vectors up
to 16384 columns.  rstd halves the sum's error and adds a division, a sum and a root (the last two
weigh half and one); y one more product (h w is exact).  dx: the mean is off by c + 10 of the mean of
magnitudes, its division and three products with rstd follow, then a product and two sums.  dweight: a block
adds its rows one after the other, the second kernel the blocks' sums, every 32nd one after the other, then five in a
tree; a term is exact but for the fused product with rstd, which counts with its sum.
"""
import math

import pytest

import mx_ref
import tensor_core_tiled_02_gb300 as tc
from layer_ref import V, check
from test_gpu_norm import EPS, ULP, draw, vector

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F16, BF16 = torch.float16, torch.bfloat16


def forward_columns(tokens, dim):
    vectors = math.ceil(dim / 8)
    if vectors > 4 * 1024:
        return 8 * math.ceil(dim / 8192)
    v = 1 if tokens * vectors <= 2048 * 152 else 2
    while vectors > 1024 * v:
        v *= 2
    return 8 * v


def gradient_plan(tokens, dim):
    """(columns a thread adds up, rows a block, blocks)"""
    vectors, threads = math.ceil(dim / 8), 64
    while threads < 2048 and 2 * threads < vectors:
        threads *= 2
    most = max(8, 608 // math.ceil(dim / 2048)) if threads > 1024 else 152 * (1 if threads >= 512 else 512 // threads)
    blocks = min(tokens, most)
    return 16 if threads <= 1024 else 8 * math.ceil(dim / 8192), math.ceil(tokens / blocks), blocks


SHAPES = [(1, 4096), (5000, 40), (5000, 264), (3000, 1003), (700, 4096), (330, 8192), (400, 16384), (200, 16392), (70, 32768), (60, 40007)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dt", [F16, BF16], ids=str)
def test_bounds_of_the_plan(shape, dt):
    t, d = shape
    h, dy, dh, w = draw(41, t, d, dt, 2.0), draw(42, t, d, dt, 0.1), draw(43, t, d, dt, 0.1), vector(44, d, dt)
    y, _, rstd = tc.rms_norm(h, w, eps=EPS, save=True)
    h64, w64, g = h.double(), w.double(), dy.double()
    r = (h64.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
    off = ((forward_columns(t, d) + 10) / 2 + 2.5) * ULP
    assert ((rstd.double()[:, None] - r).abs() <= 1.01 * off * r).all()
    want = h64 * w64 * r
    check(y, V(want, 1.01 * (off + ULP) * want.abs() + 2.0 ** -149), dt, 1.0, "y")

    c, rows, blocks = gradient_plan(t, d)
    r = rstd.double()[:, None]  # as saved
    gw = g * w64
    mean, size = (gw * h64).mean(1, keepdim=True), (gw * h64).abs().mean(1, keepdim=True)
    want = r * gw - h64 * r ** 3 * mean + dh.double()
    parts = (r * gw).abs() + h64.abs() * r ** 3 * size
    e = ULP * ((c + 10 + 4) * h64.abs() * r ** 3 * size + 2 * parts + want.abs() + dh.double().abs())
    dx, dw = tc.rms_norm_backward(dy, h, w, rstd, dh=dh)
    check(dx, V(want, 1.01 * e), dt, 1.0, "dx")
    terms = g * h64 * r
    bound = 1.01 * ULP * (rows + math.ceil(blocks / 32) + 5) * terms.abs().sum(0, keepdim=True)
    check(dw[None], V(terms.sum(0, keepdim=True), bound), dt, 1.0, "dweight")


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_ties_along_columns(fmt):
    """Values half way between two of the format's under a scale that a larger one fixes, through the
    kernel that quantises along columns (rows padded to a multiple of 8)."""
    t = torch.tensor(mx_ref.TABLE[fmt], dtype=torch.float64, device="cuda")
    half = (t[1:] + t[:-1]) / 2
    half = half[half >= 2.0 ** -8]  # in bf16's precision
    half = torch.cat((half, -half))
    half = torch.nn.functional.pad(half, (0, -len(half) % (31 * 8))).view(-1, 31)
    x = torch.cat((torch.full_like(half[:, :1], t[-1]), half), 1).to(BF16)
    assert len(x) % 8 == 0 and torch.equal(x.double()[:, 1:], half)
    m = tc.mx_quantize(x.T.contiguous(), fmt, transpose=True)
    want, byte = mx_ref.quantize(x, fmt)
    assert torch.equal(mx_ref.values(m), want) and torch.equal(mx_ref.scale_bytes(m, len(x))[0], byte)
    along = tc.mx_quantize(x, fmt)
    assert torch.equal(along.data, m.data)
