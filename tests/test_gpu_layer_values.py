"""The activations' tails on the GPU, relative to their own size."""
import math

import pytest

import layer_ref
import tensor_core_tiled_02_gb300 as tc

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def _status():
    yield
    rc, site = tc.gemm_f16_device_status(reset=True)
    assert rc == 0, f"a device wait gave up (site {site})"


def value64(act, x):
    """The activations without the cancellation of 1 + erf and 1 + tanh."""
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return 0.5 * x * torch.special.erfc(-x * math.sqrt(0.5))
    return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))


def fp32_room(act, x):
    """Relative error of the fp32 evaluation: the exponential's argument a is off by up to 2^-21
    of itself, which is a 2^-21 of the value, and a dozen operations and the fit of the tail
    (7.4e-7) add 16 x 2^-23."""
    a = {"silu": x.abs(), "gelu": 0.5 * x * x,
         "gelu_tanh": 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3).abs()}[act]
    return a * 2.0 ** -21 + 2.0 ** -19


# a sigmoid below 2^-126 comes out 0: what is left out is that times x, and in the slope of
# gelu_tanh times x (2 z)', some 2^8 where it happens
TINY = 2.0 ** -118


@pytest.mark.parametrize("tokens", [1, 5, 300, 2000])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activation_tails(act, dt, tokens):
    """x I = x exactly, so the output is the activation of a known 16-bit value, rounded once."""
    n = 256
    x = torch.linspace(-13, 13, tokens * n, device="cuda").reshape(tokens, n).to(dt)
    eye = torch.eye(n, device="cuda", dtype=dt)
    v = value64(act, x.double())
    room = (layer_ref.U[dt] + fp32_room(act, x.double())) * v.abs() + layer_ref.TINY[dt] + TINY
    got = tc.linear(x, eye, act=act)
    off = (got.double() - v).abs()
    worst = (off / room).argmax()
    assert (off <= room).all(), (x.flatten()[worst].item(), got.flatten()[worst].item(), v.flatten()[worst].item())


@pytest.mark.parametrize("tokens", [5, 300])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slope_tails(act, dt, tokens):
    """dpre = act'(pre) for dy = 1 and w = I.  The slope is value / x plus a term of the
    density's size, and its error relative to those two, not to their sum (it has a zero)."""
    n = 256
    pre = torch.linspace(-12, 12, tokens * n, device="cuda").reshape(tokens, n).to(dt)
    x = pre.double().requires_grad_(True)
    (want,) = torch.autograd.grad(value64(act, x).sum(), x)
    x = x.detach()
    first = torch.where(x == 0, torch.full_like(x, 0.5), value64(act, x) / torch.where(x == 0, torch.ones_like(x), x))
    size = first.abs() + (want - first).abs()
    room = layer_ref.U[dt] * want.abs() + fp32_room(act, x) * size + layer_ref.TINY[dt] + TINY
    eye, dy = torch.eye(n, device="cuda", dtype=dt), torch.ones(tokens, n, device="cuda", dtype=dt)
    dx, _, _ = tc.linear_backward(dy, torch.zeros_like(dy), eye, act=act, preact=pre)
    off = (dx.double() - want).abs()
    worst = (off / room).argmax()
    assert (off <= room).all(), (x.flatten()[worst].item(), dx.flatten()[worst].item(), want.flatten()[worst].item())
