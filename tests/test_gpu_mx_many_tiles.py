"""Microscaled products whose tiles come in several generations: few tokens on a vocabulary's width of
weights, many tokens on short K; against 64 bits with the bound of layer_ref.py."""
import pytest

import mx_ref
import tensor_core_tiled_02_gb300 as tc
from layer_ref import V, check
from test_mx_choice import times  # noqa: F401  (a fixture)

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _status():
    yield
    rc, site = tc.gemm_f16_device_status(reset=True)
    assert rc == 0, f"a device wait gave up (site {site})"


def draw(seed, rows, cols, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, (cols + 7) // 8 * 8, generator=g, device="cuda") * scale).to(BF16)[:, :cols]


def product(x, w, chunk=8192):
    """In pieces of w's rows: 64 bits of a wide product take room."""
    v = V(mx_ref.values(x))
    parts = [v @ V(p).T for p in mx_ref.values(w).split(chunk)]
    return V(torch.cat([p.v for p in parts], 1), torch.cat([p.e for p in parts], 1))


@pytest.mark.parametrize("tokens,k,n", [(1, 96, 41000), (5, 33, 60001), (16, 2080, 40008), (48, 256, 78000), (100, 1056, 40100)])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_few_tokens_more_tiles_than_fit_at_once(tokens, k, n, fmt, times):  # noqa: F811
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert -(-n // 128) > 2 * sms
    if tokens < 48:
        few, pairs = times(fmt, tokens, k, n, True, sms)
        assert few <= pairs, "on the kernel for few tokens"
    x, w = tc.mx_quantize(draw(1, tokens, k), fmt), tc.mx_quantize(draw(2, n, k, k ** -0.5), fmt)
    bias, r = draw(3, 1, n)[0].contiguous(), draw(4, tokens, n)
    want = product(x, w)
    check(tc.mx_linear(x, w), want, BF16, 1.0, "y")
    check(tc.mx_linear(x, w, bias=bias, act="gelu", residual=r), (want + V(bias[None])).act("gelu") + V(r), BF16, 1.0, "epilogue")


@pytest.mark.parametrize("tokens,k,n", [(8192, 64, 1100), (2600, 200, 4100), (5000, 129, 2050)])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_many_tokens_on_short_k(tokens, k, n, fmt, times):  # noqa: F811
    few, pairs = times(fmt, tokens, k, n, True, torch.cuda.get_device_properties(0).multi_processor_count)
    assert pairs < few, "on CTA pairs"
    x, w = tc.mx_quantize(draw(5, tokens, k), fmt), tc.mx_quantize(draw(6, n, k, k ** -0.5), fmt)
    r = draw(7, tokens, n)
    want = product(x, w)
    check(tc.mx_linear(x, w), want, BF16, 1.0, "y")
    out = draw(7, tokens, n)
    tc.mx_linear(x, w, act="relu", residual=out, out=out)
    check(out, want.act("relu") + V(r), BF16, 1.0, "in place")
