"""The cross entropy's values where single rows go wrong: infinite losses, widths over
which the logits are summed in several runs, targets the model is sure of, row
weights of very different size.  References in 64 bits; each test derives its bound."""
import math

import pytest

import tensor_core_tiled_02_gb300 as tc
from layer_ref import U

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F16, BF16 = torch.float16, torch.bfloat16
IGNORE = -100


@pytest.fixture(autouse=True)
def _status():
    yield
    rc, site = tc.gemm_f16_device_status(reset=True)
    assert rc == 0, f"a device wait gave up (site {site})"


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 32, 1000, 1025, 3000])
def test_infinite_loss(tokens, dt):
    """A target whose logit is -inf has an infinite loss, and so have the sum and the mean."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    h = (torch.randn(tokens, 16, generator=g, device="cuda") * 0.1).to(dt)
    h[:, 0] = 1
    w = (torch.randn(300, 16, generator=g, device="cuda") * 0.1).to(dt)
    w[0, 0] = float("-inf")
    target = torch.randint(1, 300, (tokens,), generator=g, device="cuda")
    for rows in ([0], [0, tokens - 1]):
        t = target.clone()
        t[rows] = 0
        each, lse = tc.linear_cross_entropy(h, w, t, reduction="none")
        assert torch.isfinite(lse).all()
        assert (each[rows] == math.inf).all() and int(torch.isinf(each).sum()) == len(set(rows))
        for reduction in ("sum", "mean"):
            assert tc.linear_cross_entropy(h, w, t, reduction=reduction)[0].item() == math.inf
            # where another row's loss is NaN, so is theirs
            if tokens > 1:
                bad = t.clone()
                bad[1] = 300
                assert math.isnan(tc.linear_cross_entropy(h, w, bad, reduction=reduction)[0].item())
        t[rows] = IGNORE
        if tokens > 2:
            assert math.isfinite(tc.linear_cross_entropy(h, w, t, ignore_index=IGNORE)[0].item())
