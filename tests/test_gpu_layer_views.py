"""Column ranges of one buffer as operands and outputs of one call."""
import pytest

import tensor_core_tiled_02_gb300 as tc
from layer_ref import V, check

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def draw(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


# tokens for each kernel; widths that end inside a 32-byte sector and at the stride
@pytest.mark.parametrize("tokens", [1, 2, 5, 40, 300, 2500])
@pytest.mark.parametrize("k,n,stride", [(264, 520, 800), (264, 123, 392), (128, 1000, 1128)])
def test_side_by_side(tokens, k, n, stride):
    """x, out and a guard between them in one buffer, in either order; then the residual too."""
    w = draw(1, k, (n + 7) // 8 * 8, scale=k ** -0.5)[:, :n]
    x = draw(2, tokens, k)
    want = V(x) @ V(w)
    pad = (n + 7) // 8 * 8
    for x_at, y_at in ((0, stride - pad), (stride - k, 0)):
        buf = torch.full((tokens, stride), 3.0, device="cuda", dtype=torch.bfloat16)
        buf[:, x_at:x_at + k] = x
        out = buf[:, y_at:y_at + n]
        tc.linear(buf[:, x_at:x_at + k], w, out=out)
        check(out, want, torch.bfloat16, 1.0, "y")
        assert torch.equal(buf[:, x_at:x_at + k], x)
        rest = torch.ones(stride, dtype=torch.bool)
        rest[x_at:x_at + k] = rest[y_at:y_at + n] = False
        assert (buf[:, rest.cuda()] == 3).all()
    # two outputs and the residual as column ranges
    r = draw(3, tokens, n)
    wide = torch.zeros(tokens, 2 * pad, device="cuda", dtype=torch.bfloat16)
    wide[:, :n] = r
    tc.linear(x, w, residual=wide[:, :n], out=wide[:, pad:pad + n])
    check(wide[:, pad:pad + n], want + V(r), torch.bfloat16, 1.0, "beside the residual")
    assert torch.equal(wide[:, :n], r)


def test_shared_columns_are_refused():
    buf = torch.zeros(16, 512, device="cuda", dtype=torch.float16)
    w = torch.zeros(256, 256, device="cuda", dtype=torch.float16)
    cases = [buf[:, 248:504], buf[:, 8:264], buf[1:, 256:][:15], buf.view(32, 256)[1::2]]
    for out in cases[:2]:
        with pytest.raises(tc.GemmError) as e:
            tc.linear(buf[:, :256], w, out=out)
        assert e.value.code == -5
    tc.linear(buf[:15, :256], w, out=cases[2])  # other rows, other columns
    tc.linear(buf[:, :256], w, out=cases[3])
    with pytest.raises(tc.GemmError) as e:      # rows and columns of other rows, another stride
        tc.linear(buf[:, :256], w, out=torch.as_strided(buf, (16, 256), (256, 1), 256))
    assert e.value.code == -5
