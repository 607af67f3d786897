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

def leaning(t, k, v, dt, logit, seed=0):
    """States along their targets' rows: the target's logit is `logit`, the others' are near 0."""
    g = torch.Generator(device="cuda").manual_seed(seed + t + k + v)
    w = (torch.randn(v, k, generator=g, device="cuda") * k ** -0.5).to(dt)
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    rows = w[target].float()
    h = (rows * (logit / (rows * rows).sum(1, keepdim=True))).to(dt)
    return h, w, target


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("piece", [None, 256])
@pytest.mark.parametrize("shape", [(5, 1024, 300), (5, 8192, 4001), (100, 2056, 300), (100, 8192, 1000), (300, 2048, 1000),
                                   (300, 8192, 1000), (1100, 4104, 777), (1100, 8192, 600)], ids=str)
def test_gradient_of_sure_targets(shape, piece, dt):
    """Targets with 1 - p = 1.5e-4.  p - 1 is a difference of nearly equal values: exp takes the
    logit minus the log-sum-exp, both held in fp32, so p is off by at most some 2^-22 (1 + |lse|)
    of itself as long as both passes sum the logits alike, and p - 1 by that over 1 - p of itself.
    Row by row; d and dh take a rounding each (u / sqrt 3 on average, 2 u allowed).
    (Logits that differ by 8e-6 between the passes are off by all of 1 - p.)

    With pieces the passes may split the sums over the width differently, so the bound of
    test_precision_of_wide_logits is added for each of them."""
    t, k, v = shape
    logit = math.log(v / 1.5e-4)
    h, w, target = leaning(t, k, v, dt, logit)
    scale = 65536.0
    logits = h.double() @ w.double().T
    lse = torch.logsumexp(logits, 1)
    p = torch.exp(logits - lse[:, None])
    rows = torch.arange(t, device="cuda")
    # 1 - p without the cancellation
    rest = p.clone()
    rest[rows, target] = 0
    rest = rest.sum(1)
    d = p.clone()
    d[rows, target] = -rest
    want = (d @ w.double()) * (scale / t)
    _, got_lse = tc.linear_cross_entropy(h, w, target)
    dh, dw = tc.linear_cross_entropy_backward(torch.tensor(scale, device="cuda"), h, w, target, got_lse, piece=piece)
    room = 2.0 ** -22 * (1 + lse) / rest + 2 * U[dt]
    if piece is not None and piece < v:
        room = room + 2 * 128 * 2.0 ** -25 * logit / rest
    off = (dh.double() - want).norm(dim=1) / want.norm(dim=1)
    assert (off <= room).all(), (off.max().item(), room.min().item())
    want = (d.T @ h.double()) * (scale / t)
    off = (dw.double() - want).norm() / want.norm()
    assert off.item() <= room.max().item()


# widths on both sides of the runs in which the logits are summed (512 in fp16, 1024 in bf16), and
# off their multiples; one CTA, few tokens, pairs with one tile and with several
LONG = [(300, 520, 3001), (1100, 1024, 9000), (33, 4096, 5000), (200, 4096, 20011), (1, 2048, 1000), (1, 8192, 20011), (5, 2056, 300), (5, 4104, 4001), (100, 2056, 5000), (100, 8192, 20011),
        (300, 2048, 3001), (300, 2056, 257), (300, 4104, 20011), (300, 8192, 5001), (1100, 2056, 20011), (1100, 8192, 9000)]


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shape", LONG, ids=str)
def test_precision_of_wide_logits(shape, dt):
    """Targets whose logit's terms all have one sign, the worst for an accumulation that truncates.
    2^-18 of the largest logit is allowed for it, which the runs keep to (fp16 loses 6e-9 of the
    sum a unit of K, bf16 half that), and 2^-21 of what it handles for the rest, in fp32.  (Runs of
    2048 are low by 1.2e-5 and 6e-6, and fail.)"""
    t, k, v = shape
    h, w, target = leaning(t, k, v, dt, 14.0)
    logits = h.double() @ w.double().T
    lse = torch.logsumexp(logits, 1)
    loss = lse - logits.gather(1, target[:, None])[:, 0]
    most = logits.abs().amax(1)
    room = 2.0 ** -18 * most + 2.0 ** -21 * (1 + lse.abs())
    got, got_lse = tc.linear_cross_entropy(h, w, target, reduction="none")
    assert ((got_lse.double() - lse).abs() <= room).all(), ((got_lse.double() - lse).abs() / room).max().item()
    assert ((got.double() - loss).abs() <= 2 * room).all()
    total = tc.linear_cross_entropy(h, w, target, reduction="mean")[0].double().item()
    assert abs(total - loss.mean().item()) <= 2 * room.mean().item()
    # the bottom of the vocabulary too: a target in the last, ragged tile
    target = torch.full_like(target, v - 1)
    loss = lse - logits[:, v - 1]
    got, _ = tc.linear_cross_entropy(h, w, target, reduction="none")
    assert ((got.double() - loss).abs() <= 2 * room).all()


@pytest.mark.parametrize("piece", [None, 1024])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("tokens", [6, 40, 400, 1500])
def test_row_weights_of_very_different_size(tokens, dt, piece):
    """Reduction "none" with row gradients 2^26 apart: dh row by row.  A row takes the rounding
    of d and of dh, u / sqrt 3 each on average, and where its own entries near fp16's least
    normal 2^-25 of half an ulp more, below half a u here: 2 u allowed."""
    k, v = 64, 5000
    g = torch.Generator(device="cuda").manual_seed(tokens)
    h = torch.randn(tokens, k, generator=g, device="cuda").to(dt)
    w = (torch.randn(v, k, generator=g, device="cuda") * 0.25).to(dt)
    target = torch.randint(0, v, (tokens,), generator=g, device="cuda")
    weight = 2.0 ** torch.randint(-12, 15, (tokens,), generator=g, device="cuda").float()
    weight[0], weight[1] = 2.0 ** 14, 2.0 ** -12
    weight[2] *= -1
    target[3] = IGNORE
    weight[4] = 0
    logits = h.double() @ w.double().T
    p = torch.softmax(logits, 1)
    word = target.clamp(min=0)
    p[torch.arange(tokens, device="cuda"), word] -= 1
    p = p * (weight.double() * (target != IGNORE))[:, None]
    want, want_w = p @ w.double(), p.T @ h.double()
    _, lse = tc.linear_cross_entropy(h, w, target, ignore_index=IGNORE, reduction="none")
    dh, dw = tc.linear_cross_entropy_backward(weight, h, w, target, lse, ignore_index=IGNORE, reduction="none", piece=piece)
    assert torch.count_nonzero(dh[3]) == 0 and torch.count_nonzero(dh[4]) == 0
    keep = [i for i in range(tokens) if i not in (3, 4)]
    off = (dh.double() - want)[keep].norm(dim=1) / want[keep].norm(dim=1)
    assert (off <= 2 * U[dt]).all(), (off.max().item() / U[dt])
    # (a few entries of dw pass fp16's largest value and are infinite)
    fits = want_w.abs() <= torch.finfo(dt).max
    assert ((dw.double() - want_w)[fits & torch.isfinite(dw)].norm() / want_w[fits].norm()).item() <= 2 * U[dt]
    beyond = want_w.abs() > torch.finfo(dt).max * (1 - 4 * U[dt])
    assert not (torch.isinf(dw) & ~beyond).any() and not torch.isnan(dw).any()
    # a target that is no word makes its row NaN, and no other
    target[5] = v
    dh2, _ = tc.linear_cross_entropy_backward(weight, h, w, target, lse, ignore_index=IGNORE, reduction="none", piece=piece)
    keep = [i for i in range(tokens) if i != 5]
    assert torch.isnan(dh2[5]).all() and torch.equal(dh2[keep], dh[keep])


@pytest.mark.parametrize("reduction", [0, 1], ids=["none", "mean"])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("tokens", [7, 300])
def test_one_gradient_alone(tokens, dt, reduction):
    """Through the C ABI: dh or dw left out, in workspaces of their own size, the same bits."""
    import ctypes
    import struct

    lib = tc.load_library()
    k, v, piece = 72, 1500, 512
    g = torch.Generator(device="cuda").manual_seed(tokens)
    h = torch.randn(tokens, k, generator=g, device="cuda").to(dt)
    w = (torch.randn(v, k, generator=g, device="cuda") * 0.25).to(dt)
    target = torch.randint(0, v, (tokens,), generator=g, device="cuda")
    grad = 2.0 ** torch.randint(-9, 9, (tokens if reduction == 0 else 1,), generator=g, device="cuda").float()
    _, lse = tc.linear_cross_entropy(h, w, target)

    def run(want_h, want_w):
        dh = torch.full((tokens, k), 9.0, device="cuda", dtype=dt)
        dw = torch.full((v, k), 9.0, device="cuda", dtype=dt)
        fields = [h.data_ptr(), w.data_ptr(), target.data_ptr(), lse.data_ptr(), grad.data_ptr(),
                  dh.data_ptr() if want_h else 0, dw.data_ptr() if want_w else 0, k, k, k, k, tokens, k, v,
                  0 if dt == F16 else 1, IGNORE, reduction, 0, 0]
        size = ctypes.c_size_t()
        assert lib.linear_cross_entropy_backward_workspace(struct.pack("19q", *fields), piece, ctypes.byref(size)) == 0
        ws = torch.empty(size.value, device="cuda", dtype=torch.uint8)
        fields[-2:] = [ws.data_ptr(), size.value]
        torch.cuda.synchronize()
        assert lib.linear_cross_entropy_backward(struct.pack("19q", *fields), None) == 0
        torch.cuda.synchronize()
        return dh, dw, size.value

    dh, dw, both = run(True, True)
    only_h, kept_w, _ = run(True, False)
    kept_h, only_w, small = run(False, True)
    assert torch.equal(only_h, dh) and torch.equal(only_w, dw) and small < both
    assert (kept_w == 9).all() and (kept_h == 9).all()
    ph, pw = tc.linear_cross_entropy_backward(grad if reduction == 0 else grad[0], h, w, target, lse,
                                              ignore_index=IGNORE, reduction=("none", "mean")[reduction], piece=piece)
    assert torch.equal(ph, dh) and torch.equal(pw, dw)
