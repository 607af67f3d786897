"""The vocabulary cross entropy and the clipping of gradients on the GPU against
their definitions in 64 bits."""
import math

import pytest

import tensor_core_tiled_02_gb300 as tc
from layer_ref import U, V, check

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


def make(t, k, v, dt, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + t + v)
    pitch = (k + 7) // 8 * 8
    h = torch.randn(t, pitch, generator=g, device="cuda").to(dt)[:, :k]
    w = (torch.randn(v, pitch, generator=g, device="cuda") * scale * k ** -0.5).to(dt)[:, :k]
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    target[torch.rand(t, generator=g, device="cuda") < 0.2] = IGNORE
    return h, w, target


def forward_want(h, w, target):
    logits = V(h) @ V(w).T
    lse = torch.logsumexp(logits.v, 1)
    counts = target != IGNORE
    word = torch.where(counts, target, torch.zeros_like(target))
    picked = logits.v.gather(1, word[:, None])[:, 0]
    loss = torch.where(counts, lse - picked, torch.zeros_like(lse))
    # the log-sum-exp moves by at most the largest logit's error; exponentials, sums and the
    # logarithm in fp32 add 2^-20 each of what they handle
    err = logits.e.max(1).values
    room = err + 2.0 ** -20 * (1 + lse.abs())
    return logits, lse, loss, room, counts, word


SHAPES = [(1, 8, 1), (1, 64, 2), (1, 1024, 5000), (3, 64, 255), (8, 136, 257), (33, 520, 1000), (130, 77, 777),
          (257, 264, 3001), (300, 64, 20011), (520, 1032, 4096)]


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dt):
    h, w, target = make(*shape, dt, scale=2.0)
    _, lse, loss, room, counts, _ = forward_want(h, w, target)
    for reduction in ("none", "sum", "mean"):
        got, got_lse = tc.linear_cross_entropy(h, w, target, ignore_index=IGNORE, reduction=reduction)
        assert ((got_lse.double() - lse).abs() <= room).all()
        if reduction == "none":
            assert ((got.double() - loss).abs() <= 2 * room).all()
            assert (got[~counts] == 0).all()
        else:
            n = max(1, int(counts.sum())) if reduction == "mean" else 1
            assert abs(got.double().item() - loss.sum().item() / n) <= (2 * room[counts].sum().item() + 1e-6) / n


@pytest.mark.parametrize("piece", [None, 256, 512])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, dt, piece):
    t, k, v = shape
    h, w, target = make(t, k, v, dt, seed=1, scale=2.0)
    logits, lse, _, _, counts, word = forward_want(h, w, target)
    g = torch.Generator(device="cuda").manual_seed(9)
    for reduction in ("mean", "none"):
        if reduction == "mean":
            grad = torch.tensor(512.0 if dt == F16 else 0.5, device="cuda")
            weight = torch.where(counts, grad.double() / max(1, int(counts.sum())), torch.zeros_like(lse))
        else:
            grad = torch.randn(t, generator=g, device="cuda") * 4
            weight = torch.where(counts, grad.double(), torch.zeros_like(lse))
        _, got_lse = tc.linear_cross_entropy(h, w, target, ignore_index=IGNORE, reduction=reduction)
        dh, dw = tc.linear_cross_entropy_backward(grad, h, w, target, got_lse, ignore_index=IGNORE,
                                                  reduction=reduction, piece=piece)
        p = torch.exp(logits.v - lse[:, None])
        one = torch.zeros_like(p)
        one[torch.arange(t, device="cuda"), word] = 1.0
        # p moves by its logit's and its row's error; exp in fp32 by 2^-18 of itself, the
        # difference by a rounding, the 16 bits by u
        pe = p * (2.0 * (logits.e + logits.e.max(1).values[:, None]) + 2.0 ** -18 * (1 + lse.abs()[:, None])) + 2.0 ** -22
        pe = torch.where(p < 1e-6, torch.minimum(pe, 1e-3 * p + 2.0 ** -30), pe)
        d = V((p - one) * weight[:, None], pe * weight.abs()[:, None])
        d = V(d.v, d.e + U[dt] * (d.v.abs() + d.e) + 2.0 ** -38 * weight.abs().max())
        check(dh, d @ V(w), dt, 1.3, "dh")
        check(dw, d.T @ V(h), dt, 1.3, "dw")
        assert torch.count_nonzero(dh[~counts]) == 0


def test_gradient_against_differences():
    """As for the gated block: the inner product with a direction against the central
    difference of the definition."""
    dt = BF16
    h, w, target = make(60, 72, 333, dt, seed=5, scale=2.0)
    loss, lse = tc.linear_cross_entropy(h, w, target, ignore_index=IGNORE)
    dh, dw = tc.linear_cross_entropy_backward(torch.ones((), device="cuda"), h, w, target, lse, ignore_index=IGNORE)
    keep = target != IGNORE

    def value(a, b):
        logits = (a @ b.T)[keep]
        return (torch.logsumexp(logits, 1) - logits.gather(1, target[keep][:, None])[:, 0]).mean()

    g = torch.Generator(device="cuda").manual_seed(2)
    for i, grad in enumerate((dh, dw)):
        base = [h.double(), w.double()]
        way = torch.randn(base[i].shape, generator=g, device="cuda", dtype=torch.float64)
        eps = 1e-5
        up = value(*[b + eps * way if j == i else b for j, b in enumerate(base)])
        down = value(*[b - eps * way if j == i else b for j, b in enumerate(base)])
        want = ((up - down) / (2 * eps)).item()
        got = (grad.double() * way).sum().item()
        assert abs(got - want) <= 6 * U[dt] * grad.double().norm().item(), (i, got, want)


def test_nothing_counts_and_bad_targets():
    h, w, target = make(40, 64, 300, F16)
    target[:] = IGNORE
    loss, lse = tc.linear_cross_entropy(h, w, target, ignore_index=IGNORE)
    assert loss.item() == 0.0 and torch.isfinite(lse).all()
    dh, dw = tc.linear_cross_entropy_backward(torch.ones((), device="cuda"), h, w, target, lse, ignore_index=IGNORE)
    assert torch.count_nonzero(dh) == 0 and torch.count_nonzero(dw) == 0
    target[3], target[4], target[5] = 7, 300, -1  # a word, and two that are none
    loss, lse = tc.linear_cross_entropy(h, w, target, ignore_index=IGNORE, reduction="none")
    assert torch.isfinite(loss[3]) and torch.isnan(loss[4]) and torch.isnan(loss[5])
    assert (loss[torch.tensor([0, 1, 2, 6, 39], device="cuda")] == 0).all()
    assert math.isnan(tc.linear_cross_entropy(h, w, target, ignore_index=IGNORE)[0].item())
    # ignore_index may be a word
    loss, _ = tc.linear_cross_entropy(h, w, torch.full_like(target, 7), ignore_index=7, reduction="none")
    assert (loss == 0).all()


def test_masked_rows_may_hold_anything_in_the_forward_pass():
    h, w, target = make(64, 64, 500, BF16)
    target[:] = 3
    target[10] = target[20] = IGNORE
    clean = tc.linear_cross_entropy(h, w, target, ignore_index=IGNORE)[0]
    h = h.clone()
    h[10], h[20, 5] = float("nan"), float("inf")
    assert torch.equal(tc.linear_cross_entropy(h, w, target, ignore_index=IGNORE)[0], clean)


def test_large_logits_and_words_ruled_out():
    """Logits of hundreds; and words whose weights make their logits the lowest of the type."""
    h, w, target = make(50, 64, 700, BF16)
    h, w = h * 8, w * 8
    _, lse, loss, room, counts, _ = forward_want(h, w, target)
    got, got_lse = tc.linear_cross_entropy(h, w, target, ignore_index=IGNORE, reduction="none")
    assert ((got_lse.double() - lse).abs() <= room).all() and ((got.double() - loss).abs() <= 2 * room).all()
    h = torch.ones(4, 8, device="cuda", dtype=BF16)
    w = torch.zeros(600, 8, device="cuda", dtype=BF16)
    w[:590, 0] = -3e38  # the first tiles hold nothing else
    t = torch.full((4,), 595, device="cuda")
    got, got_lse = tc.linear_cross_entropy(h, w, t, reduction="none")
    assert torch.allclose(got_lse, torch.full((4,), math.log(10.0), device="cuda"), atol=1e-6)
    assert torch.allclose(got, got_lse)


def test_no_tokens_and_repeats():
    w = torch.randn(300, 64, device="cuda").half()
    h, t = torch.empty(0, 64, device="cuda", dtype=F16), torch.empty(0, device="cuda", dtype=torch.int64)
    loss, lse = tc.linear_cross_entropy(h, w, t)
    assert loss.item() == 0 and lse.numel() == 0
    dh, dw = tc.linear_cross_entropy_backward(torch.ones((), device="cuda"), h, w, t, lse)
    assert dh.numel() == 0 and torch.count_nonzero(dw) == 0
    h, w, t = make(300, 264, 5001, BF16)
    side = torch.cuda.Stream()
    runs = []
    for stream in (None, side, None):
        torch.cuda.synchronize()
        loss, lse = tc.linear_cross_entropy(h, w, t, stream=stream)
        runs.append((loss, lse) + tc.linear_cross_entropy_backward(torch.ones((), device="cuda"), h, w, t, lse, piece=1024,
                                                                   stream=stream))
        torch.cuda.synchronize()
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


def test_loss_refusals():
    h, w, target = make(8, 64, 300, F16)
    one = torch.ones((), device="cuda")
    with pytest.raises(ValueError):
        tc.linear_cross_entropy(h, w, target.int())
    with pytest.raises(ValueError):
        tc.linear_cross_entropy(h, w.bfloat16(), target)
    with pytest.raises(ValueError):
        tc.linear_cross_entropy(h, w, target[:7])
    with pytest.raises(ValueError):
        tc.linear_cross_entropy(h, w, target, reduction="max")
    loss, lse = tc.linear_cross_entropy(h, w, target)
    with pytest.raises(ValueError):
        tc.linear_cross_entropy_backward(one, h, w, target, lse[:3])
    with pytest.raises(ValueError):
        tc.linear_cross_entropy_backward(one, h, w, target, lse, reduction="none")
    with pytest.raises(tc.GemmError):
        tc.linear_cross_entropy_backward(one, h, w, target, lse, piece=100)


# ---- clipping ---------------------------------------------------------------------


def clip_want(grads, max_norm):
    norm = math.sqrt(sum((g.double() ** 2).sum().item() for g in grads))
    return norm, min(1.0, max_norm / (norm + 1e-6))


def clip_check(got, grads, coef):
    for a, g in zip(got, grads):
        want = g.double() * coef
        u = {torch.float32: 2.0 ** -23, F16: 2.0 ** -11, BF16: 2.0 ** -8}[g.dtype]
        tiny = {torch.float32: 2.0 ** -149, F16: 2.0 ** -24, BF16: 2.0 ** -133}[g.dtype]
        # the norm's and the coefficient's own error (below), then one rounding
        assert ((a.double() - want).abs() <= (u + 2e-6) * want.abs() + tiny).all()


@pytest.mark.parametrize("max_norm", [0.0, 0.7, 1e6])
@pytest.mark.parametrize("sizes", [[1], [7, 0, 1], [32768], [32769, 5], [100000, 3, 65536, 12345], [777] * 60,
                                   [33] * 1100, [3_000_001, 17]], ids=lambda s: f"{len(s)}x{s[0]}")
def test_clip(sizes, max_norm):
    g = torch.Generator(device="cuda").manual_seed(len(sizes))
    kinds = [torch.float32, F16, BF16]
    # fp32 sums of squares: at most 2^-24 per addition of up to 64 terms, fp64 beyond
    for mixed in (False, True):
        # end to end in one buffer per type, so that most start off a 16-byte boundary
        n = sum(sizes)
        flat = {k: torch.randn(n, generator=g, device="cuda").to(k) for k in (kinds if mixed else [BF16])}
        grads, at = [], 0
        for i, s in enumerate(sizes):
            grads.append(flat[kinds[i % 3] if mixed else BF16][at:at + s])
            at += s
        norm, coef = clip_want(grads, max_norm)
        outs = [torch.full_like(x, 9) for x in grads]
        before = [x.clone() for x in grads]
        got = tc.clip_grad_norm(grads, max_norm, out=outs)
        assert abs(got.item() - norm) <= 2e-6 * norm
        clip_check(outs, before, coef)
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
        shifted = [torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:] for x in grads]  # another alignment
        tc.clip_grad_norm(grads, max_norm, out=shifted)
        assert all(torch.equal(a, b) for a, b in zip(shifted, outs))
        tc.clip_grad_norm(grads, max_norm)
        assert all(torch.equal(a, b) for a, b in zip(grads, outs))


def test_clip_special_values():
    for bad, coef in ((float("inf"), 0.0), (float("nan"), float("nan"))):
        a, b = torch.ones(1000, device="cuda"), torch.ones(50, device="cuda", dtype=BF16)
        a[77] = bad
        norm = tc.clip_grad_norm([a, b], 1.0)
        assert torch.isnan(norm) if math.isnan(bad) else torch.isinf(norm)
        assert torch.isnan(a[77]) and (torch.isnan(b).all() if math.isnan(coef) else (b == 0).all())


def test_clip_leaves_small_gradients_alone():
    a = torch.randn(40001, device="cuda").half() * 1e-3
    keep = a.clone()
    norm = tc.clip_grad_norm([a], 1e9)
    assert torch.equal(a, keep) and abs(norm.item() - keep.double().norm().item()) <= 2e-6 * norm.item()


def test_clip_refusals():
    a = torch.ones(10, device="cuda")
    for args in (([],), ([a.cpu()],), ([a.double()],), ([a, a.cpu()],), ([torch.ones(4, 6, device="cuda").T],)):
        with pytest.raises(ValueError):
            tc.clip_grad_norm(*args, 1.0)
    with pytest.raises(ValueError):
        tc.clip_grad_norm([a], 1.0, out=[a, a])
    with pytest.raises(ValueError):
        tc.clip_grad_norm([a], 1.0, out=[a.half()])
    with pytest.raises(tc.GemmError):
        tc.clip_grad_norm([a], -1.0)
    big = torch.ones(100, device="cuda")
    with pytest.raises(tc.GemmError) as e:
        tc.clip_grad_norm([big[:90]], 1.0, out=[big[5:95]])
    assert e.value.code == -5
