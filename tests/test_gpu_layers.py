"""The linear layer and the gated feed-forward block on the GPU against their
definitions in 64 bits (layer_ref.py derives the tolerances)."""
import pytest

import layer_ref
import tensor_core_tiled_02_gb300 as tc
from layer_ref import V, check

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F16, BF16 = torch.float16, torch.bfloat16
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(autouse=True)
def _status():
    yield
    rc, site = tc.gemm_f16_device_status(reset=True)
    assert rc == 0, f"a device wait gave up (site {site})"


class Draw:
    def __init__(self, seed, dt):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.dt = dt

    def __call__(self, *shape, scale=1.0, pitch=None):
        if pitch is None:
            pitch = (shape[-1] + 7) // 8 * 8
        wide = shape[:-1] + (pitch,)
        t = (torch.randn(*wide, generator=self.g, device="cuda") * scale).to(self.dt)
        return t[..., :shape[-1]]


def linear_want(x, w, bias, act, residual):
    pre = V(x) @ V(w)
    if bias is not None:
        pre = pre + V(bias)
    y = pre.act(act)
    return pre, (y + V(residual) if residual is not None else y)


# tokens, k, n: one token, one tile, ragged on every side, more tiles than SM pairs, one
# column over a tile, K shorter than a step, odd widths (rows padded to 8)
SHAPES = [(1, 8, 8), (1, 4096, 512), (2, 520, 1000), (7, 256, 4096), (17, 1031, 777), (33, 64, 264), (64, 2048, 512),
          (129, 200, 257), (200, 1000, 1544), (256, 64, 256), (257, 72, 520), (300, 4096, 1024), (511, 136, 2056),
          (1000, 520, 4096), (2500, 264, 5000)]


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear(shape, dt):
    t, k, n = shape
    d = Draw(t * 7 + k, dt)
    for i, (act, bias, residual) in enumerate([(None, False, False), ("gelu_tanh", True, True), ("silu", True, False)]):
        x, w = d(t, k), d(k, n, scale=k ** -0.5)
        b = d(n)[:n].contiguous() if bias else None
        r = d(t, n) if residual else None
        pre, want = linear_want(x, w, b, act, r)
        y, p = tc.linear(x, w, bias=b, act=act, residual=r, save_preact=True)
        check(y, want, dt, 1.0, f"y {i}")
        check(p, pre, dt, 1.0, f"preact {i}")
        check(tc.linear(x, w, bias=b, act=act, residual=r), want, dt, 1.0, f"y alone {i}")


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("act", ACTS, ids=str)
@pytest.mark.parametrize("tokens", [5, 300])
def test_linear_activations(act, dt, tokens):
    """Every activation over the range where it bends, saturates and ends."""
    d = Draw(3, dt)
    x, w = d(tokens, 64, scale=2.0), d(64, 328, scale=0.5)
    x[0] = 0
    pre, want = linear_want(x, w, None, act, None)
    check(tc.linear(x, w, act=act), want, dt, 1.0, str(act))


def test_linear_residual_in_place_and_strided_views():
    d = Draw(11, BF16)
    for t in (3, 300):
        x, w = d(t, 264, pitch=320), d(264, 520, pitch=1024)
        r = d(t, 520, pitch=528)
        _, want = linear_want(x, w, None, "relu", r)
        y = tc.linear(x, w, act="relu", residual=r, out=r)
        assert y is r
        check(y, want, BF16, 1.0, "in place")


def test_linear_masked_and_special_values():
    """Rows of zeros stay exact; an infinity or a NaN in one row of x stays in that row."""
    d = Draw(5, F16)
    for t in (4, 300):
        x, w = d(t, 256), d(256, 512, scale=0.06)
        clean = tc.linear(x, w, act="silu")
        x2 = x.clone()
        x2[1] = float("nan")
        x2[2, 7] = float("inf")
        y = tc.linear(x2, w, act="silu")
        assert torch.isnan(y[1]).all()
        keep = [i for i in range(t) if i not in (1, 2)]
        assert torch.equal(y[keep], clean[keep])
        zero = tc.linear(torch.zeros_like(x), w)
        assert torch.count_nonzero(zero).item() == 0


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("act", ACTS, ids=str)
@pytest.mark.parametrize("shape", [(1, 8, 16), (5, 520, 264), (65, 1000, 1544), (300, 136, 777), (513, 264, 2056)],
                         ids=str)
def test_linear_backward(shape, act, dt):
    t, k, n = shape
    d = Draw(t + k, dt)
    x, w, dy, pre = d(t, k), d(k, n, scale=k ** -0.5), d(t, n), d(t, n, scale=2.0)
    dx, dw, db = tc.linear_backward(dy, x, w, act=act, preact=pre, bias=True)
    full = V(dy) * V(pre).slope(act)
    dpre = full if act is None else full.round(dt)
    check(dx, dpre @ V(w).T, dt, 1.2, "dx")
    check(dw, V(x).T @ dpre, dt, 1.2, "dw")
    ones = V(torch.ones(1, t, device="cuda", dtype=torch.float64))
    check(db[None], ones @ full, dt, 1.2, "dbias")
    _, _, none = tc.linear_backward(dy, x, w, act=act, preact=pre)
    assert none is None


GATED = [(1, 8, 8, 8), (1, 4096, 1024, 512), (3, 256, 1000, 264), (9, 520, 777, 1031), (40, 1024, 264, 136),
         (130, 264, 400, 520), (256, 64, 128, 64), (300, 1000, 520, 264), (700, 200, 1544, 1000)]


def gated_want(x, wg, wu, wd, act, r, dt):
    gate, up = V(x) @ V(wg), V(x) @ V(wu)
    hidden = gate.act(act) * up
    y = hidden.round(dt) @ V(wd)
    return gate, up, hidden, (y + V(r) if r is not None else y)


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shape", GATED, ids=str)
def test_gated_ffn(shape, dt):
    t, k, f, o = shape
    d = Draw(t * 3 + f, dt)
    x, wg, wu, wd = d(t, k), d(k, f, scale=k ** -0.5), d(k, f, scale=k ** -0.5), d(f, o, scale=f ** -0.5)
    for act, residual in (("silu", True), ("gelu", False), ("relu", True)):
        r = d(t, o) if residual else None
        gate, up, hidden, want = gated_want(x, wg, wu, wd, act, r, dt)
        y, g, u, h = tc.gated_ffn(x, wg, wu, wd, act=act, residual=r, save=True)
        check(g, gate, dt, 1.0, "gate")
        check(u, up, dt, 1.0, "up")
        check(h, hidden, dt, 1.0, "hidden")
        check(y, want, dt, 1.2, "y")
        check(tc.gated_ffn(x, wg, wu, wd, act=act, residual=r), want, dt, 1.2, "y, nothing kept")


@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("shape", GATED, ids=str)
def test_gated_ffn_backward(shape, act, dt):
    t, k, f, o = shape
    d = Draw(t * 5 + f, dt)
    x, wg, wu, wd = d(t, k), d(k, f, scale=k ** -0.5), d(k, f, scale=k ** -0.5), d(f, o, scale=f ** -0.5)
    dy, g, u, h = d(t, o), d(t, f, scale=1.5), d(t, f), d(t, f)
    dx, dwg, dwu, dwd = tc.gated_ffn_backward(dy, x, wg, wu, wd, g, u, h, act=act)
    dh = V(dy) @ V(wd).T
    dg = (dh * V(u) * V(g).slope(act)).round(dt)
    du = (dh * V(g).act(act)).round(dt)
    check(dx, dg @ V(wg).T + du @ V(wu).T, dt, 1.2, "dx")
    check(dwg, V(x).T @ dg, dt, 1.2, "dw_gate")
    check(dwu, V(x).T @ du, dt, 1.2, "dw_up")
    check(dwd, V(h).T @ V(dy), dt, 1.0, "dw_down")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_ffn_gradient_against_differences(act):
    """<gradient, direction> against the central difference of the definition in
    64 bits, forward values as the kernels kept them.  The difference's own error is
    below 1e-6 at this step; the kernels' gradients carry three roundings (u each, of
    independent entries), so the sums of thousands of entries agree within
    6 u |gradient| |direction| / sqrt(entries) with room."""
    dt = BF16
    d = Draw(21, dt)
    t, k, f, o = 70, 136, 264, 72
    ws = [d(t, k), d(k, f, scale=k ** -0.5), d(k, f, scale=k ** -0.5), d(f, o, scale=f ** -0.5)]
    dy = d(t, o)
    _, g, u, h = tc.gated_ffn(*ws, act=act, save=True)
    grads = tc.gated_ffn_backward(dy, *ws, g, u, h, act=act)

    def value(x, wg, wu, wd):
        return (((layer_ref.act64(act, x @ wg) * (x @ wu)) @ wd) * dy.double()).sum()

    base = [w.double() for w in ws]
    for i in range(4):
        way = torch.randn(base[i].shape, generator=d.g, device="cuda", dtype=torch.float64)
        eps = 1e-5
        up = value(*[b + eps * way if j == i else b for j, b in enumerate(base)])
        down = value(*[b - eps * way if j == i else b for j, b in enumerate(base)])
        want = ((up - down) / (2 * eps)).item()
        got = (grads[i].double() * way).sum().item()
        room = 6 * layer_ref.U[dt] * grads[i].double().norm().item()
        assert abs(got - want) <= room, (i, got, want, room)


def test_no_tokens():
    d = Draw(1, F16)
    x, w = torch.empty(0, 64, dtype=F16, device="cuda"), d(64, 128)
    assert tc.linear(x, w).shape == (0, 128)
    dx, dw, db = tc.linear_backward(torch.empty(0, 128, dtype=F16, device="cuda"), x, w, bias=True)
    assert dx.shape == (0, 64) and torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0
    e = torch.empty(0, 128, dtype=F16, device="cuda")
    assert tc.gated_ffn(x, w, w, d(128, 64)).shape == (0, 64)
    grads = tc.gated_ffn_backward(x, x, w, w, d(128, 64), e, e, e)
    assert all(torch.count_nonzero(g) == 0 for g in grads)


def test_deterministic_on_another_stream_and_in_a_graph():
    d = Draw(8, BF16)
    side = torch.cuda.Stream()
    for t in (2, 30, 600):
        x, wg, wu, wd = d(t, 520), d(520, 1544, scale=0.04), d(520, 1544, scale=0.04), d(1544, 520, scale=0.03)
        r = d(t, 520)
        first = tc.gated_ffn(x, wg, wu, wd, residual=r, save=True)
        torch.cuda.synchronize()
        again = tc.gated_ffn(x, wg, wu, wd, residual=r, save=True, stream=side)
        side.synchronize()
        for a, b in zip(first, again):
            assert torch.equal(a, b)
        out = torch.empty_like(r)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tc.gated_ffn(x, wg, wu, wd, residual=r, out=out)
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, first[0])


# Shapes at which the choice of kernel and split differs on a 152-SM part: tokens, k, n
KINDS = [(8, 4096, 512),       # few tokens, 16 CTAs a weight tile
         (3, 2048, 1024), (40, 4096, 14336),
         (150, 1024, 4096),    # token tiles of one CTA an SM
         (600, 1024, 1024),    # several token tiles
         (256, 14336, 4096), (512, 4096, 4096), (500, 5000, 2050),   # pairs sharing a tile along K
         (1500, 520, 4104), (5000, 264, 1032)]


@pytest.mark.parametrize("shape", KINDS, ids=str)
def test_linear_every_kernel(shape):
    t, k, n = shape
    d = Draw(t + n, F16)
    x, w, b, r = d(t, k), d(k, n, scale=k ** -0.5), d(n)[:n].contiguous(), d(t, n)
    pre, want = linear_want(x, w, b, "gelu", r)
    y, p = tc.linear(x, w, bias=b, act="gelu", residual=r, save_preact=True)
    check(y, want, F16, 1.0, "y")
    check(p, pre, F16, 1.0, "preact")
    again = tc.linear(x, w, bias=b, act="gelu", residual=r)
    assert torch.equal(again, y)


# tokens, k, n: dx and dw apart; together with dx the longer; with dw the longer; dw split along its tokens
GRADS = [(40, 4096, 1024), (300, 8192, 2048), (700, 1024, 2056), (2001, 264, 1031), (4100, 520, 264), (8000, 256, 256),
         (9000, 64, 520)]


@pytest.mark.parametrize("shape", GRADS, ids=str)
def test_linear_backward_every_kernel(shape):
    t, k, n = shape
    d = Draw(t * 3 + n, BF16)
    x, w, dy = d(t, k), d(k, n, scale=k ** -0.5), d(t, n)
    dx, dw, db = tc.linear_backward(dy, x, w, bias=True)
    check(dx, V(dy) @ V(w).T, BF16, 1.0, "dx")
    check(dw, V(x).T @ V(dy), BF16, 1.0, "dw")
    check(db[None], V(torch.ones(1, t, device="cuda", dtype=torch.float64)) @ V(dy), BF16, 1.0, "dbias")


@pytest.mark.parametrize("shape", [(2000, 264, 520, 136), (4100, 520, 264, 136), (900, 512, 2048, 512)], ids=str)
def test_gated_ffn_backward_every_kernel(shape):
    t, k, f, o = shape
    d = Draw(t, F16)
    x, wg, wu, wd = d(t, k), d(k, f, scale=k ** -0.5), d(k, f, scale=k ** -0.5), d(f, o, scale=f ** -0.5)
    dy, g, u, h = d(t, o, scale=0.1), d(t, f, scale=1.5), d(t, f), d(t, f)
    dx, dwg, dwu, dwd = tc.gated_ffn_backward(dy, x, wg, wu, wd, g, u, h)
    dh = V(dy) @ V(wd).T
    dg = (dh * V(u) * V(g).slope("silu")).round(F16)
    du = (dh * V(g).act("silu")).round(F16)
    check(dx, dg @ V(wg).T + du @ V(wu).T, F16, 1.2, "dx")
    check(dwg, V(x).T @ dg, F16, 1.2, "dw_gate")
    check(dwu, V(x).T @ du, F16, 1.2, "dw_up")
    check(dwd, V(h).T @ V(dy), F16, 1.0, "dw_down")


def test_more_than_2_31_entries():
    """Outputs past 4 GiB, forward and as a weight gradient: rows at the start, either side of
    entry 2^31 and at the end."""
    d = Draw(31, BF16)
    x, w = d(66000, 64), d(64, 33000, scale=0.125)
    y = tc.linear(x, w, act="relu")
    rows = [0, 1, 2**31 // 33000 - 1, 2**31 // 33000, 2**31 // 33000 + 1, 65535, 65999]
    _, want = linear_want(x[rows], w, None, "relu", None)
    check(y[rows], want, BF16, 1.0, "y")
    del y
    x, dy = d(72, 50000), d(72, 45000)
    w = torch.empty(50000, 45000, device="cuda", dtype=BF16)  # not read: its gradient's shape
    w.zero_()
    _, dw, _ = tc.linear_backward(dy, x, w)
    rows = [0, 2**31 // 45000 - 1, 2**31 // 45000, 2**31 // 45000 + 1, 49999]
    check(dw[rows], V(x[:, rows]).T @ V(dy), BF16, 1.0, "dw")


@pytest.mark.parametrize("call", ["few", "many", "split", "gated", "backward"])
def test_wait_that_runs_out_is_reported(call):
    """With no loads issued the MMA warp's bounded wait runs out; the context stays usable."""
    d = Draw(2, F16)
    w, wd = d(256, 512), d(512, 256)
    x = {"few": d(3, 256), "many": d(2000, 256), "split": d(512, 256), "gated": d(20, 256), "backward": d(700, 256)}[call]
    if call == "split":
        w = d(4096, 4096)
        x = d(512, 4096)
    try:
        tc.gemm_f16_set_config(inject_stall=1, wait_limit=2_000_000)
        if call == "gated":
            tc.gated_ffn(x, w, w, wd)
        elif call == "backward":
            tc.linear_backward(d(700, 512), x, w)
        else:
            tc.linear(x, w)
        torch.cuda.synchronize()
        rc, site = tc.gemm_f16_device_status(reset=True)
        assert rc == -11 and site == 2
    finally:
        tc.gemm_f16_set_config()
    _, want = linear_want(x, w, None, None, None)
    check(tc.linear(x, w), want, F16, 1.0, "after")


def test_first_calls_from_several_threads():
    """Six host threads, each on a stream of its own, call into different kernels at once."""
    import threading

    d = Draw(77, BF16)
    jobs = []
    for t, k, n in [(1, 512, 1024), (64, 256, 520), (300, 1024, 264), (512, 4096, 4096), (2000, 264, 776), (150, 136, 2048)]:
        x, w = d(t, k), d(k, n, scale=k ** -0.5)
        jobs.append((x, w, V(x) @ V(w)))
    torch.cuda.synchronize()
    got, errors = [None] * len(jobs), []

    def work(i):
        try:
            side = torch.cuda.Stream()
            for _ in range(5):
                got[i] = tc.linear(jobs[i][0], jobs[i][1], stream=side)
            side.synchronize()
        except Exception as e:  # noqa: BLE001  (reported below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for y, (_, _, want) in zip(got, jobs):
        check(y, want, BF16, 1.0, "thread")


def test_refusals():
    d = Draw(4, F16)
    x, w = d(8, 64), d(64, 128)
    for bad in (dict(act="tanh"), dict(bias=d(120)), dict(bias=d(128).float()), dict(residual=d(8, 120)),
                dict(residual=d(8, 128).cpu()), dict(out=torch.empty(8, 128, device="cuda"))):
        with pytest.raises(ValueError):
            tc.linear(x, w, **bad)
    with pytest.raises(ValueError):
        tc.linear(x.float(), w.float())
    with pytest.raises(ValueError):
        tc.linear(x, w.bfloat16())
    with pytest.raises(ValueError):
        tc.linear(x, w.T)
    with pytest.raises(ValueError):
        tc.linear(x.T, d(8, 128))          # rows not contiguous
    with pytest.raises(tc.GemmError) as e:
        tc.linear(d(8, 65)[:, 1:], w)      # base address not a multiple of 16 bytes
    assert e.value.code == -4
    with pytest.raises(tc.GemmError) as e:
        tc.linear(x, d(64, 128, pitch=130))  # row stride not a multiple of 8
    assert e.value.code == -4
    with pytest.raises(tc.GemmError) as e:
        tc.linear(x, w, out=w[:8])         # the output over an operand
    assert e.value.code == -5
    with pytest.raises(ValueError):
        tc.linear_backward(d(8, 128), x, w, act="silu")  # no preact
    with pytest.raises(ValueError):
        tc.gated_ffn(x, w, d(64, 136), d(128, 64))
    with pytest.raises(ValueError):
        tc.gated_ffn(x, w, w, d(120, 64))
    with pytest.raises(tc.GemmError) as e:
        tc.linear(x[:1].expand(8, 64), w)  # a broadcast row: stride 0
    assert e.value.code == -2
