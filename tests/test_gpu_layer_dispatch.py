"""What torch is told of the memory that a layer operator allocates: dispatch modes and profilers see it,
and deterministic algorithms fill it, as they do torch's own operators' outputs."""
import pytest

import tensor_core_tiled_02_gb300 as tc

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16 = torch.bfloat16


def calls():
    """(operator, what it allocates).  128 rows: scales of rows that do not exist are not written."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randn(128, 64, generator=g, device="cuda").to(BF16) for _ in range(2))
    weight = torch.ones(64, dtype=BF16, device="cuda")
    m = tc.mx_quantize(w)
    return [(lambda: tc.linear(x, w.T.contiguous()), 1), (lambda: tc.rms_norm(x, weight, residual=w, save=True), 3),
            (lambda: tc.rms_norm_mx(x, weight), 2), (lambda: tc.mx_quantize(x), 2), (lambda: tc.mx_linear(m, m), 1),
            (lambda: tc.mx_dequantize(m), 1)]


def test_dispatch_modes_see_allocations():
    from torch.utils._python_dispatch import TorchDispatchMode

    class Seen(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            seen.append(str(func))
            return func(*args, **(kwargs or {}))

    for call, count in calls():
        seen, want = [], call()
        with Seen():
            got = call()
        assert sum(s.startswith("aten.empty.") for s in seen) == count
        flat = lambda r: [t for t in (r if isinstance(r, tuple) else (r,)) if isinstance(t, torch.Tensor)]  # noqa: E731
        assert all(torch.equal(a, b) for a, b in zip(flat(got), flat(want)))


def test_profilers_see_allocations():
    for call, count in calls():
        call()
        with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as p:
            call()
        assert sum(e.name == "aten::empty" for e in p.events()) >= count


def test_deterministic_algorithms_fill():
    """Seen in what lies behind the columns of a width that is no multiple of 8."""
    x, w = torch.zeros(3, 8, dtype=BF16, device="cuda")[:, :5], torch.ones(5, dtype=BF16, device="cuda")
    before = torch.are_deterministic_algorithms_enabled()
    try:
        torch.use_deterministic_algorithms(True)
        y = tc.rms_norm(x, w)
    finally:
        torch.use_deterministic_algorithms(before)
    assert not y.any() and y.as_strided((3, 8), (8, 1))[:, 5:].isnan().all()
