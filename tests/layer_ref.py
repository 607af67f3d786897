"""The layer operators in 64 bits, with a bound on what each rounding of the
kernels may change.

Every value carries (v, e): v from the definition in fp64, e >= 0 the most a
result may differ from it.  A product of K terms accumulated on the tensor
core in fp32 adds each group of 16 products with truncating alignment: at
most 2^-22 of the running sum of magnitudes per group, so (K/16 + 8) 2^-22
sum |a||b|.  Rounding to 16 bits adds u |v| (u = 2^-11 fp16, 2^-8 bf16) and
half the least subnormal.  The activations' slopes stay below 1.13, their own
slopes below 1.6 (silu 0.5, gelu 0.8, gelu_tanh 0.8, each with a margin of two);
fp32 evaluation is allowed 2^-18 of |x| + |value|.

Beside the element-wise bound, the 2-norm of the error over that of the values is
held to `rms` times u: a rounding's error is spread evenly over half an ulp, so it
has a root mean square of at most u / sqrt(3), and n independent ones sqrt(n / 3) u.
"""
import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def act64(name, x):
    if name in (None, "none"):
        return x
    if name == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if name == "silu":
        return x * torch.sigmoid(x)
    if name == "gelu":
        return 0.5 * x * torch.special.erfc(-x * math.sqrt(0.5))
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))


def slope64(name, x):
    x = x.detach().clone().requires_grad_(True)
    (g,) = torch.autograd.grad(act64(name, x).sum(), x)
    return g.detach()


class V:
    """A value and the most a kernel's result may be off."""

    def __init__(self, v, e=None):
        self.v = v.double()
        self.e = torch.zeros_like(self.v) if e is None else e

    def __matmul__(self, o):
        k = self.v.shape[1]
        a, b = self.v.abs() + self.e, o.v.abs() + o.e
        e = a @ b - self.v.abs() @ o.v.abs() + (k / 16 + 8) * 2.0 ** -22 * (a @ b)
        return V(self.v @ o.v, e)

    def __add__(self, o):
        v = self.v + o.v
        return V(v, self.e + o.e + 2.0 ** -23 * (v.abs() + self.e + o.e))

    def __mul__(self, o):
        v = self.v * o.v
        e = self.e * o.v.abs() + o.e * self.v.abs() + self.e * o.e
        return V(v, e + 2.0 ** -22 * (v.abs() + e))

    @property
    def T(self):
        return V(self.v.T, self.e.T)

    def act(self, name):
        if name in (None, "none"):
            return self
        v = act64(name, self.v)
        return V(v, 1.13 * self.e + 2.0 ** -18 * (v.abs() + self.v.abs().clamp(max=16) * (v != 0)) + 2.0 ** -126)

    def slope(self, name):
        if name in (None, "none"):
            return V(torch.ones_like(self.v))
        v = slope64(name, self.v)
        e = 1.6 * self.e + (0 if name == "relu" else 2.0 ** -18) * (1 + v.abs())
        return V(v, e)

    def round(self, dt):
        return V(self.v, self.e + U[dt] * (self.v.abs() + self.e) + TINY[dt])


def check(got, want, dt, rms, what):
    """`got` (16 bits, rounded from `want` once more) against want's bound."""
    assert got.dtype == dt and tuple(got.shape) == tuple(want.v.shape), what
    w = want.round(dt)
    g = got.double()
    off = (g - w.v).abs()
    bad = ~(off <= w.e)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {(off / w.e).max().item():.3g} of the bound"
    norm = w.v.norm()
    if w.v.numel() >= 256 and norm > 0 and dt in U and norm / math.sqrt(w.v.numel()) > 1e5 * TINY[dt]:
        rel = ((g - w.v).norm() / norm).item()
        assert rel <= rms * U[dt], f"{what}: 2-norm off by {rel:.3g}, {rel / U[dt]:.2f} u"
