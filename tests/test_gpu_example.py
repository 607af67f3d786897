"""The example that runs the layer operators together: its gradients against automatic
differentiation of the same model in 64 bits, and that it learns."""
import os
import sys

import pytest

import layer_ref

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_gradients_of_the_whole_model():
    import train_ffn_lm as ex

    cfg = dict(vocab=777, window=3, width=40, dim=136, ffn=264, blocks=2)
    model = ex.Model(cfg, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    windows = torch.randint(0, cfg["vocab"], (150, cfg["window"]), generator=g, device="cuda")
    target = torch.randint(0, cfg["vocab"], (150,), generator=g, device="cuda")
    target[::7] = -100
    loss, grads = model.loss_and_gradients(windows, target)

    w = {k: t.double().requires_grad_(True) for k, t in model.weights.items()}
    h = layer_ref.act64("gelu_tanh", w["embed"][windows].reshape(150, -1) @ w["w_in"] + w["b_in"])
    for i in range(cfg["blocks"]):
        h = (layer_ref.act64("silu", h @ w[f"w_gate{i}"]) * (h @ w[f"w_up{i}"])) @ w[f"w_down{i}"] + h
    want = torch.nn.functional.cross_entropy(h @ w["w_out"].T, target, ignore_index=-100)
    names = sorted(w)
    exact = dict(zip(names, torch.autograd.grad(want, [w[k] for k in names])))
    # activations and their gradients are rounded to bf16 at some ten places on the way (u / sqrt 3
    # each), so a gradient is off by some sqrt(10 / 3) u of its norm; four times that is allowed
    room = 4 * (10 / 3) ** 0.5 * layer_ref.U[torch.bfloat16]
    assert abs(loss.item() - want.item()) <= room * want.item()
    for k in names:
        off = (grads[k].double() - exact[k]).norm().item()
        assert off <= room * exact[k].norm().item(), (k, off / exact[k].norm().item())


def test_it_learns():
    import train_ffn_lm as ex

    losses, words = ex.main(["--steps", "60", "--quiet"])
    assert losses[0] > 8.0          # near ln(5000) = 8.5 at the start
    assert losses[-1] < losses[0] - 1.0
    assert len(words) == 24 and all(0 <= w < 5000 for w in words)
