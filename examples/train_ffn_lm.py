"""A small language model trained and run on the layer operators.

The model predicts the next word from a window of the last ones:

    x  = the window's embeddings, side by side            [tokens, window * width]
    h  = gelu_tanh(x w_in + b_in)                          tc.linear
    h  = (silu(h w_gate) * (h w_up)) w_down + h            tc.gated_ffn, once per block
    loss = cross entropy of h w_out^T against the next word   tc.linear_cross_entropy

A step runs these, their backward passes in reverse and tc.clip_grad_norm over
all gradients, then plain SGD with momentum on fp32 master weights.  Afterwards
the model continues a text word by word: the same calls on one token.

    python examples/train_ffn_lm.py [--steps 200]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tensor_core_tiled_02_gb300 as tc  # noqa: E402

CONFIG = dict(vocab=5000, window=4, width=128, dim=512, ffn=1376, blocks=3)


def make_text(vocab: int, n: int, seed: int = 0):
    """Words that follow one another by a fixed table nine times in ten."""
    g = torch.Generator().manual_seed(seed)
    table, noise = torch.randperm(vocab, generator=g).tolist(), torch.rand(n, generator=g).tolist()
    free = torch.randint(0, vocab, (n,), generator=g).tolist()
    words = [0]
    for i in range(1, n):
        words.append(table[words[-1]] if noise[i] < 0.9 else free[i])
    return torch.tensor(words, dtype=torch.int64)


class Model:
    def __init__(self, cfg: dict, seed: int = 0, dtype=torch.bfloat16, device="cuda"):
        self.cfg, self.dtype = cfg, dtype
        g = torch.Generator().manual_seed(seed)
        v, w, e, d, f = (cfg[k] for k in ("vocab", "window", "width", "dim", "ffn"))

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=g) * scale).to(device)

        self.master = {"embed": normal(v, e, scale=1.0), "w_in": normal(w * e, d, scale=(w * e) ** -0.5),
                       "b_in": normal(d, scale=0.0), "w_out": normal(v, d, scale=0.5 * d ** -0.5)}
        for i in range(cfg["blocks"]):
            self.master[f"w_gate{i}"] = normal(d, f, scale=d ** -0.5)
            self.master[f"w_up{i}"] = normal(d, f, scale=d ** -0.5)
            self.master[f"w_down{i}"] = normal(f, d, scale=0.5 * f ** -0.5)
        self.weights = {k: t.to(dtype) for k, t in self.master.items()}
        self.momentum = {k: torch.zeros_like(t) for k, t in self.master.items()}

    def inputs(self, windows):
        return self.weights["embed"][windows].reshape(len(windows), -1)

    def block(self, i):
        return tuple(self.weights[f"{n}{i}"] for n in ("w_gate", "w_up", "w_down"))

    def loss_and_gradients(self, windows, target):
        """One pass forward and back: the loss and every weight's gradient."""
        wt, grads = self.weights, {}
        x = self.inputs(windows)
        h, pre = tc.linear(x, wt["w_in"], bias=wt["b_in"], act="gelu_tanh", save_preact=True)
        kept = []
        for i in range(self.cfg["blocks"]):
            y, gate, up, hidden = tc.gated_ffn(h, *self.block(i), residual=h, save=True)
            kept.append((h, gate, up, hidden))
            h = y
        loss, lse = tc.linear_cross_entropy(h, wt["w_out"], target)
        one = torch.ones((), device=h.device)
        dh, grads["w_out"] = tc.linear_cross_entropy_backward(one, h, wt["w_out"], target, lse)
        for i in reversed(range(self.cfg["blocks"])):
            dx, *dw = tc.gated_ffn_backward(dh, kept[i][0], *self.block(i), *kept[i][1:])
            for name, g in zip(("w_gate", "w_up", "w_down"), dw):
                grads[f"{name}{i}"] = g
            dh = dh + dx  # through the residual and through the block
        dx, grads["w_in"], grads["b_in"] = tc.linear_backward(dh, x, wt["w_in"], act="gelu_tanh", preact=pre, bias=True)
        rows = windows.reshape(-1)
        grads["embed"] = torch.zeros_like(self.master["embed"]).index_add_(
            0, rows, dx.reshape(len(rows), -1).float())
        return loss, grads

    def step(self, windows, target, lr: float, max_norm: float = 1.0, momentum: float = 0.9):
        loss, grads = self.loss_and_gradients(windows, target)
        names = sorted(grads)
        norm = tc.clip_grad_norm([grads[k] for k in names], max_norm)  # in place
        for k in names:
            self.momentum[k].mul_(momentum).add_(grads[k].float())
            self.master[k].add_(self.momentum[k], alpha=-lr)
            self.weights[k] = self.master[k].to(self.dtype)
        return loss, norm

    def logits(self, windows):
        wt = self.weights
        h = tc.linear(self.inputs(windows), wt["w_in"], bias=wt["b_in"], act="gelu_tanh")
        for i in range(self.cfg["blocks"]):
            h = tc.gated_ffn(h, *self.block(i), residual=h)
        return tc.linear(h, self.out_in)

    def generate(self, start, words: int):
        """The likeliest continuation, one token at a time."""
        # the vocabulary's weight laid out [in, out] once, padded to a multiple of 8 words
        v, d = self.weights["w_out"].shape
        wide = torch.zeros(d, (v + 7) // 8 * 8, dtype=self.dtype, device="cuda")
        wide[:, :v] = self.weights["w_out"].T
        self.out_in = wide[:, :v]
        text = list(start)
        for _ in range(words):
            window = torch.tensor([text[-self.cfg["window"]:]], device="cuda")
            text.append(int(self.logits(window)[0].argmax()))
        return text


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--tokens", type=int, default=2000, help="tokens a step")
    ap.add_argument("--lr", type=float, default=0.2)
    ap.add_argument("--quiet", action="store_true")
    args = ap.parse_args(argv)
    cfg = CONFIG
    text = make_text(cfg["vocab"], 200_000).cuda()
    model = Model(cfg)
    n = cfg["window"]
    g = torch.Generator(device="cuda").manual_seed(1)
    losses = []
    for step in range(args.steps):
        at = torch.randint(n, len(text), (args.tokens,), generator=g, device="cuda")
        windows = text[at[:, None] + torch.arange(-n, 0, device="cuda")]
        loss, norm = model.step(windows, text[at], args.lr)
        if step % 20 == 0 or step == args.steps - 1:
            losses.append(loss.item())
            if not args.quiet:
                print(f"step {step:4d}  loss {loss.item():.4f}  gradient norm {norm.item():.3f}")
    words = model.generate(text[:n].tolist(), 20)
    if not args.quiet:
        print("continued:", words)
    rc, site = tc.gemm_f16_device_status()
    if rc != 0:
        raise RuntimeError(f"a device wait gave up at site {site}")
    return losses, words


if __name__ == "__main__":
    main()
