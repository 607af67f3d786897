"""Cases for the layer operators next to the GEMM: a linear layer with its epilogue, the gated
feed-forward block, the cross entropy of a vocabulary projection, and the clipping of gradients by
their global norm.  Each in its plain form (elementary 32-bit torch operations, rounded once at the
end) and, with `own` set, through this package's entry points.

Layouts: activations [tokens, features] and weights [in, out], row-major, as `matmul` takes them;
the vocabulary's weight is [vocabulary, features], one row a word, as an embedding table is stored.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
IGNORE = -100  # a target that takes no part in the loss


def listed():
    return [
        # the output projection of a layer for one token of a running answer, added to its input
        {"name": "linear one token", "op": "linear", "pass": "forward", "tokens": 1, "k": 4096, "n": 4096,
         "dtype": "f16", "act": "none", "bias": True, "residual": True},
        # the first projection of a two-matrix feed-forward layer over a prompt
        {"name": "linear prompt", "op": "linear", "pass": "forward", "tokens": 4096, "k": 4096, "n": 14336,
         "dtype": "bf16", "act": "gelu_tanh", "bias": True, "residual": False},
        # the gradients of that layer in a training step over ragged sequences packed end to end
        {"name": "linear gradients", "op": "linear", "pass": "backward", "tokens": 2001, "k": 2048, "n": 8192,
         "dtype": "bf16", "act": "gelu", "bias": True, "residual": False},
        # the feed-forward block for one token of a running answer: every weight is read for it
        {"name": "gated one token", "op": "gated", "pass": "forward", "tokens": 1, "k": 4096, "n": 14336,
         "dtype": "bf16", "act": "silu", "residual": True},
        # the same for a batch of running answers
        {"name": "gated batch", "op": "gated", "pass": "forward", "tokens": 33, "k": 2048, "n": 5632,
         "dtype": "f16", "act": "gelu_tanh", "residual": True},
        # the block's forward pass of a training step, which keeps what its backward pass needs
        {"name": "gated training", "op": "gated", "pass": "training", "tokens": 8192, "k": 4096, "n": 14336,
         "dtype": "bf16", "act": "silu", "residual": True},
        # its backward pass
        {"name": "gated gradients", "op": "gated", "pass": "backward", "tokens": 4096, "k": 4096, "n": 14336,
         "dtype": "bf16", "act": "silu", "residual": False},
        # a fine-tuning step on one short line of text
        {"name": "loss short", "op": "loss", "pass": "training", "tokens": 8, "k": 1024, "n": 32768, "dtype": "f16"},
        # scoring a text: the loss of each of its tokens, under a vocabulary of odd size
        {"name": "loss scoring", "op": "loss", "pass": "forward", "tokens": 1000, "k": 2048, "n": 50021,
         "dtype": "f16"},
        # the head of a training step
        {"name": "loss training", "op": "loss", "pass": "training", "tokens": 4096, "k": 4096, "n": 65536,
         "dtype": "bf16"},
        # clipping an adapter's few small gradients
        {"name": "clip adapter", "op": "clip", "pass": "clip", "tensors": 24, "elements": 400_000, "dtype": "f32",
         "size": 3.0},
        # clipping the gradients of a stack of layers: many vectors and matrices, vectors in 32 bits
        {"name": "clip layers", "op": "clip", "pass": "clip", "tensors": 290, "elements": 700_000_000,
         "dtype": "bf16", "size": 20.0},
    ]


def _between(rng, lo, hi, step=1):
    """A whole multiple of `step` from lo to hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["linear", "linear", "gated", "gated", "loss", "loss", "clip"])
    dtype = rng.choice(["f16", "bf16"])
    while True:
        if op == "clip":
            return {"op": op, "pass": "clip", "tensors": _between(rng, 1, 400),
                    "elements": _between(rng, 1000, 600_000_000), "dtype": rng.choice(["f16", "bf16", "f32"]),
                    "size": rng.choice([0.5, 3.0, 20.0])}
        case = {"op": op, "pass": "", "tokens": _between(rng, 1, 8192), "k": _between(rng, 256, 8192, 8),
                "n": _between(rng, 512, 16384, 8), "dtype": dtype}
        if op == "linear":
            case.update({"pass": rng.choice(["forward", "backward"]), "bias": rng.random() < 0.5,
                         "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])})
            case["residual"] = case["pass"] == "forward" and rng.random() < 0.5
        elif op == "gated":
            case.update({"pass": rng.choice(["forward", "training", "backward"]),
                         "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu"])})
            case["residual"] = case["pass"] != "backward" and rng.random() < 0.5
        else:
            case.update({"pass": rng.choice(["forward", "training"]), "n": _between(rng, 2000, 131072)})
        if work(case)["flops"] <= 2.8e12:
            return case


def _sizes(case):
    """Elements of each gradient: of three tensors two are vectors, the third a matrix that takes
    most of what is left; odd sizes among them."""
    count, left, sizes = case["tensors"], case["elements"], []
    for i in range(count):
        share = left / (count - i)
        n = share if (i % 3 == 2 or count < 3) else min(share, 4096 + 7 * (i % 5))
        n = max(1, int(n) if i < count - 1 else left)
        sizes.append(n)
        left = max(1, left - n)
    return sizes


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)

    s = {"case": case}
    if case["op"] == "clip":
        # gradients lie end to end in one buffer for each type, the vectors' in 32 bits, and the
        # clipped ones go to buffers laid out the same (the optimiser's)
        sizes = _sizes(case)
        wide = [case["dtype"] == "f32" or (len(sizes) >= 3 and i % 3 != 2) for i in range(len(sizes))]
        s["flat"], s["out"], s["grads"], s["outs"] = [], [], [None] * len(sizes), [None] * len(sizes)
        for kind, t in ((True, torch.float32), (False, dt)):
            which = [i for i in range(len(sizes)) if wide[i] == kind]
            if not which:
                continue
            n = sum(sizes[i] for i in which)
            # entries such that the global norm comes to about `size`
            flat = normal(n, scale=case["size"] / math.sqrt(case["elements"]), dtype=t)
            out = torch.empty_like(flat)
            s["flat"].append(flat)
            s["out"].append(out)
            at = 0
            for i in which:
                s["grads"][i], s["outs"][i] = flat[at:at + sizes[i]], out[at:at + sizes[i]]
                at += sizes[i]
        s["max_norm"] = 1.0
        return s
    t, k, n = case["tokens"], case["k"], case["n"]
    if case["op"] == "linear":
        s["x"], s["w"] = normal(t, k), normal(k, n, scale=k ** -0.5)
        s["bias"] = normal(n, scale=0.1) if case["bias"] else None
        s["residual"] = normal(t, n) if case["residual"] else None
        if case["pass"] == "backward":
            s["dy"], s["pre"] = normal(t, n, scale=0.05), normal(t, n)
    elif case["op"] == "gated":
        s["x"] = normal(t, k)
        s["w_gate"], s["w_up"] = normal(k, n, scale=k ** -0.5), normal(k, n, scale=k ** -0.5)
        s["w_down"] = normal(n, k, scale=n ** -0.5)
        s["residual"] = normal(t, k) if case["residual"] else None
        if case["pass"] == "backward":
            s["dy"], s["gate"], s["up"] = normal(t, k, scale=0.05), normal(t, n), normal(t, n)
            s["hidden"] = (_act(case["act"], s["gate"].float()) * s["up"].float()).to(dt)
    else:
        s["w"] = normal(n, k, scale=0.02)
        s["target"] = torch.randint(0, n, (t,), generator=g, device="cuda")
        # a model in training: its states lean towards the next word's row
        lean = s["w"][s["target"]].float()
        s["h"] = (torch.randn(t, k, generator=g, device="cuda") + 3.0 * lean / lean.norm(dim=1, keepdim=True)).to(dt)
        # of a packed text some tokens are not predicted
        skip = torch.rand(t, generator=g, device="cuda") < 0.1
        skip[0] = False
        s["target"][skip] = IGNORE
        # the loss's gradient: a loss scale keeps 16-bit gradients in range
        s["grad"] = torch.tensor(4096.0 if case["dtype"] == "f16" else 1.0, device="cuda")
    return s


# ---- the plain forms ------------------------------------------------------------------


def _act(name, x):
    if name == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if name == "silu":
        return x / (1 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _slope(name, x):
    if name == "relu":
        return (x > 0).to(x.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x * x * x))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)
    return torch.ones_like(x)


def _plain_linear(s, case):
    dt = s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    if case["pass"] == "backward":
        dpre = s["dy"].float() * _slope(case["act"], s["pre"].float())
        out = {"dx": (dpre @ w.T).to(dt), "dw": (x.T @ dpre).to(dt)}
        if case["bias"]:
            out["dbias"] = dpre.sum(0).to(dt)
        return out
    y = x @ w
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(case["act"], y)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(dt)


def _plain_gated(s, case):
    dt = s["x"].dtype
    x, wg, wu, wd = (s[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
    if case["pass"] == "backward":
        dy, gate, up, hidden = (s[k].float() for k in ("dy", "gate", "up", "hidden"))
        dhidden = dy @ wd.T
        dgate = dhidden * up * _slope(case["act"], gate)
        dup = dhidden * _act(case["act"], gate)
        return {"dx": (dgate @ wg.T + dup @ wu.T).to(dt), "dw_gate": (x.T @ dgate).to(dt),
                "dw_up": (x.T @ dup).to(dt), "dw_down": (hidden.T @ dy).to(dt)}
    gate, up = x @ wg, x @ wu
    hidden = _act(case["act"], gate) * up
    y = hidden @ wd
    if s["residual"] is not None:
        y = y + s["residual"].float()
    if case["pass"] == "training":
        return {"y": y.to(dt), "gate": gate.to(dt), "up": up.to(dt), "hidden": hidden.to(dt)}
    return y.to(dt)


def _plain_loss(s, case):
    dt = s["h"].dtype
    h, w, target = s["h"].float(), s["w"].float(), s["target"]
    logits = h @ w.T
    most = logits.amax(1)
    lse = most + torch.log(torch.exp(logits - most[:, None]).sum(1))
    counts = target != IGNORE
    word = torch.where(counts, target, torch.zeros_like(target))
    loss = torch.where(counts, lse - logits.gather(1, word[:, None])[:, 0], torch.zeros_like(lse))
    if case["pass"] == "forward":
        return {"loss": loss, "lse": lse}
    scale = torch.where(counts, s["grad"] / counts.sum(), torch.zeros_like(lse))
    d = torch.exp(logits - lse[:, None])
    rows = torch.arange(len(word), device=word.device)
    d[rows, word] -= 1
    d = d * scale[:, None]
    return {"loss": loss.sum() / counts.sum(), "lse": lse, "dh": (d @ w).to(dt), "dw": (d.T @ h).to(dt)}


def _plain_clip(s, case):
    norm = torch.sqrt(torch.stack([torch.sum(t.float() * t.float()) for t in s["flat"]]).sum())
    scale = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm, "grads": [(t.float() * scale).to(t.dtype) for t in s["flat"]]}


def run(s):
    case = s["case"]
    if not own:
        return {"linear": _plain_linear, "gated": _plain_gated, "loss": _plain_loss, "clip": _plain_clip}[case["op"]](s, case)
    import tensor_core_tiled_02_gb300 as tc

    if case["op"] == "linear":
        if case["pass"] == "backward":
            dx, dw, dbias = tc.linear_backward(s["dy"], s["x"], s["w"], act=case["act"], preact=s["pre"],
                                               bias=case["bias"])
            return {"dx": dx, "dw": dw, "dbias": dbias} if case["bias"] else {"dx": dx, "dw": dw}
        return tc.linear(s["x"], s["w"], bias=s["bias"], act=case["act"], residual=s["residual"])
    if case["op"] == "gated":
        if case["pass"] == "backward":
            dx, dw_gate, dw_up, dw_down = tc.gated_ffn_backward(
                s["dy"], s["x"], s["w_gate"], s["w_up"], s["w_down"], s["gate"], s["up"], s["hidden"], act=case["act"])
            return {"dx": dx, "dw_gate": dw_gate, "dw_up": dw_up, "dw_down": dw_down}
        if case["pass"] == "training":
            y, gate, up, hidden = tc.gated_ffn(s["x"], s["w_gate"], s["w_up"], s["w_down"], act=case["act"],
                                               residual=s["residual"], save=True)
            return {"y": y, "gate": gate, "up": up, "hidden": hidden}
        return tc.gated_ffn(s["x"], s["w_gate"], s["w_up"], s["w_down"], act=case["act"], residual=s["residual"])
    if case["op"] == "loss":
        if case["pass"] == "forward":
            loss, lse = tc.linear_cross_entropy(s["h"], s["w"], s["target"], ignore_index=IGNORE, reduction="none")
            return {"loss": loss, "lse": lse}
        loss, lse = tc.linear_cross_entropy(s["h"], s["w"], s["target"], ignore_index=IGNORE, reduction="mean")
        dh, dw = tc.linear_cross_entropy_backward(s["grad"], s["h"], s["w"], s["target"], lse, ignore_index=IGNORE,
                                                  reduction="mean")
        return {"loss": loss, "lse": lse, "dh": dh, "dw": dw}
    norm = tc.clip_grad_norm(s["grads"], s["max_norm"], out=s["outs"])
    return {"norm": norm, "grads": s["out"]}


# ---- what a pass cannot do without, and what it should return ---------------------------


def work(case):
    """Each input read once, each output written once, each product computed once."""
    b = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "clip":
        sizes = _sizes(case)
        wide = [case["dtype"] == "f32" or (len(sizes) >= 3 and i % 3 != 2) for i in range(len(sizes))]
        return {"bytes": 2 * sum(n * (4 if x else b) for n, x in zip(sizes, wide)) + 4, "flops": 3 * sum(sizes)}
    t, k, n = case["tokens"], case["k"], case["n"]
    if case["op"] == "linear":
        if case["pass"] == "backward":  # reads dy, pre, x, w; writes dx, dw
            pre = t * n if case["act"] != "none" else 0
            return {"bytes": b * (t * n + pre + 2 * t * k + 2 * k * n + n * case["bias"]), "flops": 4 * t * k * n}
        return {"bytes": b * (t * k + k * n + t * n * (1 + case["residual"]) + n * case["bias"]), "flops": 2 * t * k * n}
    if case["op"] == "gated":
        if case["pass"] == "backward":  # reads dy, x, gate, up, hidden and the weights; writes the gradients
            return {"bytes": b * (3 * t * k + 3 * t * n + 6 * k * n), "flops": 12 * t * k * n}
        kept = 3 * t * n if case["pass"] == "training" else 0
        return {"bytes": b * (t * k * (2 + case["residual"]) + 3 * k * n + kept), "flops": 6 * t * k * n}
    if case["pass"] == "forward":
        return {"bytes": b * (t * k + n * k) + 16 * t, "flops": 2 * t * k * n}
    return {"bytes": 2 * b * (t * k + n * k) + 16 * t, "flops": 6 * t * k * n}


def exact(case, seed):
    """In 64 bits from the definitions, gradients by automatic differentiation."""
    if case["op"] != "clip" and work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)

    def wide(t, grad=False):
        return t.double().requires_grad_(grad)

    fun = torch.nn.functional
    act = {"none": lambda v: v, "relu": fun.relu, "silu": fun.silu, "gelu": fun.gelu,
           "gelu_tanh": lambda v: fun.gelu(v, approximate="tanh")}[case.get("act", "none")]
    if case["op"] == "clip":
        flat = [wide(t) for t in s["flat"]]
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(t)) ** 2 for t in flat))
        scale = min(1.0, s["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": [t * scale for t in flat]}
    if case["op"] == "linear":
        if case["pass"] == "backward":
            pre = wide(s["pre"], True)
            (dpre,) = torch.autograd.grad(act(pre), pre, wide(s["dy"]))
            x, w, bias = wide(s["x"], True), wide(s["w"], True), torch.zeros(case["n"], dtype=torch.float64, device="cuda", requires_grad=True)
            dx, dw, dbias = torch.autograd.grad(torch.addmm(bias, x, w), (x, w, bias), dpre)
            return {"dx": dx, "dw": dw, "dbias": dbias} if case["bias"] else {"dx": dx, "dw": dw}
        y = torch.mm(wide(s["x"]), wide(s["w"]))
        y = act(y if s["bias"] is None else y + wide(s["bias"]))
        return y if s["residual"] is None else y + wide(s["residual"])
    if case["op"] == "gated":
        x, wg, wu, wd = (wide(s[k], True) for k in ("x", "w_gate", "w_up", "w_down"))
        if case["pass"] == "backward":
            # what the forward pass kept stands for what it computed
            gate, up, hidden, dy = wide(s["gate"], True), wide(s["up"], True), wide(s["hidden"]), wide(s["dy"])
            (dhidden, dwd) = torch.autograd.grad(torch.mm(hidden.requires_grad_(), wd), (hidden, wd), dy)
            dgate, dup = torch.autograd.grad(act(gate) * up, (gate, up), dhidden)
            dx, dwg, dwu = torch.autograd.grad((torch.mm(x, wg), torch.mm(x, wu)), (x, wg, wu), (dgate, dup))
            return {"dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}
        with torch.no_grad():
            gate, up = torch.mm(x, wg), torch.mm(x, wu)
            hidden = act(gate) * up
            y = torch.mm(hidden, wd)
            y = y if s["residual"] is None else y + wide(s["residual"])
        return {"y": y, "gate": gate, "up": up, "hidden": hidden} if case["pass"] == "training" else y
    h, w = wide(s["h"], True), wide(s["w"], True)
    logits = torch.mm(h, w.t())
    lse = torch.logsumexp(logits, 1)
    if case["pass"] == "forward":
        loss = fun.cross_entropy(logits, s["target"], ignore_index=IGNORE, reduction="none")
        return {"loss": loss.detach(), "lse": lse.detach()}
    loss = fun.cross_entropy(logits, s["target"], ignore_index=IGNORE)
    dh, dw = torch.autograd.grad(loss, (h, w), s["grad"].double())
    return {"loss": loss.detach(), "lse": lse.detach(), "dh": dh, "dw": dw}
