"""Cases for the norm between two layers and for products of microscaled operands: a root-mean-square
norm with the residual's addition (its gradients, and its output in 8 or 4 bits with scales), the
quantisation into blocks of 32 that share a power-of-two scale, and the linear layer on operands held
so.  Each in its plain form (elementary torch operations) and, with `own` set, through this package's
entry points.

A microscaled matrix is (data, scale, cols, format).  `data` [rows, bytes]: blocks of 32 values along a
row, e4m3 one byte a value, e2m1 half a byte (the lower half first), the last block filled with zeros.
`scale`: the blocks' exponents plus 127 in one byte each, in tiles of 128 rows by 4 blocks, tile
[row / 128, block / 4], there at [row % 32, row / 32 % 4, block % 4].
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EMAX = {"e2m1": 2, "e4m3": 8}  # exponent of a format's largest value
EPS = 1e-5


def listed():
    return [
        # the norm before a layer for one token of a running answer: nothing but latency
        {"name": "norm one token", "op": "norm", "pass": "forward", "tokens": 1, "k": 4096, "dtype": "bf16", "residual": True},
        # the same over a batch of prompts
        {"name": "norm prompts", "op": "norm", "pass": "forward", "tokens": 8192, "k": 4096, "dtype": "bf16", "residual": True},
        # its gradients for a short ragged batch, a width of no round number
        {"name": "norm gradients ragged", "op": "norm", "pass": "backward", "tokens": 517, "k": 1003, "dtype": "f16", "residual": False},
        # its gradients in a training step, with the gradient that comes along the residual
        {"name": "norm gradients", "op": "norm", "pass": "backward", "tokens": 8192, "k": 4096, "dtype": "bf16", "residual": True},
        # one token into a layer with 8-bit weights: the norm writes what the product reads
        {"name": "norm to layer one token", "op": "layer", "tokens": 1, "k": 4096, "n": 4096, "dtype": "bf16", "format": "e4m3"},
        # a chunk of a prompt the same way
        {"name": "norm to layer prompt", "op": "layer", "tokens": 2000, "k": 4096, "n": 14336, "dtype": "bf16", "format": "e4m3"},
        # activations of a batch of running answers quantised for the next product
        {"name": "quantise batch", "op": "quantise", "rows": 33, "cols": 5632, "dtype": "f16", "format": "e4m3", "transpose": False},
        # a weight [in, out] loaded into 4 bits, along its columns
        {"name": "quantise weight", "op": "quantise", "rows": 4096, "cols": 14336, "dtype": "bf16", "format": "e2m1", "transpose": True},
        # one token through 4-bit weights
        {"name": "product one token", "op": "product", "tokens": 1, "k": 4096, "n": 14336, "dtype": "bf16", "format": "e2m1",
         "act": "none", "bias": False, "residual": False},
        # a batch of running answers through the whole epilogue
        {"name": "product batch", "op": "product", "tokens": 33, "k": 5632, "n": 2048, "dtype": "f16", "format": "e2m1",
         "act": "silu", "bias": True, "residual": True},
        # a prompt through 4-bit weights
        {"name": "product prompt", "op": "product", "tokens": 4096, "k": 4096, "n": 14336, "dtype": "bf16", "format": "e2m1",
         "act": "none", "bias": False, "residual": True},
        # a training step's gradients of such a layer, straight through the rounding: dy quantised along
        # either axis, x along its tokens
        {"name": "product gradients", "op": "gradients", "tokens": 2001, "k": 2048, "n": 8192, "dtype": "bf16", "format": "e4m3"},
    ]


def _between(rng, lo, hi, step=1):
    """A whole multiple of `step` from lo to hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "layer", "quantise", "product", "product", "gradients"])
    while True:
        # widths: three in four whole multiples of 8, as layers have them
        step = rng.choice([1, 8, 8, 8])
        case = {"op": op, "tokens": _between(rng, 1, 8192), "k": _between(rng, 64, 8192, step), "dtype": rng.choice(["f16", "bf16"])}
        if op == "norm":
            case.update({"pass": rng.choice(["forward", "backward"]), "residual": rng.random() < 0.5})
            if case["tokens"] * case["k"] <= 8192 * 4096:
                return case
            continue
        case["format"] = rng.choice(["e2m1", "e4m3"])
        if op == "quantise":
            case.update({"rows": case.pop("tokens"), "cols": 2 * case.pop("k"), "transpose": rng.random() < 0.5})
            if case["rows"] * case["cols"] <= 4096 * 14336:
                return case
            continue
        case["n"] = _between(rng, 64, 16384, step)
        if op == "product":
            case.update({"act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), "bias": rng.random() < 0.5,
                         "residual": rng.random() < 0.5})
        if work(case)["flops"] <= 2 * 4096 * 4096 * 14336:
            return case


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(rows, cols, scale=1.0):
        """Rows on addresses that are multiples of 16 bytes, as this package's calls take them."""
        wide = torch.empty(rows, (cols + 7) // 8 * 8, dtype=dt, device="cuda")
        wide[:, :cols] = (torch.randn(rows, cols, generator=g, device="cuda") * scale).to(dt)
        return wide[:, :cols]

    def spread(rows, cols):
        """Activations: a few columns are far larger than the others."""
        size = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
        size[torch.rand(cols, generator=g, device="cuda") < 0.01] *= 20
        x = normal(rows, cols)
        x *= size.to(dt)
        return x

    s = {"case": case}
    k = case.get("k")
    if case["op"] == "quantise":
        s["x"] = normal(case["rows"], case["cols"], case["rows"] ** -0.5) if case["transpose"] else spread(case["rows"], case["cols"])
    elif case["op"] in ("norm", "layer"):
        s["x"] = spread(case["tokens"], k)
        s["residual"] = normal(case["tokens"], k, 2.0) if case.get("residual", True) else None
        s["weight"] = (1 + 0.2 * torch.randn(k, generator=g, device="cuda")).to(dt)
        if case["op"] == "layer":
            s["w"] = _tiled(*_encode(normal(case["n"], k, k ** -0.5), case["format"]))
        elif case["pass"] == "backward":
            s["dy"], s["dh"] = normal(case["tokens"], k, 0.05), s["residual"]
            s["rstd"] = torch.rsqrt((s["x"].float() ** 2).mean(1) + EPS)
    elif case["op"] == "product":
        s["x"] = _tiled(*_encode(spread(case["tokens"], k), case["format"]))
        s["w"] = _tiled(*_encode(normal(case["n"], k, k ** -0.5), case["format"]))
        s["bias"] = normal(1, case["n"], 0.1)[0].contiguous() if case["bias"] else None
        s["residual"] = normal(case["tokens"], case["n"]) if case["residual"] else None
    else:
        s["x"], s["dy"] = normal(case["tokens"], k), normal(case["tokens"], case["n"], 0.05)
        # the weight as the product with dy reads it: [in, out], blocks along out
        s["w"] = _tiled(*_encode(normal(k, case["n"], k ** -0.5), case["format"]))
    return s


# ---- the plain forms ------------------------------------------------------------------


def _pow2(e):
    """2^e to the bit, e from -127 to 127, in 32 bits."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).int().view(torch.float32)


def _scaled(x, fmt):
    """x [rows, cols] in blocks of 32: (values over the scale, rounded to the format; exponents)."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % 32)).reshape(rows, -1, 32)
    amax = x.abs().amax(2)
    # frexp: amax = m 2^e with m in [0.5, 1), so the exponent of its leading bit is e - 1
    e = torch.clamp(torch.frexp(amax)[1] - 1 - EMAX[fmt], min=-127)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    v = x * _pow2(-e)[:, :, None]
    lead = torch.clamp(torch.frexp(v)[1] - 1, min=0 if fmt == "e2m1" else -6)
    step = _pow2(lead - (1 if fmt == "e2m1" else 3))
    return torch.clamp(torch.round(v / step) * step, -6 if fmt == "e2m1" else -448, 6 if fmt == "e2m1" else 448), e


def _values(x, fmt):
    """The values that x stands for once it is held in the format."""
    q, e = _scaled(x, fmt)
    return (q * _pow2(e)[:, :, None]).reshape(x.shape[0], -1)[:, : x.shape[1]]


def _encode(x, fmt):
    """x's codes one by one, its exponents, its width and the format."""
    q, e = _scaled(x.float(), fmt)
    a = q.abs()
    if fmt == "e2m1":
        code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
        code = code + 8 * (q < 0)
    else:
        lead = torch.clamp(torch.frexp(a)[1] - 1, min=-6)
        m = (a * _pow2(3 - lead)).int()  # 8 .. 15, below 8 for a subnormal one
        code = torch.where(m < 8, m, (lead + 7) * 8 + m - 8) + 128 * (q < 0)
    return code.reshape(x.shape[0], -1).to(torch.uint8), e, x.shape[1], fmt


def _tiled(code, e, cols, fmt):
    """The microscaled matrix as it lies in memory."""
    rows, blocks = e.shape
    data = code[:, 0::2] + 16 * code[:, 1::2] if fmt == "e2m1" else code
    full = torch.zeros(-(-rows // 128) * 128, -(-blocks // 4) * 4, dtype=torch.uint8, device=e.device)
    full[:rows, :blocks] = e + 127
    scale = full.reshape(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    return data.contiguous(), scale, cols, fmt


def _decode(held):
    """The values of a microscaled matrix, in 32 bits."""
    data, scale, cols, fmt = held
    if fmt == "e2m1":
        data = torch.stack((data & 15, data >> 4), 2).reshape(data.shape[0], -1)
        c = (data & 7).float()
        a = torch.where(c < 4, c / 2, torch.where(c < 6, c - 2, 2 * c - 8))
        v = torch.where(data > 7, -a, a)
    else:
        c = (data & 127).int()
        a = torch.where(c < 8, c, c % 8 + 8).float() * _pow2(torch.clamp(c // 8, min=1) - 10)
        v = torch.where(data > 127, -a, a)
    rows, blocks = v.shape[0], v.shape[1] // 32
    full = scale.permute(0, 3, 2, 1, 4).reshape(scale.shape[0] * 128, -1)
    e = full[:rows, :blocks].int() - 127
    return (v.reshape(rows, blocks, 32) * _pow2(e)[:, :, None]).reshape(rows, -1)[:, :cols]


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


def _plain_norm(s, case):
    dt = s["x"].dtype
    w = s["weight"].float()
    if case["op"] == "norm" and case["pass"] == "backward":
        h, dy, r = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
        g = dy * w
        dx = r * g - h * (r * r * r) * (g * h).mean(1, keepdim=True)
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dweight": (dy * h * r).sum(0).to(dt)}
    # h is the residual stream, held in the activations' type; the norm is h's
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dt)
    if case["op"] == "layer":
        # in 64 bits: a value next to a border of the 8-bit grid goes to either side
        wide = h.double()
        y = wide * torch.rsqrt((wide * wide).mean(1, keepdim=True) + EPS) * w.double()
        return {"y": (_values(y, case["format"]).float() @ _decode(s["w"]).T).to(dt), "h": h}
    y = h.float() * torch.rsqrt((h.float() * h.float()).mean(1, keepdim=True) + EPS) * w
    return {"y": y.to(dt), "h": h} if case["residual"] else {"y": y.to(dt)}


def _plain_quantise(s, case):
    x = s["x"].T if case["transpose"] else s["x"]
    return {"values": _values(x.float(), case["format"]).to(x.dtype)}


def _plain_product(s, case):
    y = _decode(s["x"]) @ _decode(s["w"]).T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(case["act"], y)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(DTYPES[case["dtype"]])}


def _plain_gradients(s, case):
    fmt, x, dy = case["format"], s["x"].float(), s["dy"].float()
    dx = _values(dy, fmt) @ _decode(s["w"]).T
    dw = _values(x.T, fmt) @ _values(dy.T, fmt).T
    return {"dx": dx.to(s["x"].dtype), "dw": dw.to(s["x"].dtype)}


def run(s):
    case = s["case"]
    if not own:
        return {"norm": _plain_norm, "layer": _plain_norm, "quantise": _plain_quantise, "product": _plain_product,
                "gradients": _plain_gradients}[case["op"]](s, case)
    import tensor_core_tiled_02_gb300 as tc

    if case["op"] == "norm":
        if case["pass"] == "backward":
            dx, dweight = tc.rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], dh=s["dh"])
            return {"dx": dx, "dweight": dweight}
        if s["residual"] is None:
            return {"y": tc.rms_norm(s["x"], s["weight"], eps=EPS)}
        y, h = tc.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        return {"y": y, "h": h}
    if case["op"] == "layer":
        y, h = tc.rms_norm_mx(s["x"], s["weight"], format=case["format"], residual=s["residual"], eps=EPS)
        return {"y": tc.mx_linear(y, s["w"], dtype=s["x"].dtype), "h": h}
    if case["op"] == "quantise":
        held = tc.mx_quantize(s["x"], format=case["format"], transpose=case["transpose"])
        return {"values": tc.mx_dequantize(held, dtype=s["x"].dtype)}
    if case["op"] == "product":
        return {"y": tc.mx_linear(s["x"], s["w"], bias=s["bias"], act=case["act"], residual=s["residual"],
                                  dtype=DTYPES[case["dtype"]])}
    fmt, dt = case["format"], s["x"].dtype
    dx = tc.mx_linear(tc.mx_quantize(s["dy"], format=fmt), s["w"], dtype=dt)
    dw = tc.mx_linear(tc.mx_quantize(s["x"], format=fmt, transpose=True), tc.mx_quantize(s["dy"], format=fmt, transpose=True),
                      dtype=dt)
    return {"dx": dx, "dw": dw}


# ---- what a pass cannot do without, and what it should return ---------------------------


def _held(case, rows, cols):
    """Bytes of a microscaled matrix."""
    return rows * -(-cols // 32) * (33 if case["format"] == "e4m3" else 17)


def work(case):
    """Each input read once, each output written once, each product computed once."""
    if case["op"] == "quantise":
        n = case["rows"] * case["cols"]
        return {"bytes": 4 * n, "flops": 4 * n}
    t, k = case["tokens"], case["k"]
    if case["op"] == "norm":
        if case["pass"] == "backward":  # reads dy, h, perhaps dh; writes dx
            return {"bytes": 2 * t * k * (3 + case["residual"]) + 4 * k + 4 * t, "flops": 9 * t * k}
        return {"bytes": 2 * t * k * (2 + 2 * case["residual"]) + 2 * k, "flops": 5 * t * k}
    n = case["n"]
    if case["op"] == "layer":  # reads x, residual and the weight; writes h and y
        return {"bytes": 6 * t * k + 2 * k + _held(case, n, k) + 2 * t * n, "flops": 2 * t * k * n + 5 * t * k}
    if case["op"] == "product":
        return {"bytes": _held(case, t, k) + _held(case, n, k) + 2 * t * n * (1 + case["residual"]) + 2 * n * case["bias"],
                "flops": 2 * t * k * n}
    return {"bytes": 2 * (2 * t * k + t * n + k * n) + _held(case, k, n), "flops": 4 * t * k * n}


def _nearest(v, fmt):
    """In 64 bits: the format's value nearest to each of v, of two as near the one whose code is even."""
    table = ([i / 2 for i in range(4)] + [2, 3, 4, 6] if fmt == "e2m1" else
             [i / 512 for i in range(8)] + [(8 + i % 8) * 2.0 ** (i // 8 - 10) for i in range(8, 127)])
    table = torch.tensor(table, dtype=torch.float64, device=v.device)
    up = torch.searchsorted(table, v.abs().contiguous()).clamp(max=len(table) - 1)
    down = (up - 1).clamp(min=0)
    above, below = table[up] - v.abs(), v.abs() - table[down]
    pick = torch.where((above < below) | ((above == below) & (up % 2 == 0)), up, down)
    return torch.copysign(table[pick], v)


def _power(e):
    """2^e in 64 bits, from its exponent field."""
    return ((e + 1023) << 52).view(torch.float64)


def _exact_values(x, fmt):
    """In 64 bits: what x stands for once it is held in the format."""
    x = x.double()
    rows, cols = x.shape
    blocks = torch.cat((x, torch.zeros(rows, -cols % 32, dtype=x.dtype, device=x.device)), 1).view(rows, -1, 32)
    peak = blocks.abs().max(2, keepdim=True).values
    scale = _power(torch.clamp((peak.view(torch.int64) >> 52) - 1023 - EMAX[fmt], min=-127))
    return (_nearest(blocks / scale, fmt) * scale).view(rows, -1)[:, :cols]


def _exact_held(held):
    """In 64 bits: a microscaled matrix's values, looked up code by code."""
    data, scale, cols, fmt = held
    if fmt == "e2m1":
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=data.device)
        v = torch.cat((table, -table))[torch.stack((data % 16, data // 16), 2).long()].view(len(data), -1)
    else:
        v = data.view(torch.float8_e4m3fn).double()
    row = torch.arange(v.shape[0], device=data.device)[:, None]
    block = torch.arange(v.shape[1] // 32, device=data.device)[None, :]
    power = scale[row // 128, block // 4, row % 32, row // 32 % 4, block % 4].long() - 127
    return (v * torch.repeat_interleave(_power(power), 32, 1))[:, :cols]


def exact(case, seed):
    """In 64 bits from the definitions, the norm's gradients by automatic differentiation."""
    s = prepare(case, seed)
    fun = torch.nn.functional
    if case["op"] == "quantise":
        return {"values": _exact_values(s["x"].T if case["transpose"] else s["x"], case["format"])}
    if case["op"] in ("norm", "layer"):
        w = s["weight"].double().requires_grad_()

        def normed(h):
            return h / torch.sqrt(h.pow(2).mean(1, True) + EPS) * w

        if case.get("pass") == "backward":
            h = s["x"].double().requires_grad_()
            dx, dweight = torch.autograd.grad(normed(h), (h, w), s["dy"].double())
            return {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dweight": dweight}
        with torch.no_grad():
            # the stream's own rounding is part of what the norm reads
            h = s["x"].double() if s["residual"] is None else (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
            y = normed(h)
            if case["op"] == "layer":
                y = torch.mm(_exact_values(y, case["format"]), _exact_held(s["w"]).t())
            return {"y": y, "h": h} if s["residual"] is not None else {"y": y}
    if case["op"] == "gradients":
        x, dy, fmt = s["x"], s["dy"], case["format"]
        return {"dx": torch.mm(_exact_values(dy, fmt), _exact_held(s["w"]).t()),
                "dw": torch.mm(_exact_values(x.t(), fmt), _exact_values(dy.t(), fmt).t())}
    act = {"none": lambda v: v, "relu": fun.relu, "silu": fun.silu, "gelu": fun.gelu,
           "gelu_tanh": lambda v: fun.gelu(v, approximate="tanh")}[case["act"]]
    y = torch.mm(_exact_held(s["x"]), _exact_held(s["w"]).t())
    y = act(y if s["bias"] is None else y + s["bias"].double())
    return {"y": y if s["residual"] is None else y + s["residual"].double()}
