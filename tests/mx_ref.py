"""Microscaled matrices in 64 bits: what a block becomes, and what held bytes stand for.

Scales are powers of two, so quantising is exact arithmetic: the kernels' bytes are
held to these bit for bit.
"""
import torch

EMAX = {"e2m1": 2, "e4m3": 8}
# a format's values without their sign, in the order of their codes
TABLE = {"e2m1": [0, 0.5, 1, 1.5, 2, 3, 4, 6],
         "e4m3": [i / 512 for i in range(8)] + [(8 + i % 8) * 2.0 ** (i // 8 - 10) for i in range(8, 127)]}


def pow2(e):
    """2^e, e from -1022 to 1023."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def nearest(v, fmt):
    """Codes (without sign) of the values nearest to |v|, ties to the even code, saturated."""
    table = torch.tensor(TABLE[fmt], dtype=torch.float64, device=v.device)
    a = v.abs().contiguous()
    up = torch.searchsorted(table, a).clamp(max=len(table) - 1)
    down = (up - 1).clamp(min=0)
    over, under = table[up] - a, a - table[down]
    return torch.where((over < under) | ((over == under) & (up % 2 == 0)), up, down)


def exponents(x, fmt):
    """x [rows, blocks, 32] fp64: the scale byte of each block."""
    amax = x.abs().amax(2)
    e = (amax.view(torch.int64) >> 52) - 1023 - EMAX[fmt]
    byte = torch.clamp(e + 127, min=0)
    return torch.where(torch.isfinite(x).all(2), byte, torch.full_like(byte, 255))


def blocks(x):
    rows, cols = x.shape
    wide = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=x.device)
    wide[:, :cols] = x.double()
    return wide.view(rows, -1, 32)


def quantize(x, fmt):
    """(values [rows, cols] fp64, NaN in blocks of byte 255; scale bytes [rows, blocks])."""
    b = blocks(x)
    byte = exponents(b, fmt)
    s = pow2(torch.where(byte == 255, 127, byte) - 127)[:, :, None]
    table = torch.tensor(TABLE[fmt], dtype=torch.float64, device=x.device)
    v = torch.copysign(table[nearest(torch.nan_to_num(b / s), fmt)], b) * s
    v = torch.where((byte == 255)[:, :, None], torch.full_like(v, float("nan")), v)
    return v.view(x.shape[0], -1)[:, : x.shape[1]], byte


def scale_bytes(m, rows):
    """The scale bytes of an Mx, [rows, blocks], and those behind its last block in the same tiles."""
    tiles = m[1]
    full = tiles.permute(0, 3, 2, 1, 4).reshape(tiles.shape[0] * 128, tiles.shape[1] * 4)[:rows].long()
    n = -(-m[2] // 32)
    return full[:, :n], full[:, n:]


def values(m):
    """What an Mx stands for, fp64."""
    data, _, cols, fmt = m
    table = torch.tensor(TABLE[fmt], dtype=torch.float64, device=data.device)
    if fmt == "e2m1":
        code = torch.stack((data & 15, data >> 4), 2).view(data.shape[0], -1).long()
        v = torch.where(code < 8, 1.0, -1.0) * table[code & 7]
    else:
        code = data.long()
        table = torch.cat((table, torch.full((1,), float("nan"), dtype=torch.float64, device=data.device)))
        v = torch.where(code < 128, 1.0, -1.0) * table[code & 127]
    byte, _ = scale_bytes(m, data.shape[0])
    s = torch.where(byte == 255, torch.full((), float("nan"), dtype=torch.float64, device=data.device), pow2(byte - 127))
    v = (v.view(data.shape[0], -1, 32) * s[:, :, None]).view(data.shape[0], -1)
    return v[:, :cols]


def hold(x, fmt):
    """(data, scale, cols, fmt) of x, made here and not by a kernel."""
    rows, cols = x.shape
    b = blocks(x)
    byte = exponents(b, fmt)
    s = pow2(torch.where(byte == 255, 127, byte) - 127)[:, :, None]
    code = nearest(torch.nan_to_num(b / s), fmt) + (8 if fmt == "e2m1" else 128) * (b < 0)
    code = code.view(rows, -1).to(torch.uint8)
    data = (code[:, 0::2] + 16 * code[:, 1::2]).contiguous() if fmt == "e2m1" else code.contiguous()
    n = byte.shape[1]
    full = torch.zeros(-(-rows // 128) * 128, -(-n // 4) * 4, dtype=torch.uint8, device=x.device)
    full[:rows, :n] = byte.to(torch.uint8)
    full[rows:] = 255  # rows that do not exist hold anything
    scale = full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    return data, scale, cols, fmt
