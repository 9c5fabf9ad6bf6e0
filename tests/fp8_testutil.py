"""64-bit references of the 8-bit projection path, in numpy: quantising with
power-of-two block scales, the values a scaled matrix stands for, and its
scales as a plain [R, C] array."""
from __future__ import annotations

import numpy as np


def blocks(n):
    return -(-n // 128)


def e4m3_round(v):
    """fp64 -> nearest e4m3 value, ties to even (|v| <= 448; steps of 2^-9 near zero)."""
    _, ex = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(ex - 4, -9))
    return np.rint(v / step) * step


def scale_exponent(amax):
    """Smallest e >= -127 with amax <= 448 * 2^e, 0 for amax = 0, by trial."""
    amax = np.asarray(amax, dtype=np.float64)
    e = np.full(amax.shape, -127)
    for _ in range(256):
        e = np.where(amax > np.ldexp(448.0, e), e + 1, e)
    return np.where(amax == 0, 0, e)


_SHAPES = {"row": (1, 128), "col": (128, 1), "tile": (128, 128)}


def expand(e, kind, R, C):
    """Block exponents -> one per element [R, C]."""
    br, bc = _SHAPES[kind]
    return np.repeat(np.repeat(e, br, 0), bc, 1)[:R, :C]


def block_amax(x, kind):
    R, C = x.shape
    br, bc = _SHAPES[kind]
    nr, nc = -(-R // br), -(-C // bc)
    full = np.zeros((nr * br, nc * bc))
    full[:R, :C] = np.where(np.isfinite(x), np.abs(x), 0)
    return full.reshape(nr, br, nc, bc).max((1, 3))


def quantize(x, kind):
    """fp64 [R, C] -> (e4m3 values [R, C], exponents of the blocks)."""
    e = scale_exponent(block_amax(x, kind))
    s = np.ldexp(1.0, expand(e, kind, *x.shape))
    return np.where(np.isfinite(x), e4m3_round(np.where(np.isfinite(x), x, 0) / s), np.nan), e


def stored_scales(e, kind):
    """Exponents of the blocks -> the stored bytes."""
    b = (e + 127).astype(np.uint8)
    if kind == "tile":
        return b
    b = b if kind == "row" else b.T
    w = np.full((b.shape[0], -(-b.shape[1] // 4) * 4), 127, dtype=np.uint8)
    w[:, :b.shape[1]] = b
    return np.ascontiguousarray(w.reshape(b.shape[0], -1, 4).transpose(1, 0, 2))


def values(m):
    """An Fp8Matrix -> the fp64 values it stands for."""
    import torch
    data = m.data.detach().cpu().float().numpy().astype(np.float64)
    R, C = data.shape
    e = m.scales.detach().view(torch.uint8).cpu().numpy().astype(np.int64) - 127
    if m.kind != "tile":
        e = e.transpose(1, 0, 2).reshape(e.shape[1], -1)
        e = e[:, :blocks(C)] if m.kind == "row" else e[:, :blocks(R)].T
    return data * np.ldexp(1.0, expand(e, m.kind, R, C))
