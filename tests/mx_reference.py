"""MXFP4 in 64 bits: conversion, the values of codes, and the expert network
with the converted intermediate, with a bound on what float32 sums may change
(a sum next to a border between two codes, or next to a power of two that sets
a block's scale, may round either way)."""
import torch

U = 2.0 ** -24
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e2m1(mag):
    """Index of the nearest E2M1 magnitude (ties to the even index, at most 7)."""
    code = torch.zeros(mag.shape, dtype=torch.int64, device=mag.device)
    for i in range(1, 8):
        border = (GRID[i - 1] + GRID[i]) / 2
        code = torch.where((mag >= border) if i % 2 == 0 else (mag > border), i, code)
    return code


def exponent(top):
    """X of blocks whose largest magnitudes are `top` > 0 (others: 0)."""
    _, e = torch.frexp(top.double())
    return torch.where(top > 0, (e.double() - 1 - 2).clamp(-127, 125), 0.0)


def quantize(v):
    """(codes [rows, cols], scale bytes [rows, cols / 32]) of v [rows, cols] (any float type), a byte a code."""
    b = v.double().view(v.shape[0], -1, 32)
    bad = ~torch.isfinite(b).all(dim=2)
    b = torch.where(bad[..., None], 0.0, b)
    x = exponent(b.abs().amax(dim=2))
    code = e2m1(b.abs() * torch.exp2(-x)[..., None]) | (torch.signbit(b).long() << 3)
    code = torch.where(bad[..., None], 0, code)
    return code.view(v.shape).to(torch.uint8), torch.where(bad, 255, x.long() + 127).to(torch.uint8)


def pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def values(packed, scales):
    """Codes [..., rows, cols / 2] and scales [..., rows, cols / 32] -> float64 (255: NaN)."""
    c = torch.stack([packed & 15, packed >> 4], dim=-1).flatten(-2).long()
    grid = torch.tensor(GRID, dtype=torch.float64, device=packed.device)
    v = torch.where(c >= 8, -grid[c & 7], grid[c & 7])
    s = torch.where(scales == 255, float("nan"), torch.exp2(scales.double() - 127))
    return v * s.repeat_interleave(32, dim=-1)


def rounded(h, x):
    """h [rows, blocks, 32] at the exponents x [rows, blocks]."""
    grid = torch.tensor(GRID, dtype=torch.float64, device=h.device)
    s = torch.exp2(x)[..., None]
    return torch.copysign(grid[e2m1(h.abs() / s)], h) * s


def converted(h, err):
    """(Q(h), bound on its change for an h that is off by at most err), [rows, cols]."""
    b, e = h.view(h.shape[0], -1, 32), err.view(h.shape[0], -1, 32)
    top = b.abs().amax(dim=2)
    spread = e.amax(dim=2)
    q = rounded(b, exponent(top))
    off = torch.zeros_like(q)
    for x in (exponent((top - spread).clamp(min=0)), exponent(top + spread)):
        for v in (b - e, b + e):
            off = torch.maximum(off, (rounded(v, x) - q).abs())
    return q.view(h.shape), off.view(h.shape)


def expert(rows, wg, wu, wd):
    """(y, bound) of one expert in 64 bits: rows [n, d], matrices as stored ("out x in")."""
    d, F = rows.shape[1], wg.shape[0]
    a, b = rows @ wg.t(), rows @ wu.t()
    # a float32 sum of K exact products, at least eight of which are added at a time
    ca = (d / 8 + 8) * U
    ea, eb = ca * (rows.abs() @ wg.abs().t()), ca * (rows.abs() @ wu.abs().t())
    silu = a * torch.sigmoid(a)
    # |silu'| < 1.1; the hardware's exponential and reciprocal: a step each, the exponent's product |a| steps
    es = 1.1 * ea + silu.abs() * (a.abs() + 8) * 2 * U
    h = silu * b
    eh = es * b.abs() + silu.abs() * eb + es * eb + h.abs() * 2 * U
    q, eq = converted(h, eh)
    y = q @ wd.t()
    return y, eq @ wd.abs().t() + (F / 8 + 8) * U * ((q.abs() + eq) @ wd.abs().t())
