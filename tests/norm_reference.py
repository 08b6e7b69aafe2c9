"""The norms around the layer in 64 bits (values by the formula, gradients by
automatic differentiation of it), with bounds on what float32 sums and the
stored type may add to them.

``U`` is float32's half step; a sum of a row of d values is a chain of at most
``chain(d)`` additions (8 columns a chunk and up to 8 chunks in a thread, six
steps of a wave, sixteen waves)."""
import torch

U = 2.0 ** -24


def chain(d):
    chunks = d // 8
    per = 1 if chunks <= 64 else 2 if chunks <= 128 else 1 if chunks <= 256 else 2 if chunks <= 512 else 4 if chunks <= 1024 else 8
    return 8 * per + 6 + 16


def half_step(t):
    return torch.finfo(t).eps / 2


def stored(value, err, dtype):
    """Bound on a stored value: the computed one's error, then half a step of it (float32 subnormals aside)."""
    return err + half_step(dtype) * (value.abs() + err) + 1e-38


def rstd(v, eps):
    return 1 / torch.sqrt(v.square().mean(dim=1) + eps)


def norm(h, weight, eps):
    """(x, error, r, relative error of r); h exact."""
    r = rstd(h, eps)
    dr = (chain(h.shape[1]) / 2 + 4) * U
    x = h * r[:, None] * weight
    return x, x.abs() * (dr + 3 * U), r, dr


def combined(y, pos, w):
    """c [T][d] and its error for pos [T][k] (-1: not kept), w [T][k] or None."""
    T, k = pos.shape
    c = torch.zeros(T, y.shape[1], dtype=torch.float64, device=y.device)
    e = torch.zeros_like(c)
    for i in range(k):
        rows = torch.where(pos[:, i, None] >= 0, y[pos[:, i].clamp(min=0)], 0.0)
        if w is not None:
            rows = rows * w[:, i, None]
        c = c + rows
        e = e + rows.detach().abs()
    return c, k * U * e


def after(y, pos, w, h, weight, gate, eps, res_scale):
    """(out, error, r, relative error of r) of combine, norm, gate and residual."""
    c, ec = combined(y, pos, w)
    r = rstd(c, eps)
    d = c.shape[1]
    dr = (chain(d) / 2 + 4) * U + (c.abs() * ec).mean(dim=1) * r * r
    g = weight if gate is None else weight * gate
    n = c * r[:, None] * g
    err = g.abs() * r[:, None] * ec + n.abs() * (dr[:, None] + 4 * U)
    res = res_scale * h
    out = res + n
    return out, err + 2 * U * (res.abs() + n.abs()), r, dr


def loss_after(y, pos, w, weight, gate, r_of, dout):
    """The scalar whose gradients moe_combine_norm_backward gives: <dout, gate (c r(c) weight)>."""
    c, _ = combined(y, pos, w)
    n = c * r_of(c)[:, None] * weight
    if gate is not None:
        n = n * gate
    return (n * dout).sum()
