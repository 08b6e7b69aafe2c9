"""The whole layer for a few tokens in 64 bits, with bounds on what float32
sums, the rounding of the intermediate and the stored type may change."""
import torch

import mx_reference as MX

U = 2.0 ** -24


def weight(w, s, fmt):
    """One stored matrix [rows][K] as float64."""
    if fmt == "fp8":
        rows, K = w.shape
        v = w.view(torch.float8_e4m3fn).double().view(rows // 128, 128, K // 128, 128)
        return (v * s.double()[:, None, :, None]).view(rows, K)
    if fmt == "mxfp4":
        return MX.values(w, s.t())
    return w.double()


def logits(x, w_router, bias):
    """(logits, bound): a float32 sum over K whose chain is at most K / 512 + 20 (threads, a wave, eight waves) and a bias."""
    v = x.double() @ w_router.double()
    e = ((x.shape[1] / 512 + 20) * U) * (x.double().abs() @ w_router.double().abs())
    if bias is not None:
        v = v + bias.double()
        e = e + U * v.abs()
    return v, e


def selection(logits, k):
    """Ids by (-logit, id), NaN as -inf, and gates, of the float32 logits as written."""
    v = logits.double().nan_to_num(nan=-float("inf"), posinf=float("inf"), neginf=-float("inf"))
    order = torch.sort(-v, dim=1, stable=True).indices[:, :k]
    w = torch.softmax(torch.gather(v, 1, order), dim=1)
    return order.to(torch.int32), w


def expert(x, mats, act):
    """(rows, bound) of one expert: x [n, d] float64, mats (gate, up, down) float64 as stored."""
    wg, wu, wd = mats
    d, F = x.shape[1], wg.shape[0]
    half = torch.finfo(act).eps / 2
    # four quarters of K: a chain of K / 4 products (two or more are added at a time), then three sums
    ca, cd = (d / 4 + 8) * U, (F / 4 + 8) * U
    a, b = x @ wg.t(), x @ wu.t()
    ea, eb = ca * (x.abs() @ wg.abs().t()), ca * (x.abs() @ wu.abs().t())
    silu = a * torch.sigmoid(a)
    es = 1.1 * ea + silu.abs() * (a.abs() + 8) * 2 * U
    h = silu * b
    eh = es * b.abs() + silu.abs() * eb + es * eb + h.abs() * 2 * U
    eh = eh + half * (h.abs() + eh) + 1e-38     # stored in the activation format
    y = h @ wd.t()
    return y, eh @ wd.abs().t() + cd * ((h.abs() + eh) @ wd.abs().t())


def layer(x, idx, gates, weights, scales, fmt, act, e0, El):
    """(out, bound) of the layer with given ids and gates."""
    T, d = x.shape
    out = torch.zeros(T, d, dtype=torch.float64, device=x.device)
    err = torch.zeros_like(out)
    for e in sorted(set(idx.flatten().tolist())):
        j = e - e0
        if not 0 <= j < El:
            continue
        t, i = (idx == e).nonzero(as_tuple=True)
        m = [weight(w[j], None if s is None else s[j], fmt) for w, s in zip(weights, scales)]
        y, ey = expert(x[t].double(), m, act)
        g = gates[t, i, None].double()
        out.index_add_(0, t, y * g)
        err.index_add_(0, t, g * (ey + (idx.shape[1] + 4) * U * y.abs()))
    return out, err + (torch.finfo(act).eps / 2) * (out.abs() + err) + 1e-38
