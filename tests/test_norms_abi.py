"""Norms around the layer on the host side: argument checks (no call here
reaches a kernel launch), the binding's tensor checks, and the gradients of
the formula against differences of it in 64 bits."""
import ctypes
import os

import numpy as np
import pytest
import torch

import norm_reference as R
from mixture_experts_layer_15_amd import binding as B

FAKE = 0x1000  # never dereferenced: the calls below fail their host checks
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from mixture_experts_layer_15_amd import build
        build.build()
    return B.load_library()


def _p(**kw):
    base = dict(T=64, d=256, E=8, k=2, F=256, expert_begin=0, num_local=8, act="bf16", weight="bf16")
    base.update(kw)
    return B.problem(**base)


def test_norm_refusals(lib):
    def call(p=_p(), h=FAKE, w=FAKE, eps=1e-6, x=2 * FAKE, r=FAKE):
        return lib.moe_norm(ctypes.byref(p), h, w, eps, x, r, None)
    for name in ("h", "w", "x"):
        assert call(**{name: None}) == B.MOE_ERR_INVALID_ARGUMENT
    for name in ("h", "w", "x", "r"):
        assert call(**{name: FAKE + 8}) == B.MOE_ERR_INVALID_ARGUMENT
    for eps in (0.0, -1e-6, float("nan")):
        assert call(eps=eps) == B.MOE_ERR_INVALID_ARGUMENT
    assert call(p=_p(d=100)) == B.MOE_ERR_INVALID_ARGUMENT
    assert call(p=_p(act="fp8")) == B.MOE_ERR_UNSUPPORTED
    assert call(p=_p(T=0), h=None, w=None, x=None, r=None) == B.MOE_OK


def test_norm_backward_refusals(lib):
    full = dict(dx=FAKE, h=2 * FAKE, weight=FAKE, rstd=FAKE, dout=FAKE, dh=3 * FAKE, dweight=FAKE)

    def call(p=_p(), ws=FAKE, nbytes=BIG, **kw):
        a = B.NormBackwardArgs(**{**full, **kw}, res_scale=1.0)
        return lib.moe_norm_backward(ctypes.byref(p), ctypes.byref(a), ws, nbytes, None)
    assert lib.moe_norm_backward(ctypes.byref(_p()), None, FAKE, BIG, None) == B.MOE_ERR_INVALID_ARGUMENT
    for name in ("dx", "h", "weight", "rstd"):
        assert call(**{name: None}) == B.MOE_ERR_INVALID_ARGUMENT
    for name in full:
        assert call(**{name: FAKE + 4}) == B.MOE_ERR_INVALID_ARGUMENT, name
    assert call(ws=FAKE + 4) == B.MOE_ERR_INVALID_ARGUMENT
    assert call(dh=None, dweight=None) == B.MOE_ERR_INVALID_ARGUMENT
    assert call(dh=2 * FAKE) == B.MOE_ERR_INVALID_ARGUMENT      # h itself
    for T in (0, 1, 64, 100000):
        need = B.moe_workspace_size(_p(T=T), B.MOE_CALL_NORM_BACKWARD)
        assert need > 0 and need % 256 == 0
        assert call(p=_p(T=T), nbytes=need - 1) == B.MOE_ERR_WORKSPACE_TOO_SMALL
        assert call(p=_p(T=T), ws=None) == B.MOE_ERR_WORKSPACE_TOO_SMALL


def test_combine_norm_refusals(lib):
    full = dict(y=FAKE, slot_pos=FAKE, topk_w=FAKE, h=2 * FAKE, weight=FAKE, gate=FAKE, out=3 * FAKE, rstd=4 * FAKE,
                next_weight=FAKE, next_x=5 * FAKE, next_rstd=6 * FAKE)

    def call(p=_p(), eps=1e-6, **kw):
        a = B.CombineNormArgs(**{**full, **kw}, eps=eps, res_scale=1.0)
        return lib.moe_combine_norm(ctypes.byref(p), ctypes.byref(a), None)
    assert lib.moe_combine_norm(ctypes.byref(_p()), None, None) == B.MOE_ERR_INVALID_ARGUMENT
    for name in ("y", "h", "weight", "out", "next_x"):
        assert call(**{name: None}) == B.MOE_ERR_INVALID_ARGUMENT, name
    for name in full:
        assert call(**{name: 7 * FAKE + 8}) == B.MOE_ERR_INVALID_ARGUMENT, name
    assert call(next_weight=None) == call(next_weight=None, next_x=None) == B.MOE_ERR_INVALID_ARGUMENT
    assert call(next_weight=None, next_rstd=None) == B.MOE_ERR_INVALID_ARGUMENT
    assert call(slot_pos=None) == B.MOE_ERR_INVALID_ARGUMENT     # k = 2
    assert call(out=FAKE) == call(next_x=3 * FAKE) == call(next_x=FAKE) == B.MOE_ERR_INVALID_ARGUMENT  # aliases
    assert call(next_rstd=4 * FAKE) == call(eps=0.0) == B.MOE_ERR_INVALID_ARGUMENT
    assert call(p=_p(T=0), y=None, slot_pos=None, h=None, weight=None, out=None) == B.MOE_OK


def test_combine_norm_backward_refusals(lib):
    full = dict(dout=FAKE, y=2 * FAKE, slot_pos=FAKE, topk_w=FAKE, weight=FAKE, rstd=FAKE, gate=FAKE, dy=3 * FAKE,
                dtopk_w=FAKE, dweight=FAKE, dgate=FAKE)

    def call(p=_p(), ws=FAKE, nbytes=BIG, **kw):
        a = B.CombineNormBackwardArgs(**{**full, **kw})
        return lib.moe_combine_norm_backward(ctypes.byref(p), ctypes.byref(a), ws, nbytes, None)
    assert lib.moe_combine_norm_backward(ctypes.byref(_p()), None, FAKE, BIG, None) == B.MOE_ERR_INVALID_ARGUMENT
    for name in ("dout", "y", "weight", "rstd"):
        assert call(**{name: None}) == B.MOE_ERR_INVALID_ARGUMENT
    for name in full:
        assert call(**{name: FAKE + 8}) == B.MOE_ERR_INVALID_ARGUMENT, name
    assert call(dy=None, dtopk_w=None, dweight=None, dgate=None) == B.MOE_ERR_INVALID_ARGUMENT
    assert call(dy=2 * FAKE) == call(dy=FAKE) == B.MOE_ERR_INVALID_ARGUMENT
    assert call(slot_pos=None, dtopk_w=None) == B.MOE_ERR_INVALID_ARGUMENT                  # k = 2
    assert call(p=_p(k=1), slot_pos=None) == B.MOE_ERR_INVALID_ARGUMENT                     # gates need slots
    for T in (0, 1, 5000):
        need = B.moe_workspace_size(_p(T=T), B.MOE_CALL_COMBINE_NORM_BACKWARD)
        assert need > 0 and call(p=_p(T=T), nbytes=need - 1) == B.MOE_ERR_WORKSPACE_TOO_SMALL
        assert call(p=_p(T=T), ws=None) == B.MOE_ERR_WORKSPACE_TOO_SMALL


def test_binding_checks_tensors():
    p = _p(T=4, d=128, k=2)
    h = torch.zeros(4, 128, dtype=torch.bfloat16)
    w = torch.ones(128)
    for bad in (dict(h=h.float()), dict(h=h[:3]), dict(weight=w.bfloat16()), dict(x=torch.zeros(128, 4, dtype=torch.bfloat16).t())):
        a = dict(h=h, weight=w, x=h.clone(), **{k: v for k, v in bad.items() if k not in ("h", "weight", "x")})
        a.update(bad)
        with pytest.raises(B.MoEError):
            B.moe_norm(p, a["h"], a["weight"], 1e-6, a["x"])
    with pytest.raises(B.MoEError):
        B.moe_combine_norm(p, y=h, h=h, weight=w, eps=1e-6, out=h.clone(), slot_pos=torch.zeros(8, dtype=torch.int32))


def _differences(f, t, step=1e-6):
    g = torch.zeros_like(t)
    flat, out = t.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + step
        up = float(f())
        flat[i] = keep - step
        out[i] = (up - float(f())) / (2 * step)
        flat[i] = keep
    return g


def test_gradient_formula_against_differences():
    """The formulas that the kernels compute, the 64-bit reference of the GPU tests, and differences agree."""
    gen = torch.Generator().manual_seed(3)
    T, d, k, eps = 3, 16, 2, 1e-3

    def rnd(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)
    y, w, weight, gate, dout = rnd(T * k, d), torch.rand(T, k, generator=gen, dtype=torch.float64), rnd(d), rnd(d), rnd(T, d)
    pos = torch.tensor([[4, 0], [1, -1], [-1, -1]])
    leaves = [y, w, weight, gate]

    def f():
        return R.loss_after(y, pos, w, weight, gate, lambda c: R.rstd(c, eps), dout)
    by_difference = [_differences(f, t) for t in leaves]
    for t in leaves:
        t.requires_grad_(True)
    by_reference = torch.autograd.grad(f(), leaves)
    c, _ = R.combined(y.detach(), pos, w.detach())
    r = R.rstd(c, eps)[:, None]
    n, u = c * r, weight.detach() * gate.detach() * dout
    dc = r * (u - n * (n * u).mean(dim=1, keepdim=True))
    dy, dw = torch.zeros_like(by_difference[0]), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        for i in range(k):
            if pos[t, i] >= 0:
                dy[pos[t, i]] = w[t, i].detach() * dc[t]
                dw[t, i] = dc[t] @ y[pos[t, i]].detach()
    s = (dout * n).sum(dim=0)
    formula = [dy, dw, gate.detach() * s, weight.detach() * s]
    for a, b, q in zip(by_difference, by_reference, formula):
        assert torch.allclose(a, b, rtol=1e-6, atol=1e-8)
        assert torch.allclose(b, q, rtol=1e-12, atol=1e-13)
    assert np.isfinite(float(f()))
