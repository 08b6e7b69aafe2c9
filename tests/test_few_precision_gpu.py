"""What the layer for a few tokens promises beyond moe_forward: h is kept as a
value and its remainder, so that the experts' products see it within 2^-16 of
itself; and the logits within the steps of the router's own sums."""
import pytest
import torch

import few_reference as FR
from mixture_experts_layer_15_amd import binding as B
from test_few_gpu import DEV, Case

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
H = 2.0 ** -8      # half a step of bfloat16, relative


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


def _bf16(v):
    return v.to(torch.bfloat16).double()


def _intermediate(x, wg, wu):
    """(h, bound) in 64 bits: x [d], matrices [F][d] as stored."""
    d = x.shape[0]
    # a wave adds a quarter of K, two products or more at a time, then three sums; FP8 also a scale a block
    c = (d / 4 + 8) * U
    a, b = wg @ x, wu @ x
    ea, eb = c * (wg.abs() @ x.abs()), c * (wu.abs() @ x.abs())
    silu = a * torch.sigmoid(a)
    # |silu'| < 1.1; the hardware's exponential and reciprocal: a step each, the exponent's product |a| steps
    es = 1.1 * ea + silu.abs() * (a.abs() + 8) * 2 * U
    h = silu * b
    return h, es * b.abs() + silu.abs() * eb + es * eb + h.abs() * 3 * U


def _signs(c, e, lo):
    """Expert e's down matrix: +-1 / 1024 (FP8 and MXFP4 by scales) with the signs of the remainders, every second row negated."""
    F, d, fmt = c.shape[4], c.shape[1], c.fmt
    s = torch.where(lo < 0, -1.0, 1.0)[None, :].repeat(d, 1)
    s[1::2] *= -1
    if fmt == "bf16":
        c.w[2][e] = s / 1024
        return
    if fmt == "fp8":
        c.w[2][e] = torch.where(s < 0, 0xB8, 0x38).to(torch.uint8)     # -1, 1
        c.s[2][e] = 1 / 1024
    else:
        code = torch.where(s < 0, 0xA, 0x2).to(torch.uint8)            # -1, 1
        c.w[2][e] = code[:, 0::2] | (code[:, 1::2] << 4)
        c.s[2][e] = 127 - 10


@pytest.mark.parametrize("fmt,blocked", [("bf16", False), ("bf16", True), ("fp8", False), ("fp8", True), ("mxfp4", False), ("mxfp4", True)])
@pytest.mark.parametrize("T,d,F", [(1, 128, 640), (3, 256, 1024), (16, 128, 768)])
def test_the_remainders_of_h_enter_the_product(T, d, F, fmt, blocked):
    """Down rows with the signs of what bfloat16 rounding takes from h: without the remainders every result would be off by
    the sum of their magnitudes, which is more than the bound."""
    c = Case(T, d, T, 1, F, 0, T, fmt, blocked)
    c.logits = torch.full((T, T), -1.0, device=DEV)
    c.logits[torch.arange(T), torch.arange(T)] = 1.0       # token t to expert t, with gate 1
    if fmt == "fp8":
        for i in (0, 1):
            c.s[i].clamp_(min=0.5 / (100 * d ** 0.5))       # (no block of zeros)
    want, err, short = [], [], []
    for t in range(T):
        x = c.x[t].double()
        wg, wu = (FR.weight(c.w[i][t], None if c.s[i] is None else c.s[i][t], fmt) for i in (0, 1))
        h, eh = _intermediate(x, wg, wu)
        lo = h - _bf16(h)
        _signs(c, t, lo)
        wd = FR.weight(c.w[2][t], None if c.s[2] is None else c.s[2][t], fmt)
        # value and remainder: each rounded by at most half a step, the remainder's of H |h|
        ek = eh + H * H * (h.abs() + eh) + 1e-38
        y = wd @ h
        # both planes' sums: a wave adds a quarter of F, two products or more at a time; three sums, and the planes'
        ey = wd.abs() @ ek + (F / 4 + 9) * U * (wd.abs() @ (h.abs() * (1 + H) + ek))
        want.append(y)
        err.append(ey + H * (y.abs() + ey) + 1e-38)
        short.append(wd @ _bf16(h))
    want, err, short = torch.stack(want), torch.stack(err), torch.stack(short)
    assert ((short - want).abs() > err).all()               # (the test sees a missing remainder)
    if blocked:
        for i, which in enumerate((0, 0, 1)):
            B.moe_pack_weights(c.p, which, c.w[i], c.kept[i])
    c.run(router=False, bias=False)
    assert torch.equal(c.gates, torch.ones_like(c.gates))
    over = (c.out.double() - want).abs() - err
    assert float(over.max()) <= 0, (float(over.max()), float((short - want).abs().min()), float(err.max()))


def _logit_bound(x, w_router, bias):
    """(logits, bound): a thread's chain is four products for each 4096 rows of K, then six sums of a wave and fifteen of
    the waves, and the bias."""
    K = x.shape[1]
    v = x.double() @ w_router.double()
    e = 1.001 * (4 * -(-K // 4096) + 6 + 15) * U * (x.double().abs() @ w_router.double().abs())
    if bias is not None:
        v = v + bias.double()
        e = e + U * (v.abs() + e)
    return v, e + 1e-38


@pytest.mark.parametrize("fmt", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 3, 16])
@pytest.mark.parametrize("d,E", [(128, 1), (128, 37), (640, 128), (4096, 50), (4224, 256), (16384, 510)])
def test_logits(d, E, T, fmt):
    c = Case(T, d, E, 1, 128, 0, 1, fmt, False)
    # terms of one sign as well, where the roundings of a chain add up
    for same in (False, True):
        if same:
            c.x.abs_()
            c.w_router.abs_()
        for bias in (True, False):
            c.logits.fill_(float("nan"))
            c.run(bias=bias)
            want, err = _logit_bound(c.x, c.w_router, c.bias if bias else None)
            over = (c.logits.double() - want).abs() - err
            assert float(over.max()) <= 0, (same, bias, float(over.max()))
