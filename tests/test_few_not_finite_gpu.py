"""The layer for a few tokens where weights or intermediates are infinite or
NaN: such a value stays with the tokens that chose its expert, the others keep
their bits, and an infinity stays one as the formula has it."""
import pytest
import torch

import few_reference as R
from mixture_experts_layer_15_amd import binding as B
from test_few_gpu import DEV, Case

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


def _pack(c):
    """The kept weights of c.w as they are now."""
    for i, which in enumerate((0, 0, 1)):
        if c.kept[i] is not c.w[i]:
            B.moe_pack_weights(c.p, which, c.w[i], c.kept[i])


def _run(c):
    c.out.fill_(7.0)
    c.run(router=False, bias=False)
    return c.out.clone()


def _same(a, b):
    """Equal values, NaN for NaN."""
    return torch.equal(a.double().nan_to_num(nan=1e300, posinf=2e300, neginf=-2e300),
                       b.double().nan_to_num(nan=1e300, posinf=2e300, neginf=-2e300))


def _spoil(c, e, col, f, kind):
    """One value of expert e's down matrix (or the scale of its block) becomes `kind`; returns the columns that it reaches."""
    fmt = c.fmt
    if fmt in ("f32", "bf16"):
        c.w[2][e, col, f] = {"inf": INF, "-inf": -INF, "nan": NAN}[kind]
        cols = slice(col, col + 1)
    elif fmt == "fp8" and kind == "nan":
        c.w[2][e, col, f] = 0x7F
        cols = slice(col, col + 1)
    elif fmt == "fp8":
        c.s[2][e, col // 128, f // 128] = INF if kind == "inf" else -INF
        cols = slice(col // 128 * 128, col // 128 * 128 + 128)
    else:
        c.s[2][e, f // 32, col] = 255
        cols = slice(col, col + 1)
    _pack(c)
    return cols


# T, d, E, k, F, first local expert, local experts: one to sixteen tokens, one part of the list and several, a second turn
# of the workgroups, one column group a workgroup and more than one step of a row
SHAPES = [(2, 128, 4, 1, 128, 0, 4), (5, 256, 8, 2, 384, 0, 8), (16, 640, 32, 4, 256, 0, 32), (16, 384, 12, 3, 640, 2, 9),
          (4, 16640, 6, 2, 128, 0, 6), (3, 34816, 4, 1, 128, 0, 4), (3, 2048, 128, 8, 768, 0, 128)]


@pytest.mark.parametrize("fmt,blocked", [("f32", False), ("bf16", False), ("bf16", True), ("fp8", False), ("fp8", True),
                                         ("mxfp4", False), ("mxfp4", True)])
@pytest.mark.parametrize("kind", ["inf", "-inf", "nan"])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_down_weight_reaches_its_own_tokens(shape, kind, fmt, blocked):
    T, d, E, k, F, e0, El = shape
    if fmt == "mxfp4" and kind == "-inf":
        kind = "nan"
    c = Case(*shape, fmt, blocked)
    g = torch.Generator(device=DEV).manual_seed(T + d)
    # experts local and chosen by some tokens, not by all
    c.logits = torch.randn(T, E, generator=g, device=DEV)
    c.logits[0, e0], c.logits[1:, e0] = 9.0, -9.0
    c.logits[T - 1, e0 + 1], c.logits[:T - 1, e0 + 1] = 8.0, -9.0
    if fmt == "fp8":
        c.s[2].clamp_(min=1e-4)      # (a code counts only where its block's scale is not zero)
    clean = _run(c)
    assert torch.isfinite(clean).all()
    touched = torch.zeros(T, d, dtype=torch.bool, device=DEV)
    for e, t, col, f in ((0, 0, d - 3, F - 5), (1, T - 1, 7, 3)):
        touched[t, _spoil(c, e, col, f, kind)] = True
        got = _run(c)
        assert _same(got[~touched], clean[~touched])
        if fmt != "mxfp4":           # (its byte 255 is no value: only the others' bits are promised)
            assert not torch.isfinite(got[touched]).any()
        if kind != "nan" and fmt in ("f32", "bf16"):
            want, _ = R.layer(c.x, c.idx, c.gates, c.w, c.s, fmt, c.out.dtype, e0, El)
            assert torch.isinf(want[touched]).all() and _same(got[touched].double(), want[touched])


@pytest.mark.parametrize("fmt,blocked", [("f32", False), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("T", [1, 5])
def test_an_infinite_intermediate_stays_infinite(T, fmt, blocked):
    """An infinite h of one expert: its token's results are infinities, of the sign that the formula gives."""
    d, E, k, F = 256, 8, 1, 256
    c = Case(T, d, E, k, F, 0, E, fmt, blocked)
    c.logits = -torch.ones(T, E, device=DEV)
    c.logits[:, 1] = 1.0
    c.logits[0, 3] = 2.0
    clean = _run(c)
    c.x[0, 17] = 1.5
    c.w[1][3, 40, 17] = INF
    c.w[2][3, :, 40] = c.w[2][3, :, 40].where(c.w[2][3, :, 40] != 0, 1.0)
    _pack(c)
    got = _run(c)
    want, _ = R.layer(c.x, c.idx, c.gates, c.w, c.s, fmt, c.out.dtype, 0, E)
    assert torch.isinf(want[0]).all()
    assert _same(got[0].double(), want[0])
    assert torch.equal(got[1:], clean[1:])


@pytest.mark.parametrize("blocked", [False, True])
def test_an_intermediate_behind_the_bfloat16_range(blocked):
    """h between bfloat16's largest value and float32's rounds to an infinity, as in moe_forward."""
    T, d, E, k, F = 3, 128, 4, 1, 128
    c = Case(T, d, E, k, F, 0, E, "bf16", blocked)
    c.logits = torch.full((T, E), -1.0, device=DEV)
    c.logits[torch.arange(T), torch.arange(T)] = 1.0
    clean = _run(c)
    c.x[1] = 0
    c.x[1, 9] = 1.0
    for m, e in ((0, 63), (1, 64)):
        c.w[m][1, 50, 9] = 181 / 128 * 2.0 ** e     # the product: 1.9996 * 2^127
    c.w[2][1] = c.w[2][1].where(c.w[2][1] != 0, 1.0)
    _pack(c)
    got = _run(c)
    out = torch.empty_like(got)
    B.moe_forward(c.p, x=c.x, w_router=None, router_bias=None, w_gate=c.kept[0], w_up=c.kept[1], w_down=c.kept[2], out=out,
                  logits=c.logits.clone(), ws=B.workspace(c.p, B.MOE_CALL_FORWARD, DEV))
    assert torch.isinf(out[1]).all()
    assert _same(got[1], out[1])
    assert torch.equal(got[[0, 2]], clean[[0, 2]])


def test_captured_with_a_fault_that_comes_and_goes():
    """A graph replayed with finite weights, with a NaN among them, and with finite ones again."""
    c = Case(6, 640, 16, 3, 384, 0, 16, "bf16", True)
    g = torch.Generator(device=DEV).manual_seed(4)
    c.logits = torch.randn(6, 16, generator=g, device=DEV)
    c.logits[:5, 2], c.logits[5, 2] = -9.0, 9.0
    clean = _run(c)
    good = c.kept[2].clone()
    c.w[2][2, 33] = NAN
    _pack(c)
    bad = c.kept[2].clone()
    c.kept[2].copy_(good)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(router=False, bias=False)
    for weights in (good, bad, good, bad, bad, good):
        c.kept[2].copy_(weights)
        c.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        want = clean.clone()
        if weights is bad:
            want[5, 33] = NAN
        assert _same(c.out, want)
