"""The layer for a few tokens within the bounds of tests/few_reference.py, in
every format and layout, from one token to sixteen."""
import threading

import pytest
import torch

import few_reference as R
from mixture_experts_layer_15_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _act(fmt):
    return torch.float32 if fmt == "f32" else torch.bfloat16


def _experts(El, d, F, fmt, g):
    ws, ss = [], []
    for rows, K in ((F, d), (F, d), (d, F)):
        s = None
        if fmt in ("f32", "bf16"):
            w = (torch.randn(El, rows, K, generator=g, device=DEV) / K ** 0.5).to(_act(fmt))
        elif fmt == "fp8":
            w = (torch.randn(El, rows, K, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s = (0.5 + torch.rand(El, rows // 128, K // 128, generator=g, device=DEV)) / (100 * K ** 0.5)
            s *= torch.randint(0, 4, s.shape, generator=g, device=DEV) != 0     # some blocks are zero
        else:
            w = torch.randint(0, 256, (El, rows, K // 2), generator=g, device=DEV, dtype=torch.uint8)
            top = 127 - round(float(torch.log2(torch.tensor(2.9 * K ** 0.5))))
            s = torch.randint(top - 2, top + 2, (El, K // 32, rows), generator=g, device=DEV, dtype=torch.uint8)
        ws.append(w)
        ss.append(s)
    return ws, ss


class Case:
    def __init__(self, T, d, E, k, F, e0, El, fmt, blocked, seed=0):
        g = _gen(seed + T * d + E + k)
        self.shape, self.fmt = (T, d, E, k, F, e0, El), fmt
        self.p = B.problem(T, d, E, k, F, e0, El, "f32" if fmt == "f32" else "bf16", fmt, blocked)
        act = _act(fmt)
        self.x = torch.randn(T, d, generator=g, device=DEV).to(act)
        self.w_router = (torch.randn(d, E, generator=g, device=DEV) / d ** 0.5).to(act)
        self.bias = torch.randn(E, generator=g, device=DEV) * 0.1
        self.w, self.s = _experts(El, d, F, fmt, g)
        self.kept = self.w
        if blocked:
            self.kept = [torch.empty_like(w) for w in self.w]
            for which, src, dst in zip((0, 0, 1), self.w, self.kept):
                B.moe_pack_weights(self.p, which, src, dst)
        nan = float("nan")
        self.out = torch.full((T, d), nan, dtype=act, device=DEV)
        self.logits = torch.full((T, E), nan, device=DEV)
        self.idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
        self.gates = torch.full((T, k), nan, device=DEV)
        self.ws = B.workspace(self.p, B.MOE_CALL_FORWARD_FEW, DEV).fill_(0xFF)

    def run(self, stream=None, router=True, bias=True, **kw):
        a = dict(logits=self.logits, topk_idx=self.idx, topk_w=self.gates, out=self.out, ws=self.ws)
        a.update(kw)
        B.moe_forward_few(self.p, x=self.x, w_router=self.w_router if router else None, router_bias=self.bias if bias else None,
                          w_gate=self.kept[0], w_up=self.kept[1], w_down=self.kept[2], s_gate=self.s[0], s_up=self.s[1], s_down=self.s[2],
                          stream=stream, **a)

    def check(self, router=True, bias=True):
        T, d, E, k, F, e0, El = self.shape
        if router:
            want, err = R.logits(self.x, self.w_router, self.bias if bias else None)
            assert ((self.logits.double() - want).abs() <= err).all()
        idx, gates = R.selection(self.logits, k)
        assert torch.equal(self.idx, idx)
        assert torch.allclose(self.gates.double(), gates, rtol=(k + 16) * 2.0 ** -23, atol=1e-38)
        want, err = R.layer(self.x, idx, self.gates, self.w, self.s, self.fmt, _act(self.fmt), e0, El)
        got = self.out.double()
        assert torch.isfinite(got).all()
        over = (got - want).abs() - err
        assert float(over.max()) <= 0, (float(over.max()), float((got - want).abs().max()), float(want.abs().max()))
        if float(want.norm()):
            assert float((got - want).norm() / want.norm()) < (1e-5 if self.fmt == "f32" else 8e-3)


# T, d, E, k, F, first local expert, local experts
SHAPES = [(1, 128, 1, 1, 128, 0, 1), (1, 2048, 128, 8, 768, 0, 128), (2, 256, 5, 3, 384, 0, 5), (3, 640, 20, 3, 384, 0, 20),
          (4, 384, 150, 6, 128, 30, 70), (5, 2176, 8, 2, 256, 0, 8), (16, 256, 8, 2, 640, 0, 8), (16, 128, 512, 16, 128, 0, 512),
          (7, 1152, 31, 30, 128, 3, 20), (1, 256, 300, 256, 128, 0, 300), (16, 7168, 6, 2, 128, 2, 2), (9, 128, 16, 4, 2048, 0, 16)]


@pytest.mark.parametrize("fmt,blocked", [("f32", False), ("bf16", False), ("bf16", True), ("fp8", False), ("fp8", True),
                                         ("mxfp4", False), ("mxfp4", True)])
@pytest.mark.parametrize("shape", SHAPES)
def test_layer(shape, fmt, blocked):
    c = Case(*shape, fmt, blocked)
    c.run()
    c.check()
    first = c.out.clone()
    for bias in (True, False):      # again on the used scratch, and without a bias
        c.out.fill_(float("nan"))
        c.run(bias=bias)
        if bias:
            assert torch.equal(c.out, first)
        else:
            c.check(bias=False)


@pytest.mark.parametrize("fmt", ["f32", "bf16"])
def test_given_logits(fmt):
    """Logits as an input: ties, infinities, NaN; optional outputs left out; no local expert touched."""
    T, d, E, k, F = 8, 256, 100, 5, 128
    c = Case(T, d, E, k, F, 0, E, fmt, False)
    g = _gen(1)
    c.logits = torch.randint(0, 3, (T, E), generator=g, device=DEV).float()
    c.logits[1] = -0.0
    c.logits[1, ::2] = 0.0
    c.logits[2, 10:] = -float("inf")
    c.logits[3, :] = float("nan")
    c.logits[3, 50:60] = 1.0
    c.logits[4] = -3e38
    c.logits[4, 77] = 3e38
    kept = c.logits.clone()
    c.run(router=False, bias=False)
    assert torch.equal(c.logits.view(torch.int32), kept.view(torch.int32))
    c.check(router=False)
    out = c.out.clone()
    c.out.fill_(float("nan"))
    c.run(router=False, bias=False, topk_idx=None, topk_w=None)
    assert torch.equal(c.out, out)
    # every token routed to experts of another rank
    r = Case(T, d, E, k, F, 90, 10, fmt, False)
    r.logits = torch.arange(E, 0, -1, device=DEV).float().repeat(T, 1)
    r.run(router=False, bias=False)
    assert not r.out.any()
    # and one row of a batch only
    r.logits[3] = torch.arange(E, device=DEV).float()
    r.out.fill_(float("nan"))
    r.run(router=False, bias=False)
    r.check(router=False)
    assert r.out[3].any() and not r.out[:3].any() and not r.out[4:].any()


def test_logits_of_the_workspace_and_router_without_bias():
    c = Case(6, 640, 64, 4, 256, 0, 64, "bf16", True)
    c.run(bias=False)
    c.check(bias=False)
    out = c.out.clone()
    c.run(bias=False, logits=None, topk_idx=None, topk_w=None)
    assert torch.equal(c.out, out)


def test_nan_stays_in_its_token():
    c = Case(5, 256, 16, 2, 256, 0, 16, "bf16", True)
    g = _gen(3)
    c.logits = torch.randn(5, 16, generator=g, device=DEV)
    c.run(router=False, bias=False)
    clean = c.out.clone()
    c.x[2, 100] = float("nan")
    c.run(router=False, bias=False)
    assert torch.isnan(c.out[2]).all()
    keep = torch.arange(5, device=DEV) != 2
    assert torch.equal(c.out[keep], clean[keep])


@pytest.mark.parametrize("fmt", ["f32", "bf16", "fp8", "mxfp4"])
def test_agrees_with_the_layer_of_many_kernels(fmt):
    T, d, E, k, F = 16, 2048, 32, 8, 768
    c = Case(T, d, E, k, F, 4, 24, fmt, fmt != "f32")
    c.s = [None if s is None else s.clamp(min=1e-6) if fmt == "fp8" else s for s in c.s]
    c.run()
    out = torch.empty_like(c.out)
    lg = c.logits.clone()
    B.moe_forward(c.p, x=c.x, w_router=None, router_bias=None, w_gate=c.kept[0], w_up=c.kept[1], w_down=c.kept[2], s_gate=c.s[0], s_up=c.s[1],
                  s_down=c.s[2], out=out, logits=lg, ws=B.workspace(c.p, B.MOE_CALL_FORWARD, DEV))
    rel = float((out.double() - c.out.double()).norm() / out.double().norm())
    assert rel < (1e-5 if fmt == "f32" else 1e-2)


def test_captured_with_changing_routing():
    """Replays with other tokens (other experts) between eager calls on the same and on other scratch."""
    for fmt in ("bf16", "mxfp4"):
        c = Case(4, 640, 64, 6, 384, 0, 64, fmt, True)
        c.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run()
        g = _gen(11)
        other = B.workspace(c.p, B.MOE_CALL_FORWARD_FEW, DEV)
        for n in range(6):
            c.x.copy_(torch.randn(4, 640, generator=g, device=DEV))
            c.out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            got = c.out.clone()
            c.check()
            c.run(ws=other if n % 2 else c.ws)
            torch.cuda.synchronize()
            assert torch.equal(c.out, got)


def test_many_calls_in_a_row_on_one_scratch():
    """The scratch of one call is the next one's without a wait between them: a row or counter read stale would show."""
    cases = [Case(T, 1024, 32, 4, 512, 0, 32, "bf16", True, seed=T) for T in (1, 16, 3, 8)]
    want = []
    for c in cases:
        c.run()
        torch.cuda.synchronize()
        c.check()
        want.append(c.out.clone())
    ws = torch.empty(max(c.ws.numel() for c in cases), dtype=torch.uint8, device=DEV)
    outs = []
    for n in range(40):
        c = cases[n % 4]
        out = torch.empty_like(c.out)
        c.run(ws=ws, out=out)
        outs.append(out)
    torch.cuda.synchronize()
    for n, out in enumerate(outs):
        assert torch.equal(out, want[n % 4]), n


def test_several_streams_and_host_threads():
    """Calls on four streams at once, from two host threads each with its own workspace, beside a large copy."""
    cases = [Case(T, 2048, 64, 8, 768, 0, 64, fmt, True, seed=T) for T, fmt in ((1, "bf16"), (16, "fp8"), (5, "mxfp4"), (16, "bf16"))]
    want = []
    for c in cases:
        c.run()
        torch.cuda.synchronize()
        want.append(c.out.clone())
    streams = [torch.cuda.Stream() for _ in cases]
    big = torch.zeros(64 << 20, device=DEV)
    errors = []

    def work(part):
        try:
            for _ in range(10):
                for n in part:
                    cases[n].run(stream=streams[n])
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(part,)) for part in ((0, 1), (2, 3))]
    for t in threads:
        t.start()
    for _ in range(5):
        big.add_(1.0)
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for c, w in zip(cases, want):
        assert torch.equal(c.out, w)
