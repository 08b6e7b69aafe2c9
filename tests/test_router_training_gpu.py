"""Router training on the GPU, through the C ABI, against the definitions in
64 bits: the balance loss with its counts, the router's backward pass, the
combine's backward pass, the gradient norm and clipping, and a whole step of
them together.

Tolerances.  u = 2^-24 is half a step of float32, 2^-8 relative that of
bfloat16.  A float32 sum of a chain of n additions is off by at most n u times
the sum of magnitudes.  A softmax term exp(v - m): the argument (at most X in
magnitude) is rounded once when formed and once when scaled to base two, so
the term is off by 2 X u, the hardware exponential by 2 u, the sum of E terms
in a tree of at most 8 + 6 levels by 16 u, the division by 2 u: together
(2 X + 24) u relative.
"""
import numpy as np
import pytest
import torch

from mixture_experts_layer_15_amd import binding as B
from mixture_experts_layer_15_amd import synth

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
BF16 = 2.0 ** -8
ACT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def chain(T):
    """Longest float32 chain of a sum over tokens in the row kernels: the rows of a workgroup."""
    return T / 512 + 20


def routed(T, E, k, seed, spread=2.0):
    """Logits with a skewed load, top-k ids and gates (CPU tensors)."""
    g = gen(seed)
    L = torch.randn(T, E, generator=g) * spread + 2.0 * (torch.arange(E) + 1.0).pow(-1.1)
    top, idx = torch.topk(L, k, dim=1)
    return L, idx.to(torch.int32), torch.softmax(top, dim=1)


def make_mask(T, kind, seed):
    if kind is None:
        return None
    if kind == "none_left":
        return torch.zeros(T, dtype=torch.uint8)
    if kind == "tail":
        return (torch.arange(T) < max(1, (2 * T) // 3)).to(torch.uint8)
    return (torch.rand(T, generator=gen(seed + 99)) < 0.6).to(torch.uint8)


def dev(t):
    return None if t is None else t.to(DEV)


def softmax64(L):
    """p and log-sum-exp in 64 bits; a row of -inf only gives zeros."""
    L = L.double()
    m = L.max(dim=1, keepdim=True).values
    base = torch.where(m == -torch.inf, torch.zeros_like(m), m)
    e = torch.exp(L - base)
    s = e.sum(dim=1, keepdim=True)
    dead = s == 0
    p = torch.where(dead, torch.zeros_like(e), e / s)
    lse = torch.where(dead, torch.zeros_like(s), base + torch.log(s))
    return p, lse


def balance64(L, idx, mask, E, k):
    keep = torch.ones(len(L), dtype=torch.bool) if mask is None else mask.bool()
    ids = idx[keep].reshape(-1).long()
    ids = ids[(ids >= 0) & (ids < E)]
    counts = torch.bincount(ids, minlength=E)
    n = int(keep.sum())
    if n == 0:
        z = torch.zeros(E, dtype=torch.float64)
        return counts, 0, z, torch.zeros(2, dtype=torch.float64), torch.zeros(0, 1, dtype=torch.float64)
    p, lse = softmax64(L[keep])
    mean = p.mean(dim=0)
    losses = torch.stack([E / (n * k) * (counts.double() * mean).sum(), lse.square().mean()])
    return counts, n, mean, losses, lse


def run_balance(T, E, k, L, idx, mask, stream=None):
    p = B.problem(T, 128, E, k, 128, 0, E, "f32", "f32")
    o = dict(counts=torch.full((E,), -5, dtype=torch.int32, device=DEV),
             n_tokens=torch.full((1,), -5, dtype=torch.int32, device=DEV),
             prob_mean=torch.full((E,), 7.0, device=DEV), losses=torch.full((2,), 7.0, device=DEV))
    ws = B.workspace(p, B.MOE_CALL_BALANCE_LOSS, DEV)
    ws.fill_(0xA5)  # the contents on entry do not matter
    B.moe_balance_loss(p, dev(L), dev(idx), dev(mask), o["counts"], o["n_tokens"], o["prob_mean"], o["losses"], ws)
    torch.cuda.synchronize()
    return {n: t.cpu() for n, t in o.items()}


def check_balance(got, L, idx, mask, E, k):
    counts, n, mean, losses, lse = balance64(L, idx, mask, E, k)
    assert torch.equal(got["counts"].long(), counts)
    assert int(got["n_tokens"]) == n
    T = len(L)
    finite = L[torch.isfinite(L)]
    X = float(finite.max() - finite.min()) if finite.numel() else 0.0
    tol = (2 * X + 24 + chain(T)) * U
    assert torch.all((got["prob_mean"].double() - mean).abs() <= tol * mean + 1e-30)
    assert abs(float(got["losses"][0]) - float(losses[0])) <= (tol + 2 * U) * float(losses[0])
    # lse is off by u of its largest part and the logarithm's own few u
    d = (float(finite.abs().max()) + 8) * 2 * U if finite.numel() else 0.0
    ztol = float((2 * lse.abs() * d + d * d).mean()) if n else 0.0
    assert abs(float(got["losses"][1]) - float(losses[1])) <= ztol + 2 * U * float(losses[1])


BALANCE = [(1, 1, 1, None), (1, 8, 2, None), (3, 4, 4, "random"), (16, 8, 2, None), (17, 8, 2, "random"),
           (64, 8, 2, None), (64, 128, 8, "tail"), (100, 5, 2, None), (200, 3, 1, "random"),
           (333, 20, 3, "random"), (333, 50, 7, None), (257, 64, 6, "random"), (511, 100, 4, "tail"),
           (1000, 127, 8, "random"), (1001, 150, 6, "tail"), (700, 129, 5, None), (513, 256, 8, "random"),
           (300, 300, 16, "random"), (300, 511, 3, None), (300, 512, 8, "tail"), (130, 512, 512, None),
           (8192, 128, 8, "random"), (20011, 16, 2, "random"), (9000, 30, 4, None), (64, 8, 2, "none_left"),
           (2000, 64, 4, "none_left")]


@pytest.mark.parametrize("T,E,k,mask", BALANCE)
def test_balance_loss(T, E, k, mask):
    L, idx, _ = routed(T, E, k, seed=T + E)
    m = make_mask(T, mask, T)
    got = run_balance(T, E, k, L, idx, m)
    check_balance(got, L, idx, m, E, k)
    again = run_balance(T, E, k, L, idx, m)
    assert all(torch.equal(got[n], again[n]) for n in got)


def test_balance_ids_outside_and_twice():
    T, E, k = 300, 24, 4
    L, idx, _ = routed(T, E, k, seed=1)
    idx[::3, 1] = -1
    idx[1::5, 0] = E
    idx[2::7, 2] = 2 ** 31 - 1
    idx[4::9] = 5       # one expert four times
    m = make_mask(T, "random", 2)
    check_balance(run_balance(T, E, k, L, idx, m), L, idx, m, E, k)


@pytest.mark.parametrize("T,E", [(40, 8), (700, 150)])
def test_balance_masked_experts_and_dead_rows(T, E):
    """-inf logits (experts switched off), and rows that have nothing else."""
    k = 2
    L, idx, _ = routed(T, E, k, seed=5)
    L[:, 1::3] = -torch.inf
    L[3] = -torch.inf
    L[T - 1] = -torch.inf
    check_balance(run_balance(T, E, k, L, idx, None), L, idx, None, E, k)
    L[:] = -torch.inf
    got = run_balance(T, E, k, L, idx, None)
    assert torch.all(got["prob_mean"] == 0) and torch.all(got["losses"] == 0)
    assert int(got["n_tokens"]) == T and int(got["counts"].sum()) == T * k


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).max,
                                 torch.finfo(torch.float32).min])
def test_balance_ignores_what_masked_tokens_hold(bad):
    T, E, k = 500, 20, 3
    L, idx, _ = routed(T, E, k, seed=6)
    m = make_mask(T, "random", 6)
    clean = run_balance(T, E, k, L, idx, m)
    L2, idx2 = L.clone(), idx.clone()
    L2[m == 0] = bad
    idx2[m == 0] = -7
    got = run_balance(T, E, k, L2, idx2, m)
    assert all(torch.equal(got[n], clean[n]) for n in got)


def test_balance_nan_of_a_kept_token_shows():
    T, E, k = 500, 20, 3
    for bad in (float("nan"), float("inf")):
        L, idx, _ = routed(T, E, k, seed=7)
        L[77, 4] = bad
        got = run_balance(T, E, k, L, idx, None)
        assert torch.isnan(got["prob_mean"]).any() and torch.isnan(got["losses"]).all()
        L[77] = bad
        got = run_balance(T, E, k, L, idx, None)
        assert torch.isnan(got["prob_mean"]).all() and torch.isnan(got["losses"]).all()


def test_balance_zero_tokens():
    p = B.problem(0, 128, 10, 2, 128, 0, 10, "bf16", "bf16")
    o = [torch.full((10,), 3, dtype=torch.int32, device=DEV), torch.full((1,), 3, dtype=torch.int32, device=DEV),
         torch.full((10,), 3.0, device=DEV), torch.full((2,), 3.0, device=DEV)]
    B.moe_balance_loss(p, None, None, None, *o, B.workspace(p, B.MOE_CALL_BALANCE_LOSS, DEV))
    torch.cuda.synchronize()
    assert all(torch.all(t == 0) for t in o)


# ---- the router's backward pass

def dlogits64(L, idx, w, g, counts, n, dl, mask, E, k):
    """dL and, element by element, a bound of the float32 error."""
    T = len(L)
    keep = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    r = torch.zeros(T, E, dtype=torch.float64)
    b = torch.zeros(T, E, dtype=torch.float64)
    if dl is not None and n > 0:
        p, lse = softmax64(L)
        finite = L[keep][torch.isfinite(L[keep])]
        X = float(finite.max() - finite.min()) if finite.numel() else 0.0
        big = float(finite.abs().max()) if finite.numel() else 0.0
        s = (2 * X + 24) * U
        c = counts.double() - counts.double().sum() / E
        ca, cz = float(dl[0]) * E / (float(n) * n * k), float(dl[1]) * 2 / n
        mean = (c * p).sum(dim=1, keepdim=True)
        r += ca * p * (c - mean) + cz * lse * p
        spread = c.abs() + (c.abs() * p).sum(dim=1, keepdim=True)
        b += abs(ca) * p * spread * (2 * s + 20 * U)
        b += abs(cz) * p * (lse.abs() * (s + 4 * U) + (big + 8) * 2 * U)
    if g is not None:
        w, g, ids = w.double(), g.double(), idx.long()
        ok = (ids >= 0) & (ids < E)
        wg = torch.where(ok, w * g, torch.zeros_like(w))
        mean = wg.sum(dim=1, keepdim=True)
        step = torch.where(ok, w * (g - mean), torch.zeros_like(w))
        err = torch.where(ok, w.abs() * (g.abs() * 3 + wg.abs().sum(dim=1, keepdim=True) * (k + 3)) * U,
                          torch.zeros_like(w))
        at = torch.where(ok, ids, torch.zeros_like(ids))
        r.scatter_add_(1, at, step)
        b.scatter_add_(1, at, err)
        # each slot's addition to what is there rounds once
        mag = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, at, step.abs())
        b += (k + 1) * U * (mag + r.abs())
    b += 2 * U * r.abs()
    r[~keep] = 0
    b[~keep] = 0
    return r, b


OUT = ("dlogits", "dx", "dw_router", "dbias")


class Router:
    """One problem of the router's backward pass (CPU tensors) and its call."""

    def __init__(self, T, d, E, k, act, mask=None, gates=True, losses=True, seed=0):
        g = gen(1000 * seed + T + 7 * E + d)
        self.T, self.d, self.E, self.k, self.act = T, d, E, k, act
        self.L, self.idx, self.w = routed(T, E, k, seed + T + E)
        self.x = torch.randn(T, d, generator=g).to(ACT[act])
        self.w_router = (torch.randn(d, E, generator=g) / d ** 0.5).to(ACT[act])
        self.g = torch.randn(T, k, generator=g) * (0.05 / max(T, 1)) if gates else None
        self.dl = torch.tensor([1e-2, 1e-3]) if losses else None
        self.mask = make_mask(T, mask, seed + T)
        counts, n, _, _, _ = balance64(self.L, self.idx, self.mask, E, k)
        self.counts, self.n = counts.to(torch.int32), torch.tensor([n], dtype=torch.int32)
        self.p = B.problem(T, d, E, k, 128, 0, E, act, act)

    def buffers(self, want=OUT):
        shapes = dict(dlogits=((self.T, self.E), torch.float32), dx=((self.T, self.d), ACT[self.act]),
                      dw_router=((self.d, self.E), torch.float32), dbias=((self.E,), torch.float32))
        return {n: torch.full(shapes[n][0], 7.0, dtype=shapes[n][1], device=DEV) for n in want}

    def inputs(self):
        t = dict(x=self.x, w_router=self.w_router, logits=self.L, topk_idx=self.idx, topk_w=self.w,
                 dtopk_w=self.g, token_mask=self.mask, counts=self.counts, n_tokens=self.n, dlosses=self.dl)
        if self.g is None:
            t["topk_idx"] = t["topk_w"] = None
        if self.dl is None:
            t["logits"] = t["counts"] = t["n_tokens"] = None
        return {n: dev(v) for n, v in t.items()}

    def run(self, want=OUT):
        o = self.buffers(want)
        ws = B.workspace(self.p, B.MOE_CALL_ROUTE_BACKWARD, DEV)
        ws.fill_(0xFF)  # NaN patterns
        B.moe_route_backward(self.p, **self.inputs(), **o, ws=ws)
        torch.cuda.synchronize()
        return {n: t.cpu() for n, t in o.items()}

    def check(self, got):
        T, d, E, k = self.T, self.d, self.E, self.k
        dl, b = dlogits64(self.L, self.idx, self.w, self.g, self.counts, int(self.n), self.dl, self.mask, E, k)
        keep = torch.ones(T, dtype=torch.bool) if self.mask is None else self.mask.bool()
        x = torch.where(keep[:, None], self.x.double(), 0.0)
        w = self.w_router.double()
        if "dlogits" in got:
            assert torch.all((got["dlogits"].double() - dl).abs() <= b + 1e-37)
            assert torch.all(got["dlogits"][~keep] == 0)
        if "dbias" in got:
            e = (got["dbias"].double() - dl.sum(dim=0)).abs()
            assert torch.all(e <= b.sum(dim=0) + chain(T) * U * dl.abs().sum(dim=0) + 1e-37)
        if "dw_router" in got:
            ref = x.t() @ dl
            mag = x.abs().t() @ dl.abs()
            e = (got["dw_router"].double() - ref).abs()
            # at worst every product's addition rounds the same way ...
            assert torch.all(e <= x.abs().t() @ b + (3 * T + 8) * U * mag + 1e-37)
            # ... taken as independent, they add up like their root; the three planes drop nothing
            den = float(torch.linalg.norm(ref))
            if den > 0:
                rel = float(torch.linalg.norm(e)) / den
                own = float(torch.linalg.norm(x.abs().t() @ b)) / den
                assert rel <= own + 2 * U * (3 * T + 16) ** 0.5, rel
        if "dx" in got:
            ref = dl @ w.t()
            mag = dl.abs() @ w.abs().t()
            bf = self.act == "bf16"
            tol = b @ w.abs().t() + (2 * E + 8) * U * mag + (BF16 * ref.abs() if bf else 0.0)
            if bf:
                # dL in a float16 of 11 bits (half a step, eps / 2, is 2^-11 relative), each row scaled to a largest value
                # of at least 2^14: below the normal numbers half a step of 2^-24, 2^-39 of the largest; the
                # rows of the matrix (8 bits, exact) likewise
                tol += 2.0 ** -11 * mag
                tol += 2.0 ** -39 * dl.abs().amax(dim=1, keepdim=True) * w.abs().sum(dim=1)
                tol += 2.0 ** -39 * dl.abs().sum(dim=1, keepdim=True) * w.abs().amax(dim=1)
            assert torch.all((got["dx"].double() - ref).abs() <= tol * (1 + BF16) + 1e-37)
            assert torch.all(got["dx"][~keep] == 0)


ROUTER = [(1, 128, 1, 1, "bf16", None), (1, 128, 8, 2, "f32", None), (2, 256, 4, 1, "bf16", None),
          (64, 128, 8, 2, "f32", None), (64, 128, 8, 2, "f32", "random"), (37, 384, 20, 3, "f32", "tail"),
          (150, 256, 130, 4, "f32", "random"), (300, 128, 65, 5, "f32", None),
          (31, 128, 8, 2, "bf16", "random"), (64, 2048, 128, 8, "bf16", None), (127, 256, 32, 4, "bf16", None),
          (129, 384, 33, 3, "bf16", "random"), (200, 128, 64, 6, "bf16", "tail"), (333, 640, 20, 3, "bf16", "random"),
          (257, 256, 100, 8, "bf16", None), (400, 512, 127, 8, "bf16", "random"), (513, 128, 129, 8, "bf16", "tail"),
          (500, 256, 150, 6, "bf16", "random"), (300, 384, 256, 8, "bf16", "tail"), (260, 128, 300, 16, "bf16", "random"),
          (270, 256, 511, 20, "bf16", None), (200, 128, 512, 8, "bf16", "random"), (100, 128, 512, 512, "bf16", None),
          (2100, 1024, 128, 8, "bf16", "random"), (4100, 256, 8, 2, "bf16", "random"), (64, 256, 16, 2, "bf16", "none_left"),
          (40000, 128, 16, 2, "bf16", "random"), (3000, 128, 24, 2, "f32", "random")]


@pytest.mark.parametrize("T,d,E,k,act,mask", ROUTER)
def test_route_backward(T, d, E, k, act, mask):
    r = Router(T, d, E, k, act, mask)
    got = r.run()
    r.check(got)
    again = r.run()
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("want", [("dlogits",), ("dx",), ("dw_router",), ("dbias",), ("dw_router", "dbias"),
                                  ("dx", "dbias"), ("dlogits", "dx")])
def test_route_backward_single_outputs_have_the_same_bits(act, want):
    r = Router(213, 256, 40, 4, act, "random")
    full = r.run()
    r.check(full)
    got = r.run(want)
    assert all(torch.equal(got[n], full[n]) for n in want)


@pytest.mark.parametrize("gates,losses", [(True, False), (False, True)])
@pytest.mark.parametrize("E", [24, 50, 256])
def test_route_backward_one_gradient_alone(gates, losses, E):
    r = Router(190, 128, E, 3, "bf16", "random", gates=gates, losses=losses)
    r.check(r.run())


def test_route_backward_even_load_has_no_balance_gradient():
    """Counts that are all equal: the centred counts are zero, and so is the gradient, exactly."""
    r = Router(256, 128, 8, 8, "bf16", gates=False)
    r.dl = torch.tensor([1e-2, 0.0])
    assert torch.all(r.counts == r.counts[0])
    got = r.run()
    assert all(torch.all(t == 0) for t in got.values())


def test_route_backward_ids_outside_and_twice():
    r = Router(300, 128, 24, 4, "bf16", "random")
    r.idx[::3, 1] = -1
    r.idx[1::5, 0] = 24
    r.idx[2::7, 2] = 2 ** 31 - 1
    r.idx[4::9] = 5
    r.check(r.run())


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_route_backward_ignores_what_masked_tokens_hold(act, bad):
    r = Router(400, 256, 20, 3, act, "random")
    clean = r.run()
    r.check(clean)
    off = r.mask == 0
    for t in (r.x, r.L, r.w, r.g):
        t[off] = bad
    r.idx[off] = 12345
    got = r.run()
    assert all(torch.equal(got[n], clean[n]) for n in got)


def test_route_backward_experts_switched_off():
    """-inf logits have no probability and no gradient; a row of them has none at all."""
    r = Router(300, 128, 30, 3, "bf16")
    r.L[:, 1::3] = -torch.inf
    r.L[17] = -torch.inf
    r.g[:] = 0
    got = r.run()
    r.check(got)
    assert torch.all(got["dlogits"][:, 1::3] == 0) and torch.all(got["dlogits"][17] == 0)


def test_token_gradient_keeps_values_far_below_a_rows_largest():
    """The float16 form of a row of dL: a value 2^-30 of the largest, which meets the only nonzero row of the
    matrix, comes out within the row's 2^-39 and the formats' roundings."""
    T, d, E = 40, 128, 2
    r = Router(T, d, E, 2, "bf16", losses=False)
    r.idx[:] = torch.tensor([0, 1])
    r.w[:] = torch.tensor([0.5, 2.0 ** -31])
    r.g[:] = torch.tensor([1.0, -1.0])
    r.w_router[:, 0] = 0
    got = r.run(("dx",))
    r.check(got)
    ref = -1.5 * 2.0 ** -31 * r.w_router[:, 1].double()   # w (g - mean), mean = 0.5 to 2^-31
    assert torch.all((got["dx"].double() - ref).abs() <= ref.abs() * (BF16 + 2.0 ** -7))


def test_route_backward_infinite_gradient_stays_infinite():
    """A slot whose gate gradient overflows reaches the matrix' gradient as inf or NaN of its own experts only."""
    r = Router(70, 128, 40, 2, "bf16", losses=False)
    r.g[5] = torch.tensor([3e38, -3e38])
    r.w[5] = torch.tensor([4.0, 4.0])
    got = r.run()
    hit = torch.zeros(40, dtype=torch.bool)
    hit[r.idx[5].long()] = True
    assert not torch.isfinite(got["dw_router"][:, hit]).any()
    assert torch.isfinite(got["dw_router"][:, ~hit]).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_route_backward_zero_tokens(act):
    p = B.problem(0, 256, 12, 2, 128, 0, 12, act, act)
    dw, db = torch.full((256, 12), 3.0, device=DEV), torch.full((12,), 3.0, device=DEV)
    dummy = torch.zeros(2, device=DEV)
    B.moe_route_backward(p, dlosses=dummy, dw_router=dw, dbias=db, ws=B.workspace(p, B.MOE_CALL_ROUTE_BACKWARD, DEV))
    torch.cuda.synchronize()
    assert torch.all(dw == 0) and torch.all(db == 0)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_zero_tokens_through_empty_tensors(act):
    """A rank without tokens: empty tensors (null addresses), gradients of zeros."""
    E, d, k = 12, 256, 2
    p = B.problem(0, d, E, k, 128, 0, E, act, act)
    e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device=DEV)  # noqa: E731
    dw, db = torch.full((d, E), 3.0, device=DEV), torch.full((E,), 3.0, device=DEV)
    ws = B.workspace(p, B.MOE_CALL_ROUTE_BACKWARD, DEV)
    ids, a = e(0, k, t=torch.int32), ACT[act]
    B.moe_route_backward(p, x=e(0, d, t=a), topk_idx=ids, topk_w=e(0, k), dtopk_w=e(0, k), dw_router=dw, dbias=db, ws=ws)
    B.moe_route_backward(p, topk_idx=ids, topk_w=e(0, k), dtopk_w=e(0, k), dlogits=e(0, E), ws=ws)
    B.moe_combine_backward(p, e(0, d, t=a), e(0, d, t=a), ids, e(0, k), e(0, d, t=a), e(0, k))
    torch.cuda.synchronize()
    assert torch.all(dw == 0) and torch.all(db == 0)


def test_route_backward_counts_of_many_ranks():
    """Counts and tokens of a batch on many ranks: their sum passes 2^31."""
    r = Router(300, 128, 20, 4, "bf16", "random", gates=False)
    r.counts = torch.randint(1 << 29, (1 << 31) - 1, (20,), generator=gen(1), dtype=torch.int64)
    r.n = (r.counts.sum(dtype=torch.int64) // 20).clamp(max=2 ** 31 - 1).reshape(1)
    r.counts, r.n = r.counts.to(torch.int32), r.n.to(torch.int32)
    r.dl = torch.tensor([1e4, 0.0])
    r.check(r.run())


def test_gradients_against_differences_of_the_losses():
    """The kernel's dL against central differences of its own definition in 64 bits along random directions
    (h = 1e-5: the h^2 term is below 1e-9 of the slope's scale); the kernel's float32 error is the element bound."""
    T, E, k = 60, 16, 3
    r = Router(T, 128, E, k, "bf16", "random", gates=False)
    r.dl = torch.tensor([0.5, 0.25])
    got = r.run(("dlogits",))["dlogits"].double()
    _, b = dlogits64(r.L, r.idx, r.w, None, r.counts, int(r.n), r.dl, r.mask, E, k)
    dl = r.dl.double()
    g = gen(4)
    for _ in range(10):
        v = torch.randn(T, E, generator=g, dtype=torch.float64)
        h = 1e-5
        up, down = (balance64(r.L.double() + s * h * v, r.idx, r.mask, E, k)[3] @ dl for s in (1, -1))
        slope = float((got * v).sum())
        tol = float((b * v.abs()).sum()) + 1e-8 * float((got * v).abs().sum())
        assert abs((float(up) - float(down)) / (2 * h) - slope) <= tol


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_offsets_past_32_bits(act):
    """Logits, their gradient and its planes of more than 2^32 bytes: a few tokens at both ends are kept, the
    rows between hold NaN.  The results are those of the kept tokens alone."""
    n, d, E, k = 300, 128, 512, 4
    T = 2 ** 21 + 77
    r = Router(n, d, E, k, act)
    rows = torch.cat([torch.arange(100), torch.arange(T - 200, T)]).to(DEV)

    def spread(t, fill):
        out = torch.full((T,) + t.shape[1:], fill, dtype=t.dtype, device=DEV)
        out[rows] = t.to(DEV)
        return out

    p = B.problem(T, d, E, k, 128, 0, E, act, act)
    nan = float("nan")
    L, idx = spread(r.L, nan), spread(r.idx, 0)
    mask = spread(torch.ones(n, dtype=torch.uint8), 0)
    o = dict(counts=torch.full((E,), -5, dtype=torch.int32, device=DEV),
             n_tokens=torch.full((1,), -5, dtype=torch.int32, device=DEV),
             prob_mean=torch.full((E,), 7.0, device=DEV), losses=torch.full((2,), 7.0, device=DEV))
    B.moe_balance_loss(p, L, idx, mask, o["counts"], o["n_tokens"], o["prob_mean"], o["losses"],
                       B.workspace(p, B.MOE_CALL_BALANCE_LOSS, DEV))
    got = dict(dlogits=torch.full((T, E), 7.0, device=DEV), dx=torch.full((T, d), 7.0, dtype=ACT[act], device=DEV),
               dw_router=torch.full((d, E), 7.0, device=DEV), dbias=torch.full((E,), 7.0, device=DEV))
    B.moe_route_backward(p, x=spread(r.x, nan), w_router=dev(r.w_router), logits=L, topk_idx=idx,
                         topk_w=spread(r.w, nan), dtopk_w=spread(r.g, nan), token_mask=mask, counts=o["counts"],
                         n_tokens=o["n_tokens"], dlosses=dev(r.dl), **got,
                         ws=B.workspace(p, B.MOE_CALL_ROUTE_BACKWARD, DEV))
    torch.cuda.synchronize()
    check_balance({m: t.cpu() for m, t in o.items()}, r.L, r.idx, None, E, k)
    r.check({m: (t[rows] if len(t) == T else t).cpu() for m, t in got.items()})
    for m in ("dlogits", "dx"):
        got[m][rows] = 0
        assert int(torch.count_nonzero(got[m])) == 0


# ---- the combine's backward pass

def run_combine(T, d, E, local, k, act, gates=True, want=("dy", "dtopk_w"), seed=0):
    g = gen(seed + T + d)
    idx = torch.argsort(torch.rand(T, E, generator=g), dim=1)[:, :k].to(torch.int32)
    p = B.problem(T, d, E, k, 128, 0, local, act, act)
    di = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    pos = di(T * k)
    B.moe_permute(p, idx.to(DEV), di(local), di(local + 1), di(T * k), pos, B.workspace(p, B.MOE_CALL_PERMUTE, DEV))
    torch.cuda.synchronize()
    pos = pos.cpu()
    w = torch.rand(T, k, generator=g)
    y = torch.randn(T * k, d, generator=g).to(ACT[act])
    dout = torch.randn(T, d, generator=g).to(ACT[act])
    kept = (pos >= 0).nonzero()[:, 0]
    rows = pos[kept].long()
    tail = torch.ones(T * k, dtype=torch.bool)
    tail[rows] = False
    y[tail] = float("nan")   # rows behind the last kept slot are not read
    dy = torch.full((T * k, d), 7.0, dtype=ACT[act], device=DEV) if "dy" in want else None
    dw = torch.full((T, k), 7.0, device=DEV) if "dtopk_w" in want else None
    B.moe_combine_backward(p, dev(dout), dev(y), dev(pos), dev(w) if gates else None, dy, dw)
    torch.cuda.synchronize()
    do = dout.double()[kept // k]
    wk = w.reshape(-1)[kept].double() if gates else torch.ones(len(kept), dtype=torch.float64)
    if dy is not None:
        ref = do * wk[:, None]
        # one float32 product, one rounding to the format
        tol = ref.abs() * (U + (BF16 if act == "bf16" else 0)) * (1 + BF16)
        got = dy.cpu()
        assert torch.all((got[rows].double() - ref).abs() <= tol)
        assert torch.all(got[tail] == 7.0)
    if dw is not None:
        ref = torch.zeros(T * k, dtype=torch.float64)
        mag = torch.zeros(T * k, dtype=torch.float64)
        prod = do * y[rows].double()
        ref[kept], mag[kept] = prod.sum(dim=1), prod.abs().sum(dim=1)
        # a lane's share of the row, then six levels of the wave
        assert torch.all((dw.cpu().reshape(-1).double() - ref).abs() <= (d / 64 + 10) * U * mag)
        assert torch.all(dw.cpu().reshape(-1)[pos < 0] == 0)


@pytest.mark.parametrize("T,d,E,local,k", [(1, 128, 4, 4, 1), (1, 2048, 128, 128, 8), (5, 256, 16, 2, 3),
                                           (64, 2048, 128, 128, 8), (333, 640, 20, 7, 5), (100, 7168, 64, 8, 8),
                                           (50, 384, 100, 100, 70), (1025, 512, 8, 8, 2)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_combine_backward(T, d, E, local, k, act):
    run_combine(T, d, E, local, k, act)


@pytest.mark.parametrize("gates", [True, False])
@pytest.mark.parametrize("want", [("dy",), ("dtopk_w",), ("dy", "dtopk_w")])
def test_combine_backward_parts(gates, want):
    run_combine(77, 256, 12, 5, 3, "bf16", gates=gates, want=want)


def test_combine_backward_positions_outside_are_not_kept():
    T, d, k = 4, 128, 2
    p = B.problem(T, d, 4, k, 128, 0, 4, "bf16", "bf16")
    pos = torch.tensor([0, -1, 8, 1, 2 ** 31 - 1, -2 ** 31, 2, 3], dtype=torch.int32, device=DEV)
    dout = torch.ones(T, d, dtype=torch.bfloat16, device=DEV)
    y = torch.ones(T * k, d, dtype=torch.bfloat16, device=DEV)
    dy, dw = torch.full_like(y, 7.0), torch.full((T, k), 7.0, device=DEV)
    B.moe_combine_backward(p, dout, y, pos, None, dy, dw)
    torch.cuda.synchronize()
    assert dw.cpu().reshape(-1).tolist() == [128.0, 0, 0, 128.0, 0, 0, 128.0, 128.0]
    assert torch.all(dy[:4] == 1) and torch.all(dy[4:] == 7)


def test_combine_backward_of_more_slots_than_one_grid_dimension_holds():
    # a wave a slot, 71 million slots: more than 2^32 threads; slots at both ends and in between are kept
    T, d, k = 2 ** 22 - 8, 512, 17
    p = B.problem(T, d, 17, k, 128, 0, 17, "bf16", "bf16")
    S = T * k
    at = torch.tensor([0, 1, 5 * k + 3, S // 2, 2 ** 26 - 1, 2 ** 26, 2 ** 26 + 1, S - k, S - 1])
    n = len(at)
    pos = torch.full((S,), -1, dtype=torch.int32, device=DEV)
    pos[at.to(DEV)] = torch.arange(n, dtype=torch.int32, device=DEV)
    dout = torch.full((T, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    g = gen(5)
    rows = torch.randint(-3, 4, (n, d), generator=g).to(torch.bfloat16)
    dout[(at // k).to(DEV)] = rows.to(DEV)   # (a token of two kept slots has one of its rows)
    y = torch.randint(-3, 4, (n, d), generator=g).to(torch.bfloat16).to(DEV)
    dy, dw = torch.full_like(y, 7.0), torch.full((S,), 7.0, device=DEV)
    # no position names a row behind the n that are there: addresses, since the whole arrays have 73 GB
    B.moe_combine_backward(p, dout, y.data_ptr(), pos, None, dy.data_ptr(), dw)
    torch.cuda.synchronize()
    mine = dout[(at // k).to(DEV)]
    assert torch.equal(dy, mine)   # small integers: exact
    assert torch.equal(dw[at.to(DEV)].cpu(), (mine.cpu().double() * y.cpu().double()).sum(dim=1).float())
    dw[at.to(DEV)] = 0
    assert int(torch.count_nonzero(dw)) == 0


# ---- gradient norm and clipping

def norm64(ts):
    return float(np.sqrt(sum(float(t.double().square().sum()) for t in ts)))


def run_clip(ts, max_norm, out=None):
    """Norm, then clipped tensors (device); in place where out is None."""
    lst = B.grad_list(ts, out)
    norm = torch.full((1,), -3.0, device=DEV)
    ws = torch.full((max(B.moe_grad_workspace_size(lst), 256),), 0xFF, dtype=torch.uint8, device=DEV)
    B.moe_grad_norm(lst, norm, ws)
    B.moe_grad_clip(lst, norm, max_norm)
    torch.cuda.synchronize()
    return float(norm)


def check_clip(before, after, max_norm, norm):
    ref = norm64(before)
    assert abs(norm - ref) <= 2 * U * ref
    c = max_norm / ref if ref > max_norm else 1.0
    for b, a in zip(before, after):
        t = b.double() * c
        # the norm's and the scale's rounding, the product's, the format's
        tol = t.abs() * (4 * U + (BF16 if b.dtype is torch.bfloat16 else 0)) * (1 + BF16)
        if c == 1.0:
            assert torch.equal(a, b)
        else:
            assert torch.all((a.double() - t).abs() <= tol + 1e-40)


def tensors(sizes, seed=0):
    g = gen(seed)
    return [torch.randn(n, generator=g).to(torch.bfloat16 if i % 3 == 1 else torch.float32)
            for i, n in enumerate(sizes)]


@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [7, 9, 1], [16384], [16385, 3], [100003, 65536, 1, 12345],
                                   [1 << 20, 777], [33] * 113, [129, 4097, 1] * 100, [40_000_000, 13]])
@pytest.mark.parametrize("limit", [0.5, 1e9])
@pytest.mark.parametrize("place", ["in", "out"])
def test_norm_and_clipping(sizes, limit, place):
    before = tensors(sizes)
    ts = [t.to(DEV) for t in before]
    out = None if place == "in" else [torch.full_like(t, 7.0) for t in ts]
    norm = run_clip(ts, limit, out)
    check_clip(before, [t.cpu() for t in (out or ts)], limit, norm)
    if out:
        assert all(torch.equal(t.cpu(), b) for t, b in zip(ts, before))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift_in,shift_out", [(0, 0), (1, 1), (3, 3), (1, 0), (0, 5), (2, 7)])
def test_clipping_of_odd_addresses(dtype, shift_in, shift_out):
    """Tensors that start anywhere in a packed buffer; what lies between them stays."""
    n = [5, 20011, 64, 1, 30000]
    src = torch.randn(sum(n) + 16, generator=gen(1)).to(dtype).to(DEV)
    dst = torch.full_like(src, 7.0)
    at = np.cumsum([0] + n[:-1])
    ts = [src[shift_in + a:shift_in + a + m] for a, m in zip(at, n) if m != 64]
    out = [dst[shift_out + a:shift_out + a + m] for a, m in zip(at, n) if m != 64]
    before = [t.cpu().clone() for t in ts]
    norm = run_clip(ts, 1.0, out)
    check_clip(before, [t.cpu() for t in out], 1.0, norm)
    gap = at[2] + shift_out
    assert torch.all(dst[:shift_out] == 7) and torch.all(dst[gap:gap + 64] == 7)
    assert torch.all(dst[shift_out + sum(n):] == 7)


@pytest.mark.parametrize("scale", [1e30, 1e-30, 1e-42])
def test_norm_has_no_overflow_or_underflow(scale):
    ts = [torch.randn(5000, generator=gen(2)) * scale, torch.randn(777, generator=gen(3)) * scale]
    dv = [t.to(DEV) for t in ts]
    norm = run_clip(dv, 1.0)
    ref = norm64(ts)
    assert abs(norm - ref) <= 2 * U * ref + 2.0 ** -150   # half a step of the subnormal numbers
    if scale > 1:
        check_clip(ts, [t.cpu() for t in dv], 1.0, norm)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite_changes_nothing(bad):
    before = tensors([1000, 2000])
    before[1][77] = bad
    ts = [t.to(DEV) for t in before]
    out = [torch.full_like(t, 7.0) for t in ts]
    norm = run_clip(ts, 1.0, out)
    assert not np.isfinite(norm)
    assert all(torch.equal(t.cpu().view(torch.int16), b.view(torch.int16)) for t, b in zip(out, before))
    norm = run_clip(ts, 1.0)
    assert not np.isfinite(norm)
    assert all(torch.equal(t.cpu().view(torch.int16), b.view(torch.int16)) for t, b in zip(ts, before))


def test_clipping_takes_any_norm_and_an_empty_list_is_done():
    t = torch.full((100,), 3.0, device=DEV)
    norm = torch.tensor([6.0], device=DEV)   # for instance of this rank's and other ranks' tensors
    B.moe_grad_clip([t], norm, 2.0)
    assert torch.all(t == 1.0)
    B.moe_grad_clip([t], norm, float("inf"))
    assert torch.all(t == 1.0)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    B.moe_grad_norm([], norm, ws)
    B.moe_grad_norm([t[:0]], norm, ws)
    torch.cuda.synchronize()
    assert float(norm) == 0.0


# ---- streams, graphs, and a step of all of them

class Step:
    """A step of router tuning with frozen experts: route, permute, experts, combine; then, from the gradient
    of the output, the gates, the losses and the router, and clipping.  Buffers are made once."""

    def __init__(self, wl, mask=None, seed=3):
        pr = synth.make_problem(wl, seed=seed)
        self.wl, self.pr = wl, pr
        T, d, E, k = wl.T, wl.d, wl.E, wl.k
        act = pr.x.dtype
        self.p = B.problem(T, d, E, k, wl.F, 0, E, wl.act, wl.weight)
        self.i = {n: dev(getattr(pr, n)) for n in ("x", "w_router", "bias", "w_gate", "w_up", "w_down", "s_gate",
                                                   "s_up", "s_down")}
        self.mask = dev(mask)
        f = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
        i32 = torch.int32
        self.o = dict(logits=f(T, E), idx=f(T, k, t=i32), w=f(T, k), ecounts=f(E, t=i32), offsets=f(E + 1, t=i32),
                      sorted=f(T * k, t=i32), pos=f(T * k, t=i32), y=f(T * k, d, t=act), out=f(T, d, t=act),
                      counts=f(E, t=i32), n=f(1, t=i32), mean=f(E), losses=f(2), dtopk_w=f(T, k), dw=f(d, E),
                      db=f(E), dx=f(T, d, t=act), norm=f(1))
        self.dout = (torch.randn(T, d, generator=gen(seed)) / T).to(act)
        self.ddout = dev(self.dout)
        self.dl = torch.tensor([1e-2, 1e-3], device=DEV)
        self.grads = B.grad_list([self.o["dw"], self.o["db"]])
        calls = (B.MOE_CALL_ROUTE, B.MOE_CALL_PERMUTE, B.MOE_CALL_EXPERT_FFN, B.MOE_CALL_BALANCE_LOSS,
                 B.MOE_CALL_ROUTE_BACKWARD)
        n = max([B.moe_workspace_size(self.p, c) for c in calls] + [B.moe_grad_workspace_size(self.grads)])
        self.ws = torch.empty(n, dtype=torch.uint8, device=DEV)   # one scratch for the whole stream

    def run(self, stream=None, clip=True):
        p, i, o, ws = self.p, self.i, self.o, self.ws
        kw = dict(stream=stream)
        B.moe_route(p, i["x"], i["w_router"], i["bias"], o["logits"], o["idx"], o["w"], ws, **kw)
        B.moe_permute(p, o["idx"], o["ecounts"], o["offsets"], o["sorted"], o["pos"], ws, **kw)
        B.moe_expert_ffn(p, i["x"], o["sorted"], o["offsets"], i["w_gate"], i["w_up"], i["w_down"], i["s_gate"],
                         i["s_up"], i["s_down"], None, o["y"], ws, **kw)
        B.moe_combine(p, o["y"], o["pos"], o["w"], o["out"], **kw)
        B.moe_combine_backward(p, self.ddout, o["y"], o["pos"], o["w"], None, o["dtopk_w"], **kw)
        B.moe_balance_loss(p, o["logits"], o["idx"], self.mask, o["counts"], o["n"], o["mean"], o["losses"], ws, **kw)
        B.moe_route_backward(p, x=i["x"], w_router=i["w_router"], logits=o["logits"], topk_idx=o["idx"],
                             topk_w=o["w"], dtopk_w=o["dtopk_w"], token_mask=self.mask, counts=o["counts"],
                             n_tokens=o["n"], dlosses=self.dl, dx=o["dx"], dw_router=o["dw"], dbias=o["db"], ws=ws,
                             **kw)
        B.moe_grad_norm(self.grads, o["norm"], ws, **kw)
        if clip:
            B.moe_grad_clip(self.grads, o["norm"], 0.25 * self.limit if hasattr(self, "limit") else 1e9, **kw)

    def outputs(self):
        torch.cuda.synchronize()
        return {n: t.cpu().clone() for n, t in self.o.items()}


STEPS = {
    "f32": synth.WORKLOADS["tiny"],
    "bf16": synth.WORKLOADS["prefill"].replace(name="tuning_bf16", T=700, d=256, E=20, num_local=20, k=3, F=256,
                                               bias=("zipf", 1.1, 2.0), seed=21),
    "fp8": synth.WORKLOADS["dsv3_rank"].replace(name="tuning_fp8", T=300, d=256, E=16, num_local=16, k=4, F=256,
                                                seed=22),
}


@pytest.mark.parametrize("case", list(STEPS))
@pytest.mark.parametrize("masked", [False, True])
def test_a_step_of_router_tuning(case, masked):
    """The whole step against 64-bit autograd through the layer's definition: the expert outputs y are constants
    (the frozen experts' rows, as computed), the selection is the one taken."""
    wl = STEPS[case]
    mask = make_mask(wl.T, "tail", 1) if masked else None
    s = Step(wl, mask)
    s.dout[mask == 0 if masked else slice(0, 0)] = 0
    s.ddout.copy_(s.dout)
    s.run(clip=False)
    o = s.outputs()
    T, d, E, k = wl.T, wl.d, wl.E, wl.k
    assert torch.equal(o["counts"], o["ecounts"]) or masked
    x, wr = s.pr.x.double(), s.pr.w_router.double().requires_grad_(True)
    bias = (torch.zeros(E) if s.pr.bias is None else s.pr.bias).double().requires_grad_(True)
    L = x @ wr + bias
    L = L + (o["logits"].double() - L).detach()   # at the float32 logits the selection was taken on
    gates = torch.softmax(torch.gather(L, 1, o["idx"].long()), dim=1)
    y = o["y"].double()[o["pos"].long()].reshape(T, k, d)
    out = (gates[:, :, None] * y).sum(dim=1)
    keep = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    n = int(keep.sum())
    counts = torch.bincount(o["idx"][keep].reshape(-1).long(), minlength=E)
    bal = E / (n * k) * (counts * torch.softmax(L[keep], dim=1).mean(dim=0)).sum()
    z = torch.logsumexp(L[keep], dim=1).square().mean()
    assert torch.equal(o["counts"].long(), counts) and int(o["n"]) == n
    total = (out * s.dout.double()).sum() + 1e-2 * bal + 1e-3 * z
    dw, db = torch.autograd.grad(total, [wr, bias])
    # dL is off by about (k + 40) u relative (gates, their gradient from d products, softmax), the sum over tokens
    # by its root; float32 coefficients 1e-2 and 1e-3 by u
    tol = U * (2 * (d / 64 + 80) + 2 * (3 * T + 16) ** 0.5)
    for got, ref in ((o["dw"], dw), (o["db"], db)):
        mag = float(torch.linalg.norm(ref))
        assert float(torch.linalg.norm(got.double() - ref)) <= tol * mag * 4
    ref = float(torch.sqrt(dw.square().sum() + db.square().sum()))
    assert abs(float(o["norm"]) - ref) <= 4 * tol * ref
    # clipping to a quarter of the norm leaves exactly that norm
    s.limit = float(o["norm"])
    s.run()
    c = s.outputs()
    got = norm64([c["dw"], c["db"]])
    assert abs(got - 0.25 * s.limit) <= 4 * U * got + U * got * 4


def test_a_captured_step_replays_with_new_inputs():
    """The step in a graph, replayed with inputs changed in between, each replay against the eager calls."""
    s = Step(STEPS["bf16"], make_mask(STEPS["bf16"].T, "random", 3))
    e = Step(STEPS["bf16"], make_mask(STEPS["bf16"].T, "random", 3))
    s.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        s.run()
    for rep in range(4):
        x = torch.randn(s.i["x"].shape, generator=gen(50 + rep)).to(s.i["x"].dtype)
        for o in (s, e):
            o.i["x"].copy_(x)
            o.mask.copy_(make_mask(len(x), "random", 60 + rep))
        g.replay()
        e.run()
        a, b = s.outputs(), e.outputs()
        assert all(torch.equal(a[n], b[n]) for n in a), rep


def test_two_streams_at_once_give_the_same_bits():
    steps = [Step(STEPS["bf16"]), Step(STEPS["fp8"], make_mask(300, "random", 1))]
    alone = []
    for s in steps:
        s.run()
        alone.append(s.outputs())
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for s, st in zip(steps, streams):
            s.run(stream=st)
    for s, a in zip(steps, alone):
        got = s.outputs()
        assert all(torch.equal(got[n], a[n]) for n in a)


def test_host_tensors_are_refused():
    p = B.problem(4, 128, 8, 2, 128, 0, 8, "f32", "f32")
    z = torch.zeros
    with pytest.raises(B.MoEError, match="logits is on cpu"):
        B.moe_balance_loss(p, z(4, 8), z(4, 2, dtype=torch.int32), None, z(8, dtype=torch.int32, device=DEV),
                           z(1, dtype=torch.int32, device=DEV), z(8, device=DEV), z(2, device=DEV),
                           B.workspace(p, B.MOE_CALL_BALANCE_LOSS, DEV))
    with pytest.raises(B.MoEError, match="gradients"):
        B.moe_grad_norm([z(4)], z(1, device=DEV), z(256, dtype=torch.uint8, device=DEV))
