"""Every kernel variant of the router's backward pass (the cases of
router_plans, which a host test holds to the library's own rules) against the
definition in 64 bits.

Tolerances: those of test_router_training_gpu, with u = 2^-24 half a step of
float32; a bfloat16 result rounds by 2^-8, and of dL two bfloat16 planes (16
bits and a sign: 2^-17) go into the tokens' gradient.
"""
import pytest
import torch

import router_plans as R
from mixture_experts_layer_15_amd import binding as B
from test_router_training_gpu import ACT, BF16, DEV, U, balance64, chain, dlogits64, make_mask, routed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


def name(c):
    T, d, E, _, act, mask, want = c
    return f"{act}-{T}x{d}x{E}-{'masked' if mask else 'whole'}-{'all' if want == R.ALL else 'dw' if want == R.DW else 'dx'}"


class Problem:
    def __init__(self, T, d, E, k, act, mask, want):
        self.T, self.d, self.E, self.k, self.act, self.want = T, d, E, k, act, want
        g = torch.Generator(device=DEV).manual_seed(T + 7 * E + d)
        L, idx, w = routed(T, E, k, T + E)
        self.mask = make_mask(T, mask, T)
        counts, n, _, _, _ = balance64(L, idx, self.mask, E, k)
        gates = torch.randn(T, k, generator=torch.Generator().manual_seed(T)) * (0.05 / T)
        dl = torch.tensor([1e-2, 1e-3])
        self.host = (L, idx, w, gates, counts.to(torch.int32), n, dl)
        self.inputs = dict(logits=L, topk_idx=idx, topk_w=w, dtopk_w=gates, counts=counts.to(torch.int32),
                           n_tokens=torch.tensor([n], dtype=torch.int32), dlosses=dl, token_mask=self.mask)
        self.inputs = {m: None if t is None else t.to(DEV) for m, t in self.inputs.items()}
        self.x = torch.randn(T, d, generator=g, device=DEV).to(ACT[act])
        self.w_router = (torch.randn(d, E, generator=g, device=DEV) / d ** 0.5).to(ACT[act])
        self.keep = torch.ones(T, dtype=torch.bool, device=DEV) if self.mask is None else self.mask.bool().to(DEV)
        self.x[~self.keep] = float("nan")   # padding
        self.p = B.problem(T, d, E, k, 128, 0, E, act, act)
        self.ws = B.workspace(self.p, B.MOE_CALL_ROUTE_BACKWARD, DEV)

    def run(self, x):
        shapes = dict(dlogits=((self.T, self.E), torch.float32), dx=((self.T, self.d), ACT[self.act]),
                      dw_router=((self.d, self.E), torch.float32), dbias=((self.E,), torch.float32))
        o = {m: torch.full(shapes[m][0], 7.0, dtype=shapes[m][1], device=DEV) for m in self.want}
        self.ws.fill_(0xFF)
        B.moe_route_backward(self.p, x=x, w_router=self.w_router, **self.inputs, **o, ws=self.ws)
        torch.cuda.synchronize()
        return o


@pytest.mark.parametrize("case", R.CASES, ids=name)
def test_router_backward_variant(case):
    r = Problem(*case)
    T, d, E, k = r.T, r.d, r.E, r.k
    L, idx, w, gates, counts, n, coef = r.host
    dl, b = (t.to(DEV) for t in dlogits64(L, idx, w, gates, counts, n, coef, r.mask, E, k))
    got = r.run(r.x)
    assert torch.all((got["dlogits"].double() - dl).abs() <= b + 1e-37)
    assert torch.all(got["dlogits"][~r.keep] == 0)
    if "dbias" in got:
        e = (got["dbias"].double() - dl.sum(dim=0)).abs()
        assert torch.all(e <= b.sum(dim=0) + chain(T) * U * dl.abs().sum(dim=0) + 1e-37)
    if "dw_router" in got:
        x = torch.where(r.keep[:, None], r.x.double(), 0.0)
        ref = x.t().contiguous() @ dl
        e = (got["dw_router"].double() - ref).abs()
        xt = x.abs().t().contiguous()
        own = xt @ b
        assert torch.all(e <= own + (3 * T + 8) * U * (xt @ dl.abs()) + 1e-37)
        den = float(torch.linalg.norm(ref))
        assert float(torch.linalg.norm(e)) <= float(torch.linalg.norm(own)) + 2 * U * (3 * T + 16) ** 0.5 * den
        del x, xt, ref, e, own
    if "dx" in got:
        wt = r.w_router.double().t().contiguous()
        ref, mag = dl @ wt, dl.abs() @ wt.abs()
        tol = b @ wt.abs() + (2 * E + 8) * U * mag
        if r.act == "bf16":
            tol += 2.0 ** -17 * mag + BF16 * ref.abs()
        assert torch.all((got["dx"].double() - ref).abs() <= tol * (1 + BF16) + 1e-37)
        assert torch.all(got["dx"][~r.keep] == 0)
        del ref, mag, tol
    again = r.run(r.x)
    assert all(torch.equal(got[m], again[m]) for m in got)


@pytest.mark.parametrize("case", [c for c in R.CASES if "dw_router" in c[6]], ids=name)
def test_matrix_gradient_has_every_bit_of_dl(case):
    """Each column of x has one token, a power of two: its row of the matrix' gradient is that token's dL (as the same
    call returns it) times the power of two, bit for bit, however the products split the 24 bits."""
    r = Problem(*case)
    c = torch.arange(r.d, device=DEV)
    t = (c * 7919 + 13) % r.T
    s = 2.0 ** ((c * 5) % 17 - 8).float() * (1.0 - 2.0 * (c % 2))
    x = torch.zeros(r.T, r.d, device=DEV)
    x[t, c] = s
    x[~r.keep] = float("nan")
    got = r.run(x.to(ACT[r.act]))
    dl = got["dlogits"]
    top = dl.bfloat16().float()
    rest = (dl - top) - (dl - top).bfloat16().float()
    # two planes would not do (where a token is kept)
    assert (rest != 0).any() or not r.keep.any() or r.E == 1
    assert torch.equal(got["dw_router"], dl[t] * s[:, None])
