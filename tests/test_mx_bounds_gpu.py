"""The 4-bit expert network with segment bounds that do not ascend: nothing but
y and the workspace is written, and the next call is as before."""
import pytest
import torch

from mixture_experts_layer_15_amd import binding as B
from test_mx_gpu import DEV, _convert, _dispatch, _gen, _ids, _packed, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


# tokens, columns, experts, slots, features, blocked: in tiles and streamed
@pytest.mark.parametrize("T,d,E,k,F,blocked", [(2048, 256, 4, 2, 256, False), (2048, 256, 4, 2, 256, True), (100, 384, 7, 3, 640, False),
                                               (500, 256, 64, 2, 384, True), (3, 128, 512, 4, 128, True), (640, 128, 512, 8, 128, True)])
def test_bounds_that_do_not_ascend(T, d, E, k, F, blocked):
    g = _gen(T + E)
    p = B.problem(T, d, E, k, F, 0, E, "bf16", "mxfp4", blocked)
    w = _weights(E, F, d, g)
    kept = _packed(p, w) if blocked else w
    offsets, order = _dispatch(p, _ids(T, E, k, g, 0.0))
    S = T * k
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    codes, scales = _convert(x[None], B.MOE_MX_SCALES_ROW)
    gates = torch.rand(S, generator=g, device=DEV)
    need = B.moe_workspace_size(p, B.MOE_CALL_EXPERT_FFN_MX)
    # a guard behind the workspace that would hold the groups of every expert at its fullest
    guard = E * (S + 256) * (F // 2 + F // 32) if E <= 64 else 64 << 20
    ws = torch.full((need + guard,), 0xA5, dtype=torch.uint8, device=DEV)
    y = torch.full((S + 64, d), 7.0, dtype=torch.bfloat16, device=DEV)

    def run(off):
        y.fill_(7.0)
        B.moe_expert_ffn_mx(p, codes.contiguous(), scales.contiguous(), order, off, kept["w_gate"], kept["w_up"], kept["w_down"],
                            w["s_gate"], w["s_up"], w["s_down"], gates, y[:S], ws[:need])
        torch.cuda.synchronize()
        assert (ws[need:] == 0xA5).all() and (y[S:] == 7.0).all()
        return y.clone()

    good = run(offsets)
    e = torch.arange(E + 1, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    for off in ((e % 2) * S, S - (e % 2) * S, torch.full_like(e, S), torch.randint(-2 ** 31, 2 ** 31 - 1, (E + 1,), generator=g, **i32),
                torch.randint(0, S + 1, (E + 1,), generator=g, **i32)):
        run(off.to(torch.int32).contiguous())
    assert torch.equal(run(offsets), good)
