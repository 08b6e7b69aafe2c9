"""The layer for a few tokens on the host side: argument checks (no call here
reaches a kernel launch) and the binding's tensor checks."""
import ctypes
import os

import pytest
import torch

from mixture_experts_layer_15_amd import binding as B

FAKE = 0x1000  # never dereferenced: the calls below fail their host checks
BIG = 1 << 40
FULL = dict(x=FAKE, w_router=FAKE, router_bias=FAKE, w_gate=FAKE, w_up=FAKE, w_down=FAKE, s_gate=FAKE, s_up=FAKE, s_down=FAKE,
            out=2 * FAKE, logits=3 * FAKE, topk_idx=4 * FAKE, topk_w=5 * FAKE)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from mixture_experts_layer_15_amd import build
        build.build()
    return B.load_library()


def _p(**kw):
    base = dict(T=4, d=256, E=8, k=2, F=256, expert_begin=0, num_local=8, act="bf16", weight="fp8")
    base.update(kw)
    return B.problem(**base)


def _call(lib, p=None, ws=FAKE, nbytes=BIG, **kw):
    a = B.ForwardArgs(**{**FULL, **kw})
    return lib.moe_forward_few(ctypes.byref(p or _p()), ctypes.byref(a), ws, nbytes, None)


def test_limits_match_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "moe.h")).read()
    assert f"#define MOE_FEW_MAX_TOKENS {B.MOE_FEW_MAX_TOKENS}\n" in text
    assert f"#define MOE_FEW_MAX_SLOTS {B.MOE_FEW_MAX_SLOTS}\n" in text


def test_refusals(lib):
    assert lib.moe_forward_few(ctypes.byref(_p()), None, FAKE, BIG, None) == B.MOE_ERR_INVALID_ARGUMENT
    for name in ("x", "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down", "out"):
        assert _call(lib, **{name: None}) == B.MOE_ERR_INVALID_ARGUMENT, name
    assert _call(lib, w_router=None, logits=None) == B.MOE_ERR_INVALID_ARGUMENT
    for name in FULL:
        assert _call(lib, **{name: FULL[name] + 4}) == B.MOE_ERR_INVALID_ARGUMENT, name
    for name in ("counts", "offsets", "sorted_slot", "slot_pos", "events"):
        assert _call(lib, **{name: FAKE}) == B.MOE_ERR_INVALID_ARGUMENT, name
    assert _call(lib, out=FAKE) == _call(lib, topk_w=3 * FAKE) == B.MOE_ERR_INVALID_ARGUMENT   # aliases
    assert _call(lib, ws=FAKE + 8) == B.MOE_ERR_INVALID_ARGUMENT
    assert _call(lib, _p(d=100)) == _call(lib, _p(k=9)) == B.MOE_ERR_INVALID_ARGUMENT
    for kw in (dict(T=17), dict(T=16, E=64, num_local=64, k=17), dict(T=2, E=512, num_local=512, k=129), dict(act="f32")):
        assert _call(lib, _p(**kw)) == B.MOE_ERR_UNSUPPORTED, kw
        assert B.moe_workspace_size(_p(**kw), B.MOE_CALL_FORWARD_FEW) == 0


def test_workspace_and_no_tokens(lib):
    for kw in (dict(T=0), dict(T=1), dict(T=16), dict(T=1, E=512, num_local=512, k=256), dict(T=16, E=512, num_local=512, k=16)):
        need = B.moe_workspace_size(_p(**kw), B.MOE_CALL_FORWARD_FEW)
        assert need > 0 and need % 256 == 0
        assert _call(lib, _p(**kw), nbytes=need - 1) == B.MOE_ERR_WORKSPACE_TOO_SMALL
        assert _call(lib, _p(**kw), ws=None) == B.MOE_ERR_WORKSPACE_TOO_SMALL
    assert _call(lib, _p(T=0), x=None, out=None, logits=None) == B.MOE_OK


def test_binding_checks_tensors(lib):
    p = _p(weight="bf16", d=128, F=128)
    bf = torch.bfloat16
    ok = dict(x=torch.zeros(4, 128, dtype=bf), w_router=torch.zeros(128, 8, dtype=bf), w_gate=torch.zeros(8, 128, 128, dtype=bf),
              w_up=torch.zeros(8, 128, 128, dtype=bf), w_down=torch.zeros(8, 128, 128, dtype=bf), out=torch.zeros(4, 128, dtype=bf))
    for bad in (dict(x=ok["x"].float()), dict(x=ok["x"][:3]), dict(w_gate=ok["w_gate"][:7]), dict(w_up=ok["w_up"].transpose(1, 2)),
                dict(topk_idx=torch.zeros(8)), dict(logits=torch.zeros(4, 7)), dict(router_bias=torch.zeros(9))):
        with pytest.raises(B.MoEError):
            B.moe_forward_few(p, ws=None, **{**ok, **bad})
