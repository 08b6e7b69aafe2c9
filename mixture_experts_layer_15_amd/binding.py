"""Thin ctypes binding of the C ABI in ``include/moe.h``.

Argument marshalling: tensors become device pointers, the stream becomes the
current HIP stream, status codes become exceptions (the calls for training the
router, for the norms, for a few tokens and in 4 bits check their tensors too).
Every step of the layer runs in the HIP library; there is no fallback of any kind.  PyTorch is
used for device memory and streams.
"""
from __future__ import annotations

import ctypes
import itertools
import os
import struct
from typing import Optional

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("MOE_MI355X_LIB", os.path.join(PKG, "libmoe_mi355x.so"))

MOE_OK, MOE_ERR_INVALID_ARGUMENT, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_HIP = range(5)
MOE_F32, MOE_BF16, MOE_FP8_E4M3, MOE_MXFP4 = range(4)
MOE_CALL_PERMUTE, MOE_CALL_EXPERT_FFN, MOE_CALL_FORWARD, MOE_CALL_ROUTE = range(4)
MOE_CALL_BALANCE_LOSS, MOE_CALL_ROUTE_BACKWARD = 4, 5
MOE_CALL_NORM_BACKWARD, MOE_CALL_COMBINE_NORM_BACKWARD = 6, 7
MOE_CALL_EXPERT_FFN_MX, MOE_CALL_FORWARD_FEW = 8, 9
MOE_FEW_MAX_TOKENS, MOE_FEW_MAX_SLOTS = 16, 256   # include/moe.h
MOE_MX_SCALES_ROW, MOE_MX_SCALES_BLOCK = range(2)
MOE_GRAD_MAX_TENSORS = 4096   # include/moe.h
MOE_FORWARD_EVENTS = 7
MOE_LAYOUT_ROWS, MOE_LAYOUT_BLOCKED = range(2)
MOE_NOALLOC_SCRATCH_BYTES = 64 << 20   # include/moe.h

FMT = {"f32": MOE_F32, "bf16": MOE_BF16, "fp8": MOE_FP8_E4M3, "mxfp4": MOE_MXFP4}


class MoEError(RuntimeError):
    def __init__(self, call: str, status: int, text: str):
        super().__init__(f"{call} failed: {text} ({status})")
        self.status = status


class Problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "d", "E", "k", "F", "expert_begin", "num_local", "act", "weight",
                 "weight_layout")]


class ForwardArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("x", "w_router", "router_bias", "w_gate", "w_up", "w_down", "s_gate", "s_up",
                 "s_down", "out", "logits", "topk_idx", "topk_w", "counts", "offsets",
                 "sorted_slot", "slot_pos", "events")]


class RouteBackwardArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("x", "w_router", "logits", "topk_idx", "topk_w", "dtopk_w", "token_mask",
                 "counts", "n_tokens", "dlosses", "dlogits", "dx", "dw_router", "dbias")]


class NormBackwardArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("dx", "h", "weight", "rstd", "dout", "dh", "dweight")] + [("res_scale", ctypes.c_float)]


class CombineNormArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("y", "slot_pos", "topk_w", "h", "weight", "gate", "out", "rstd", "next_weight",
                 "next_x", "next_rstd")] + [("eps", ctypes.c_float), ("res_scale", ctypes.c_float)]


class CombineNormBackwardArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("dout", "y", "slot_pos", "topk_w", "weight", "rstd", "gate", "dy", "dtopk_w",
                 "dweight", "dgate")]


_GRAD = "PPqi4x"   # moe_grad_t
_GRAD_CODE = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}

_lib = None


def load_library() -> ctypes.CDLL:
    """Load the built library; raise if it is missing (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it first with "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    P = ctypes.POINTER(Problem)
    lib.moe_workspace_size.argtypes = [P, i32]
    lib.moe_workspace_size.restype = sz
    lib.moe_status_string.argtypes = [ctypes.c_int]
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_route.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_permute.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_expert_ffn.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_combine.argtypes = [P, vp, vp, vp, vp, vp]
    lib.moe_forward.argtypes = [P, ctypes.POINTER(ForwardArgs), vp, sz, vp]
    lib.moe_forward_noalloc.argtypes = [P, ctypes.POINTER(ForwardArgs), vp]
    i64p, i32p, f64p = (ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int32),
                        ctypes.POINTER(ctypes.c_double))
    lib.moe_eplb_plan.argtypes = [i64p, i32, i32, i32, i32p, i32p, i32p, f64p]
    lib.moe_eplb_remap.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp]
    lib.moe_pack_weights.argtypes = [P, i32, vp, vp, vp]
    lib.moe_balance_loss.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_route_backward.argtypes = [P, ctypes.POINTER(RouteBackwardArgs), vp, sz, vp]
    lib.moe_combine_backward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp]
    lib.moe_grad_workspace_size.argtypes = [vp, i32]
    lib.moe_grad_workspace_size.restype = sz
    lib.moe_grad_norm.argtypes = [vp, i32, vp, vp, sz, vp]
    lib.moe_grad_clip.argtypes = [vp, i32, vp, ctypes.c_float, vp]
    lib.moe_norm.argtypes = [P, vp, vp, ctypes.c_float, vp, vp, vp]
    lib.moe_norm_backward.argtypes = [P, ctypes.POINTER(NormBackwardArgs), vp, sz, vp]
    lib.moe_combine_norm.argtypes = [P, ctypes.POINTER(CombineNormArgs), vp]
    lib.moe_combine_norm_backward.argtypes = [P, ctypes.POINTER(CombineNormBackwardArgs), vp, sz, vp]
    lib.moe_forward_few.argtypes = [P, ctypes.POINTER(ForwardArgs), vp, sz, vp]
    lib.moe_mx_quantize.argtypes = [i32, i32, i32, i32, vp, vp, vp, i32, vp]
    lib.moe_mx_dequantize.argtypes = [i32, i32, i32, i32, vp, vp, vp, i32, vp]
    lib.moe_expert_ffn_mx.argtypes = [P] + [vp] * 13 + [sz, vp]
    for f in ("moe_route", "moe_permute", "moe_expert_ffn", "moe_combine", "moe_forward",
              "moe_forward_noalloc", "moe_eplb_plan", "moe_eplb_remap", "moe_pack_weights",
              "moe_balance_loss", "moe_route_backward", "moe_combine_backward", "moe_grad_norm",
              "moe_grad_clip", "moe_norm", "moe_norm_backward", "moe_combine_norm",
              "moe_combine_norm_backward", "moe_mx_quantize", "moe_mx_dequantize",
              "moe_expert_ffn_mx", "moe_forward_few"):
        getattr(lib, f).restype = ctypes.c_int
    _lib = lib
    return lib


def problem(T, d, E, k, F, expert_begin=0, num_local=None, act="bf16", weight="bf16",
            blocked=False) -> Problem:
    num_local = E - expert_begin if num_local is None else num_local
    return Problem(T, d, E, k, F, expert_begin, num_local,
                   FMT[act] if isinstance(act, str) else act,
                   FMT[weight] if isinstance(weight, str) else weight,
                   MOE_LAYOUT_BLOCKED if blocked else MOE_LAYOUT_ROWS)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(call: str, status: int) -> None:
    if status != MOE_OK:
        text = load_library().moe_status_string(status).decode()
        raise MoEError(call, status, text)


def moe_status_string(status: int) -> str:
    return load_library().moe_status_string(status).decode()


def moe_workspace_size(p: Problem, call: int) -> int:
    return int(load_library().moe_workspace_size(ctypes.byref(p), call))


def moe_route(p, x, w_router, router_bias, logits, topk_idx, topk_w, ws=None,
              stream=None) -> None:
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = load_library().moe_route(ctypes.byref(p), _ptr(x), _ptr(w_router), _ptr(router_bias),
                                  _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _ptr(ws), nbytes,
                                  _stream(stream))
    _check("moe_route", st)


def moe_permute(p, topk_idx, counts, offsets, sorted_slot, slot_pos, ws, stream=None) -> None:
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = load_library().moe_permute(ctypes.byref(p), _ptr(topk_idx), _ptr(counts), _ptr(offsets),
                                    _ptr(sorted_slot), _ptr(slot_pos), _ptr(ws), nbytes,
                                    _stream(stream))
    _check("moe_permute", st)


def moe_expert_ffn(p, x, sorted_slot, offsets, w_gate, w_up, w_down, s_gate, s_up, s_down,
                   topk_w, y, ws, stream=None) -> None:
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = load_library().moe_expert_ffn(
        ctypes.byref(p), _ptr(x), _ptr(sorted_slot), _ptr(offsets), _ptr(w_gate), _ptr(w_up),
        _ptr(w_down), _ptr(s_gate), _ptr(s_up), _ptr(s_down), _ptr(topk_w), _ptr(y), _ptr(ws),
        nbytes, _stream(stream))
    _check("moe_expert_ffn", st)


def moe_combine(p, y, slot_pos, topk_w, out, stream=None) -> None:
    st = load_library().moe_combine(ctypes.byref(p), _ptr(y), _ptr(slot_pos), _ptr(topk_w),
                                    _ptr(out), _stream(stream))
    _check("moe_combine", st)


def moe_forward(p, *, x, w_router, router_bias, w_gate, w_up, w_down, out, ws,
                s_gate=None, s_up=None, s_down=None, logits=None, topk_idx=None, topk_w=None,
                counts=None, offsets=None, sorted_slot=None, slot_pos=None, events=None,
                stream=None) -> None:
    """``events``: None, or a ctypes array of MOE_FORWARD_EVENTS hipEvent_t handles."""
    a = _forward_args(x, w_router, router_bias, w_gate, w_up, w_down, out, s_gate, s_up, s_down,
                      logits, topk_idx, topk_w, counts, offsets, sorted_slot, slot_pos, events)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = load_library().moe_forward(ctypes.byref(p), ctypes.byref(a), _ptr(ws), nbytes,
                                    _stream(stream))
    _check("moe_forward", st)


def _forward_args(x, w_router, router_bias, w_gate, w_up, w_down, out, s_gate, s_up, s_down,
                  logits, topk_idx, topk_w, counts, offsets, sorted_slot, slot_pos, events):
    return ForwardArgs(_ptr(x), _ptr(w_router), _ptr(router_bias), _ptr(w_gate), _ptr(w_up),
                       _ptr(w_down), _ptr(s_gate), _ptr(s_up), _ptr(s_down), _ptr(out),
                       _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(offsets),
                       _ptr(sorted_slot), _ptr(slot_pos),
                       None if events is None else ctypes.addressof(events))


def moe_forward_noalloc(p, *, x, w_router, router_bias, w_gate, w_up, w_down, out,
                        s_gate=None, s_up=None, s_down=None, logits=None, topk_idx=None,
                        topk_w=None, counts=None, offsets=None, sorted_slot=None, slot_pos=None,
                        events=None, stream=None) -> None:
    """moe_forward with the library's own scratch array (no workspace argument)."""
    a = _forward_args(x, w_router, router_bias, w_gate, w_up, w_down, out, s_gate, s_up, s_down,
                      logits, topk_idx, topk_w, counts, offsets, sorted_slot, slot_pos, events)
    st = load_library().moe_forward_noalloc(ctypes.byref(p), ctypes.byref(a), _stream(stream))
    _check("moe_forward_noalloc", st)


def moe_eplb_plan(load, G: int, R: int):
    """Host placement plan (see moe.h).  ``load``: per-expert counts (any
    integer sequence).  Returns numpy ``(replicas [E], phys_to_log [E+R],
    log_to_phys [E, G], rank_load [G])``."""
    import numpy as np
    ld = np.ascontiguousarray(np.asarray(load, dtype=np.int64))
    E = int(ld.shape[0])
    rep = np.zeros(E, dtype=np.int32)
    p2l = np.zeros(max(E + R, 1), dtype=np.int32)
    l2p = np.zeros((E, max(G, 1)), dtype=np.int32)
    rl = np.zeros(max(G, 1), dtype=np.float64)
    c = ctypes
    st = load_library().moe_eplb_plan(
        ld.ctypes.data_as(c.POINTER(c.c_int64)), E, G, R,
        rep.ctypes.data_as(c.POINTER(c.c_int32)), p2l.ctypes.data_as(c.POINTER(c.c_int32)),
        l2p.ctypes.data_as(c.POINTER(c.c_int32)), rl.ctypes.data_as(c.POINTER(c.c_double)))
    _check("moe_eplb_plan", st)
    return rep, p2l, l2p, rl


def moe_eplb_remap(T, k, E, G, topk_idx, replicas, log_to_phys, topk_phys, stream=None) -> None:
    st = load_library().moe_eplb_remap(T, k, E, G, _ptr(topk_idx), _ptr(replicas),
                                       _ptr(log_to_phys), _ptr(topk_phys), _stream(stream))
    _check("moe_eplb_remap", st)


def moe_pack_weights(p, which: int, src, dst, stream=None) -> None:
    """Blocked layout of one expert matrix set (which 0: gate or up, 1: down)."""
    st = load_library().moe_pack_weights(ctypes.byref(p), which, _ptr(src), _ptr(dst),
                                         _stream(stream))
    _check("moe_pack_weights", st)


# ---- router training
#
# These calls check the tensors they are given (type, size, contiguity, the
# current device), since a gradient of another layout would be read wrongly
# without an error; integers pass as device addresses, unchecked.

def _refuse(call: str, text: str):
    raise MoEError(call, MOE_ERR_INVALID_ARGUMENT, text)


def _arg(call: str, name: str, t, dtype, numel: int, device: int) -> Optional[int]:
    if t is None or type(t) is int:
        return t
    if t.dtype is dtype and t.numel() == numel and t.is_contiguous() and t.get_device() == device:
        return t.data_ptr()
    if t.dtype is not dtype:
        _refuse(call, f"{name} is {t.dtype}, not {dtype}")
    if t.numel() != numel:
        _refuse(call, f"{name} has {t.numel()} values, not {numel}")
    if not t.is_contiguous():
        _refuse(call, f"{name} is not contiguous")
    _refuse(call, f"{name} is on {t.device}, not on the current device")


def _ws_arg(call: str, ws, device: int):
    if ws is None:
        return None, 0
    if not ws.is_contiguous() or ws.get_device() != device:
        _refuse(call, "ws is not a contiguous tensor of the current device")
    return ws.data_ptr(), ws.numel() * ws.element_size()


_gpu = None


def _current(call: str, stream):
    """(device, stream handle) of a call; device -1 without a GPU."""
    global _gpu
    if _gpu is None:
        _gpu = torch.cuda.is_available()
    device = torch.cuda.current_device() if _gpu else -1
    if stream is None:
        # the handle alone: building a torch.cuda.Stream for it takes 2.8 us
        return device, torch._C._cuda_getCurrentRawStream(device) if _gpu else None
    if isinstance(stream, int):
        return device, stream
    if stream.device.index != device:
        _refuse(call, f"the stream is one of {stream.device}, not of the current device")
    return device, stream.cuda_stream


_ACT_DTYPE = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16}


def _act(call: str, p: Problem):
    if p.act not in _ACT_DTYPE:
        raise MoEError(call, MOE_ERR_UNSUPPORTED, "activations are f32 or bf16")
    return _ACT_DTYPE[p.act]


def _mask_arg(call: str, mask, T: int, device: int):
    dtype = torch.uint8
    if isinstance(mask, torch.Tensor) and mask.dtype is torch.bool:
        dtype = torch.bool   # one byte, 0 or 1
    return _arg(call, "token_mask", mask, dtype, T, device)


def moe_balance_loss(p, logits, topk_idx, token_mask, counts, n_tokens, prob_mean, losses, ws,
                     stream=None) -> None:
    """Balance and z loss over the router's softmax, and per-expert counts (see moe.h).
    ``token_mask``: uint8 or bool [T], or None."""
    c = "moe_balance_loss"
    dev, st = _current(c, stream)
    f32, i32 = torch.float32, torch.int32
    wp, wn = _ws_arg(c, ws, dev)
    _check(c, load_library().moe_balance_loss(
        ctypes.byref(p), _arg(c, "logits", logits, f32, p.T * p.E, dev),
        _arg(c, "topk_idx", topk_idx, i32, p.T * p.k, dev), _mask_arg(c, token_mask, p.T, dev),
        _arg(c, "counts", counts, i32, p.E, dev), _arg(c, "n_tokens", n_tokens, i32, 1, dev),
        _arg(c, "prob_mean", prob_mean, f32, p.E, dev), _arg(c, "losses", losses, f32, 2, dev),
        wp, wn, st))


def moe_route_backward(p, *, ws, x=None, w_router=None, logits=None, topk_idx=None, topk_w=None,
                       dtopk_w=None, token_mask=None, counts=None, n_tokens=None, dlosses=None,
                       dlogits=None, dx=None, dw_router=None, dbias=None, stream=None) -> None:
    """Gradient of the router from that of its gates and of the balance losses (see moe.h)."""
    c = "moe_route_backward"
    dev, st = _current(c, stream)
    f32, i32, act = torch.float32, torch.int32, _act(c, p)
    S = p.T * p.k
    a = RouteBackwardArgs(
        _arg(c, "x", x, act, p.T * p.d, dev), _arg(c, "w_router", w_router, act, p.d * p.E, dev),
        _arg(c, "logits", logits, f32, p.T * p.E, dev), _arg(c, "topk_idx", topk_idx, i32, S, dev),
        _arg(c, "topk_w", topk_w, f32, S, dev), _arg(c, "dtopk_w", dtopk_w, f32, S, dev),
        _mask_arg(c, token_mask, p.T, dev), _arg(c, "counts", counts, i32, p.E, dev),
        _arg(c, "n_tokens", n_tokens, i32, 1, dev), _arg(c, "dlosses", dlosses, f32, 2, dev),
        _arg(c, "dlogits", dlogits, f32, p.T * p.E, dev), _arg(c, "dx", dx, act, p.T * p.d, dev),
        _arg(c, "dw_router", dw_router, f32, p.d * p.E, dev),
        _arg(c, "dbias", dbias, f32, p.E, dev))
    wp, wn = _ws_arg(c, ws, dev)
    _check(c, load_library().moe_route_backward(ctypes.byref(p), ctypes.byref(a), wp, wn, st))


def moe_combine_backward(p, dout, y, slot_pos, topk_w, dy, dtopk_w, stream=None) -> None:
    """Gradients of the expert rows and the gates from that of the layer's output (see moe.h)."""
    c = "moe_combine_backward"
    dev, st = _current(c, stream)
    f32, act = torch.float32, _act(c, p)
    S = p.T * p.k
    _check(c, load_library().moe_combine_backward(
        ctypes.byref(p), _arg(c, "dout", dout, act, p.T * p.d, dev),
        _arg(c, "y", y, act, S * p.d, dev), _arg(c, "slot_pos", slot_pos, torch.int32, S, dev),
        _arg(c, "topk_w", topk_w, f32, S, dev), _arg(c, "dy", dy, act, S * p.d, dev),
        _arg(c, "dtopk_w", dtopk_w, f32, S, dev), st))


class GradList:
    """The host array of ``moe_grad_t`` for a list of gradient tensors, and the tensors
    themselves, so that their memory lives as long as the list."""

    def __init__(self, grads, out=None):
        c = "grad_list"
        grads = list(grads)
        out = grads if out is None else list(out)
        if len(out) != len(grads):
            _refuse(c, f"{len(out)} outputs for {len(grads)} gradients")
        T = torch.Tensor   # (maps over the methods: a list of 100 tensors takes 50 us)
        codes = list(map(_GRAD_CODE.get, [g.dtype for g in grads]))
        if None in codes:
            raise MoEError(c, MOE_ERR_UNSUPPORTED,
                           f"a gradient is {grads[codes.index(None)].dtype}, not float32 or bfloat16")
        sizes = list(map(T.numel, grads))
        devices = set(map(T.get_device, grads))
        if not all(map(T.is_contiguous, grads)):
            _refuse(c, "a gradient is not contiguous")
        if len(devices) > 1:
            _refuse(c, "the gradients are on more than one device")
        self.device = devices.pop() if devices else None
        at = list(map(T.data_ptr, grads))
        to = at
        if out is not grads:
            if (list(map(_GRAD_CODE.get, [o.dtype for o in out])) != codes
                    or list(map(T.numel, out)) != sizes or not all(map(T.is_contiguous, out))
                    or not set(map(T.get_device, out)) <= {self.device}):
                _refuse(c, "an output has another type, size, layout or device than its gradient")
            to = list(map(T.data_ptr, out))
        flat = itertools.chain.from_iterable(zip(at, to, sizes, codes))
        self.n = len(grads)
        self.tensors = (grads, out)
        self.array = struct.pack(_GRAD * self.n, *flat)


def grad_list(grads, out=None) -> GradList:
    """The gradients that moe_grad_norm and moe_grad_clip work on; ``out``: where clipping
    writes (default: in place).  A program keeps it as long as the tensors stay."""
    return GradList(grads, out)


def _grads(call: str, grads, device: int) -> GradList:
    if not isinstance(grads, GradList):
        grads = GradList(grads)
    if grads.n and device >= 0 and grads.device != device:
        _refuse(call, "the gradients are not on the current device")
    return grads


def moe_grad_workspace_size(grads) -> int:
    g = grads if isinstance(grads, GradList) else GradList(grads)
    return int(load_library().moe_grad_workspace_size(g.array, g.n))


def moe_grad_norm(grads, norm, ws, stream=None) -> None:
    """Global L2 norm of a list of gradients (a sequence of tensors or a ``grad_list``)."""
    c = "moe_grad_norm"
    dev, st = _current(c, stream)
    g = _grads(c, grads, dev)
    wp, wn = _ws_arg(c, ws, dev)
    _check(c, load_library().moe_grad_norm(g.array, g.n, _arg(c, "norm", norm, torch.float32, 1, dev),
                                           wp, wn, st))


def moe_grad_clip(grads, norm, max_norm: float, stream=None) -> None:
    """Gradients scaled so that a global norm above ``max_norm`` becomes ``max_norm``."""
    c = "moe_grad_clip"
    dev, st = _current(c, stream)
    g = _grads(c, grads, dev)
    _check(c, load_library().moe_grad_clip(g.array, g.n, _arg(c, "norm", norm, torch.float32, 1, dev),
                                           max_norm, st))


# ---- norms around the layer (tensors checked as above)

def moe_norm(p, h, weight, eps: float, x, rstd=None, stream=None) -> None:
    """The norm before the layer: x = h r weight, r into ``rstd`` (see moe.h)."""
    c = "moe_norm"
    dev, st = _current(c, stream)
    f32, act, n = torch.float32, _act(c, p), p.T * p.d
    _check(c, load_library().moe_norm(
        ctypes.byref(p), _arg(c, "h", h, act, n, dev), _arg(c, "weight", weight, f32, p.d, dev), eps,
        _arg(c, "x", x, act, n, dev), _arg(c, "rstd", rstd, f32, p.T, dev), st))


def moe_norm_backward(p, *, dx, h, weight, rstd, ws, dout=None, res_scale: float = 1.0, dh=None,
                      dweight=None, stream=None) -> None:
    """Gradient of the norm before the layer, joined to ``res_scale * dout`` (see moe.h)."""
    c = "moe_norm_backward"
    dev, st = _current(c, stream)
    f32, act, n = torch.float32, _act(c, p), p.T * p.d
    a = NormBackwardArgs(
        _arg(c, "dx", dx, act, n, dev), _arg(c, "h", h, act, n, dev),
        _arg(c, "weight", weight, f32, p.d, dev), _arg(c, "rstd", rstd, f32, p.T, dev),
        _arg(c, "dout", dout, act, n, dev), _arg(c, "dh", dh, act, n, dev),
        _arg(c, "dweight", dweight, f32, p.d, dev), res_scale)
    wp, wn = _ws_arg(c, ws, dev)
    _check(c, load_library().moe_norm_backward(ctypes.byref(p), ctypes.byref(a), wp, wn, st))


def moe_combine_norm(p, *, y, h, weight, eps: float, out, slot_pos=None, topk_w=None, gate=None,
                     res_scale: float = 1.0, rstd=None, next_weight=None, next_x=None,
                     next_rstd=None, stream=None) -> None:
    """Combine, norm, gate and residual after the layer, and the next block's norm (see moe.h)."""
    c = "moe_combine_norm"
    dev, st = _current(c, stream)
    f32, act, n, S = torch.float32, _act(c, p), p.T * p.d, p.T * p.k
    a = CombineNormArgs(
        _arg(c, "y", y, act, S * p.d, dev), _arg(c, "slot_pos", slot_pos, torch.int32, S, dev),
        _arg(c, "topk_w", topk_w, f32, S, dev), _arg(c, "h", h, act, n, dev),
        _arg(c, "weight", weight, f32, p.d, dev), _arg(c, "gate", gate, f32, p.d, dev),
        _arg(c, "out", out, act, n, dev), _arg(c, "rstd", rstd, f32, p.T, dev),
        _arg(c, "next_weight", next_weight, f32, p.d, dev), _arg(c, "next_x", next_x, act, n, dev),
        _arg(c, "next_rstd", next_rstd, f32, p.T, dev), eps, res_scale)
    _check(c, load_library().moe_combine_norm(ctypes.byref(p), ctypes.byref(a), st))


def moe_combine_norm_backward(p, *, dout, y, weight, rstd, ws, slot_pos=None, topk_w=None, gate=None,
                              dy=None, dtopk_w=None, dweight=None, dgate=None, stream=None) -> None:
    """Gradients of the expert rows, the gates, the norm's weight and the channel gate (see moe.h)."""
    c = "moe_combine_norm_backward"
    dev, st = _current(c, stream)
    f32, act, n, S = torch.float32, _act(c, p), p.T * p.d, p.T * p.k
    a = CombineNormBackwardArgs(
        _arg(c, "dout", dout, act, n, dev), _arg(c, "y", y, act, S * p.d, dev),
        _arg(c, "slot_pos", slot_pos, torch.int32, S, dev), _arg(c, "topk_w", topk_w, f32, S, dev),
        _arg(c, "weight", weight, f32, p.d, dev), _arg(c, "rstd", rstd, f32, p.T, dev),
        _arg(c, "gate", gate, f32, p.d, dev), _arg(c, "dy", dy, act, S * p.d, dev),
        _arg(c, "dtopk_w", dtopk_w, f32, S, dev), _arg(c, "dweight", dweight, f32, p.d, dev),
        _arg(c, "dgate", dgate, f32, p.d, dev))
    wp, wn = _ws_arg(c, ws, dev)
    _check(c, load_library().moe_combine_norm_backward(ctypes.byref(p), ctypes.byref(a), wp, wn, st))


# ---- the layer for a few tokens (tensors checked as above)

_WEIGHT_DTYPE = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16}


def _weight_arg(call: str, name: str, w, p: Problem, device: int):
    n = p.num_local * p.F * p.d
    if p.weight in _WEIGHT_DTYPE:
        return _arg(call, name, w, _WEIGHT_DTYPE[p.weight], n, device)
    # FP8 codes as bytes or as torch's type
    dtype = torch.uint8
    if isinstance(w, torch.Tensor) and p.weight == MOE_FP8_E4M3 and w.dtype is torch.float8_e4m3fn:
        dtype = w.dtype
    return _arg(call, name, w, dtype, n if p.weight == MOE_FP8_E4M3 else n // 2, device)


def moe_forward_few(p, *, x, w_router, w_gate, w_up, w_down, out, ws, router_bias=None, s_gate=None,
                    s_up=None, s_down=None, logits=None, topk_idx=None, topk_w=None, stream=None) -> None:
    """The whole layer for at most 16 tokens, in two kernels (see moe.h)."""
    c = "moe_forward_few"
    dev, st = _current(c, stream)
    f32, act, n, S, El = torch.float32, _act(c, p), p.T * p.d, p.T * p.k, p.num_local
    scale = {}
    for name, s in (("s_gate", s_gate), ("s_up", s_up), ("s_down", s_down)):
        if p.weight == MOE_FP8_E4M3:
            scale[name] = _arg(c, name, s, f32, El * (p.F // 128) * (p.d // 128), dev)
        elif p.weight == MOE_MXFP4:
            scale[name] = _arg(c, name, s, torch.uint8, El * p.F * p.d // 32, dev)
    a = ForwardArgs(
        x=_arg(c, "x", x, act, n, dev), w_router=_arg(c, "w_router", w_router, act, p.d * p.E, dev),
        router_bias=_arg(c, "router_bias", router_bias, f32, p.E, dev),
        w_gate=_weight_arg(c, "w_gate", w_gate, p, dev), w_up=_weight_arg(c, "w_up", w_up, p, dev),
        w_down=_weight_arg(c, "w_down", w_down, p, dev), out=_arg(c, "out", out, act, n, dev),
        logits=_arg(c, "logits", logits, f32, p.T * p.E, dev),
        topk_idx=_arg(c, "topk_idx", topk_idx, torch.int32, S, dev),
        topk_w=_arg(c, "topk_w", topk_w, f32, S, dev), **scale)
    wp, wn = _ws_arg(c, ws, dev)
    _check(c, load_library().moe_forward_few(ctypes.byref(p), ctypes.byref(a), wp, wn, st))


# ---- 4-bit activations (tensors checked as above)

def _convert(call: str, values, codes, scales, layout: int, stream):
    dev, st = _current(call, stream)
    if values.dim() < 2 or values.shape[-1] == 0 or values.shape[-1] % 32:
        _refuse(call, f"values of shape {tuple(values.shape)}: at least two dimensions, the last a multiple of 32")
    if values.dtype not in _GRAD_CODE:
        raise MoEError(call, MOE_ERR_UNSUPPORTED, f"values are {values.dtype}, not float32 or bfloat16")
    rows, cols = values.shape[-2:]
    n = values.numel()
    batch = n // (rows * cols) if n else 0
    return (batch, rows, cols, _GRAD_CODE[values.dtype], _arg(call, "values", values, values.dtype, n, dev),
            _arg(call, "codes", codes, torch.uint8, n // 2, dev),
            _arg(call, "scales", scales, torch.uint8, n // 32, dev), layout, st)


def moe_mx_quantize(values, codes, scales, layout: int = MOE_MX_SCALES_ROW, stream=None) -> None:
    """MXFP4 codes and scales of ``values`` [..., rows, cols] (see moe.h)."""
    c = "moe_mx_quantize"
    b, r, n, t, v, q, s, layout, st = _convert(c, values, codes, scales, layout, stream)
    _check(c, load_library().moe_mx_quantize(b, r, n, t, v, q, s, layout, st))


def moe_mx_dequantize(codes, scales, values, layout: int = MOE_MX_SCALES_ROW, stream=None) -> None:
    """The values [..., rows, cols] that MXFP4 codes and scales stand for (see moe.h)."""
    c = "moe_mx_dequantize"
    b, r, n, t, v, q, s, layout, st = _convert(c, values, codes, scales, layout, stream)
    _check(c, load_library().moe_mx_dequantize(b, r, n, t, q, s, v, layout, st))


def moe_expert_ffn_mx(p, x_codes, x_scales, sorted_slot, offsets, w_gate, w_up, w_down, s_gate, s_up,
                      s_down, topk_w, y, ws, stream=None) -> None:
    """The expert network on 4-bit activations and weights (see moe.h)."""
    c = "moe_expert_ffn_mx"
    dev, st = _current(c, stream)
    u8, i32, S, W = torch.uint8, torch.int32, p.T * p.k, p.num_local * p.F * p.d
    wp, wn = _ws_arg(c, ws, dev)
    _check(c, load_library().moe_expert_ffn_mx(
        ctypes.byref(p), _arg(c, "x_codes", x_codes, u8, p.T * p.d // 2, dev),
        _arg(c, "x_scales", x_scales, u8, p.T * p.d // 32, dev),
        _arg(c, "sorted_slot", sorted_slot, i32, S, dev),
        _arg(c, "offsets", offsets, i32, p.num_local + 1, dev),
        _arg(c, "w_gate", w_gate, u8, W // 2, dev), _arg(c, "w_up", w_up, u8, W // 2, dev),
        _arg(c, "w_down", w_down, u8, W // 2, dev), _arg(c, "s_gate", s_gate, u8, W // 32, dev),
        _arg(c, "s_up", s_up, u8, W // 32, dev), _arg(c, "s_down", s_down, u8, W // 32, dev),
        _arg(c, "topk_w", topk_w, torch.float32, S, dev),
        _arg(c, "y", y, torch.bfloat16, S * p.d, dev), wp, wn, st))


def workspace(p: Problem, call: int, device="cuda") -> torch.Tensor:
    """A device scratch tensor of the size the library asks for (torch memory)."""
    n = moe_workspace_size(p, call)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)
