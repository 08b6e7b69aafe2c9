"""The router-training operators on real workloads: the balance loss, the
router's and the combine's backward passes, and the global gradient norm with
clipping.

``own`` False: elementary torch operations in 32 bits (64 for the norm over
many tensors).  ``own`` True: the library's calls.
"""
import math

import torch

own = False

ACT = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # -- balance loss and per-expert counts
        # a layer of eight experts on a decode-sized batch: latency
        dict(name="balance_small", op="balance", T=64, E=8, k=2, pad=0),
        # a training batch of the Qwen3-30B-A3B shape, a quarter of it padding
        dict(name="balance_padded", op="balance", T=8192, E=128, k=8, pad=25),
        # an expert count and a token count that are multiples of nothing
        dict(name="balance_odd", op="balance", T=4099, E=150, k=6, pad=10),
        # a global batch of the DeepSeek-V3 shape
        dict(name="balance_large", op="balance", T=131072, E=256, k=8, pad=0),
        # -- the router's backward pass: gates and losses to logits, tokens, matrix, bias
        # the float32 layer
        dict(name="router_small_f32", op="router", T=64, d=128, E=8, k=2, act="f32", pad=0, dx=True),
        # an odd expert count, a padded batch that ends inside a tile
        dict(name="router_odd", op="router", T=1001, d=640, E=20, k=3, act="bf16", pad=20, dx=True),
        # router tuning on the Qwen3-30B-A3B shape: no gradient for the tokens
        dict(name="router_tuning", op="router", T=8192, d=2048, E=128, k=8, act="bf16", pad=0, dx=False),
        # the DeepSeek-V3 shape with every gradient
        dict(name="router_large", op="router", T=16384, d=7168, E=256, k=8, act="bf16", pad=0, dx=True),
        # -- the combine's backward pass
        # the Qwen3-30B-A3B decode batch
        dict(name="combine_small", op="combine", T=64, d=2048, E=128, local=128, k=8, act="bf16", dy=True),
        # the Qwen3-30B-A3B prefill batch
        dict(name="combine_large", op="combine", T=8192, d=2048, E=128, local=128, k=8, act="bf16", dy=True),
        # -- global gradient norm and clipping
        # the router gradients of 48 layers packed in one buffer, odd starts among them
        dict(name="clip_routers", op="clip", layers=48, d=2048, E=127, F=0, clips=True),
        # one layer's gradients, the expert matrices included
        dict(name="clip_experts", op="clip", layers=1, d=2048, E=128, F=768, clips=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "router", "combine", "clip"])
    if op == "clip":
        while True:
            c = dict(op=op, layers=_log(rng, 1, 60), d=128 * _log(rng, 1, 56), E=_log(rng, 1, 256),
                     F=rng.choice([0, 128 * _log(rng, 1, 16)]), clips=rng.random() < 0.7)
            if _numel(c) <= 600_000_000:
                return c
    E = _log(rng, 4, 512)
    k = rng.randint(1, min(16, E // 2))
    if op == "balance":
        return dict(op=op, T=_log(rng, 1, 131072 * 256 // max(E, 256)), E=E, k=k, pad=rng.choice([0, 0, 10, 45]))
    act = rng.choice(["bf16", "bf16", "f32"])
    d = 128 * _log(rng, 1, 56)
    if op == "router":
        most = 16384 * 7168 * 256 // (d * max(E, 128)) // (1 if act == "bf16" else 16)
        return dict(op=op, T=_log(rng, 1, min(16384, most)), d=d, E=E, k=k, act=act,
                    pad=rng.choice([0, 0, 10, 45]), dx=rng.random() < 0.7)
    most = 8192 * 2048 * 8 * 2 // (d * k * (2 if act == "bf16" else 4))
    return dict(op=op, T=_log(rng, 1, min(16384, most)), d=d, E=E, local=rng.choice([E, E, max(1, E // 8)]),
                k=k, act=act, dy=rng.random() < 0.7)


def _sizes(case):
    """(float32 tensors, bfloat16 tensors): router matrix and bias of each layer; its three expert matrices."""
    d, E, F = case["d"], case["E"], case["F"]
    return [d * E, E] * case["layers"], [E * F * d] * (3 * case["layers"] if F else 0)


def _numel(case):
    a, b = _sizes(case)
    return sum(a) + sum(b)


def _views(flat, sizes):
    return list(torch.split(flat, sizes)) if sizes else []


def _routed(case, g, dev):
    """Router logits with a skewed load, their top-k ids and gates, and the mask of a padded batch."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn(T, E, generator=g, device=dev)
    logits += 2.0 * (torch.arange(E, device=dev, dtype=torch.float32) + 1).pow(-1.1)
    top, idx = torch.topk(logits, k, dim=1)
    w = torch.softmax(top, dim=1)
    mask = None
    if case.get("pad"):  # sequences of 512 tokens, each filled up to a length of its own
        length = torch.randint(512 - 512 * 2 * case["pad"] // 100, 513, ((T + 511) // 512,), generator=g, device=dev)
        t = torch.arange(T, device=dev)
        mask = (t % 512 < length[t // 512]).to(torch.uint8)
    return logits, idx.to(torch.int32), w, mask


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case)
    if case["op"] == "clip":
        s32, s16 = _sizes(case)
        s["flat32"] = torch.randn(sum(s32), generator=g, device=dev)
        s["flat16"] = torch.randn(sum(s16), generator=g, device=dev).to(torch.bfloat16)
        # a norm of about 3.2 or 0.32 against a limit of 1
        scale = (3.2 if case["clips"] else 0.32) / math.sqrt(_numel(case))
        s["flat32"] *= scale
        s["flat16"] *= scale
        s["out32"], s["out16"] = torch.zeros_like(s["flat32"]), torch.zeros_like(s["flat16"])
        s["grads"] = _views(s["flat32"], s32) + _views(s["flat16"], s16)
        s["out"] = _views(s["out32"], s32) + _views(s["out16"], s16)
        s["norm"] = torch.zeros(1, device=dev)
        s["max_norm"] = 1.0
        return s
    T, E, k = case["T"], case["E"], case["k"]
    logits, idx, w, mask = _routed(case, g, dev)
    s.update(topk_idx=idx, topk_w=w, mask=mask)

    def out(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype, device=dev)

    if case["op"] == "balance":
        s.update(logits=logits, counts=out(E, dtype=torch.int32), n_tokens=out(1, dtype=torch.int32),
                 prob_mean=out(E), losses=out(2))
        return s
    d, act = case["d"], ACT[case["act"]]
    if case["op"] == "router":
        valid = torch.ones(T, device=dev, dtype=torch.bool) if mask is None else mask.bool()
        # what the balance loss gave for this batch, and the step's gradients: those of means over tokens
        s.update(logits=logits, n_tokens=valid.sum(dtype=torch.int32).reshape(1),
                 counts=out(E, dtype=torch.int32).index_add_(
                     0, idx.reshape(-1), valid.to(torch.int32).repeat_interleave(k)),
                 dlosses=torch.tensor([1e-2, 1e-3], device=dev),
                 dtopk_w=torch.randn(T, k, generator=g, device=dev) * (0.05 / T),
                 x=torch.randn(T, d, generator=g, device=dev).to(act),
                 w_router=(torch.randn(d, E, generator=g, device=dev) / math.sqrt(d)).to(act),
                 dlogits=out(T, E), dw_router=out(d, E), dbias=out(E),
                 dx_out=out(T, d, dtype=act) if case["dx"] else None)
        return s
    # combine: expert outputs in expert order, the slots of the local experts kept
    flat = idx.reshape(-1).long()
    key = torch.where(flat < case["local"], flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    pos = torch.empty(T * k, dtype=torch.int32, device=dev)
    pos[order] = torch.arange(T * k, dtype=torch.int32, device=dev)
    s.update(slot_pos=torch.where(key < E, pos, torch.full_like(pos, -1)),
             y=torch.randn(T * k, d, generator=g, device=dev).to(act),
             dout=(torch.randn(T, d, generator=g, device=dev) / T).to(act), dtopk_w=out(T, k),
             dy_out=out(T * k, d, dtype=act) if case["dy"] else None)
    return s


# ---- plain forms

def _softmax(logits):
    m = logits.max(dim=1, keepdim=True).values
    e = (logits - m).exp()
    z = e.sum(dim=1, keepdim=True)
    return e / z, (m + z.log()).squeeze(1)


def _plain_balance(s):
    T, E, k = s["T"], s["E"], s["k"]
    p, lse = _softmax(s["logits"])
    if s["mask"] is None:
        n = torch.full((1,), T, dtype=torch.int32, device=p.device)
        ones = torch.ones(T * k, dtype=torch.int32, device=p.device)
    else:
        keep = s["mask"] != 0
        p = torch.where(keep[:, None], p, 0.0)
        lse = torch.where(keep, lse, 0.0)
        n = keep.sum(dtype=torch.int32).reshape(1)
        ones = keep.to(torch.int32).repeat_interleave(k)
    counts = torch.zeros(E, dtype=torch.int32, device=p.device).index_add_(0, s["topk_idx"].reshape(-1), ones)
    inv = 1.0 / n.clamp(min=1).float()
    mean = p.sum(dim=0) * inv
    balance = (counts.float() * mean).sum() * (E / k) * inv
    z = lse.square().sum() * inv
    return dict(counts=counts, n_tokens=n, prob_mean=mean, losses=torch.cat([balance.reshape(1), z.reshape(1)]))


def _plain_router(s):
    E, k = s["E"], s["k"]
    idx = s["topk_idx"].long()
    p, lse = _softmax(s["logits"])
    n = s["n_tokens"].clamp(min=1).float()
    c = s["counts"].float()
    a, b = s["dlosses"][0], s["dlosses"][1]
    g = s["dtopk_w"]
    gates = s["topk_w"] * (g - (s["topk_w"] * g).sum(dim=1, keepdim=True))
    dl = (a * E / (n * n * k)) * p * (c - (p * c).sum(dim=1, keepdim=True)) + (2 * b / n) * lse[:, None] * p
    dl = dl.scatter_add(1, idx, gates)
    if s["mask"] is not None:
        dl = torch.where((s["mask"] != 0)[:, None], dl, 0.0)
    r = dict(dlogits=dl, dw_router=s["x"].float().t() @ dl, dbias=dl.sum(dim=0))
    if s["dx"]:
        r["dx"] = (dl @ s["w_router"].float().t()).to(s["x"].dtype)
    return r


def _plain_combine(s):
    T, k = s["T"], s["k"]
    pos = s["slot_pos"].long()
    kept = (pos >= 0).nonzero().squeeze(1)
    rows, slots = pos[kept], kept
    dout = s["dout"].float()[slots // k]
    dw = torch.zeros(T * k, device=dout.device)
    dw[slots] = (dout * s["y"][rows].float()).sum(dim=1)
    r = dict(dtopk_w=dw.view(T, k))
    if s["dy"]:
        r["dy"] = torch.zeros_like(s["dy_out"])
        r["dy"][rows] = (dout * s["topk_w"].reshape(-1)[slots, None]).to(s["y"].dtype)
    return r


def _plain_clip(s):
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum()
    norm = total.sqrt().float()
    coef = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
    for g, o in zip(s["grads"], s["out"]):
        o.copy_(g.float() * coef)
    return dict(norm=norm.reshape(1), out32=s["out32"], out16=s["out16"])


# ---- the library's calls

_scratch = {}


def _workspace(nbytes, dev):
    """The program's scratch memory: one buffer, as large as the largest call so far has asked for."""
    if _scratch.get("ws") is None or _scratch["ws"].numel() < nbytes:
        _scratch["ws"] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    return _scratch["ws"]


def _own(s):
    from mixture_experts_layer_15_amd import binding as B
    if s["op"] == "clip":
        tensors = B.grad_list(s["grads"], s["out"])
        ws = _workspace(B.moe_grad_workspace_size(tensors), s["norm"].device)
        B.moe_grad_norm(tensors, s["norm"], ws)
        B.moe_grad_clip(tensors, s["norm"], s["max_norm"])
        return dict(norm=s["norm"], out32=s["out32"], out16=s["out16"])
    act = s.get("act", "f32")
    p = B.problem(s["T"], s.get("d", 128), s["E"], s["k"], 128, 0, s.get("local", s["E"]), act, act)
    if s["op"] == "balance":
        ws = _workspace(B.moe_workspace_size(p, B.MOE_CALL_BALANCE_LOSS), s["logits"].device)
        B.moe_balance_loss(p, s["logits"], s["topk_idx"], s["mask"], s["counts"], s["n_tokens"], s["prob_mean"],
                           s["losses"], ws)
        return dict(counts=s["counts"], n_tokens=s["n_tokens"], prob_mean=s["prob_mean"], losses=s["losses"])
    if s["op"] == "router":
        ws = _workspace(B.moe_workspace_size(p, B.MOE_CALL_ROUTE_BACKWARD), s["logits"].device)
        B.moe_route_backward(p, x=s["x"], w_router=s["w_router"], logits=s["logits"], topk_idx=s["topk_idx"],
                             topk_w=s["topk_w"], dtopk_w=s["dtopk_w"], token_mask=s["mask"], counts=s["counts"],
                             n_tokens=s["n_tokens"], dlosses=s["dlosses"], dlogits=s["dlogits"], dx=s["dx_out"],
                             dw_router=s["dw_router"], dbias=s["dbias"], ws=ws)
        r = dict(dlogits=s["dlogits"], dw_router=s["dw_router"], dbias=s["dbias"])
        if s["dx"]:
            r["dx"] = s["dx_out"]
        return r
    B.moe_combine_backward(p, s["dout"], s["y"], s["slot_pos"], s["topk_w"], s["dy_out"], s["dtopk_w"])
    r = dict(dtopk_w=s["dtopk_w"])
    if s["dy"]:
        r["dy"] = s["dy_out"]
    return r


def run(s):
    if own:
        return _own(s)
    return {"balance": _plain_balance, "router": _plain_router, "combine": _plain_combine, "clip": _plain_clip}[s["op"]](s)


def work(case):
    if case["op"] == "clip":
        s32, s16 = _sizes(case)
        n = sum(s32) + sum(s16)
        return {"bytes": 2 * (4 * sum(s32) + 2 * sum(s16)) + 4, "flops": 3 * n}
    T, E, k = case["T"], case["E"], case["k"]
    mask = T if case.get("pad") else 0
    if case["op"] == "balance":
        return {"bytes": 4 * T * E + 4 * T * k + mask + 8 * E + 12, "flops": 6 * T * E}
    d, b = case["d"], 4 if case["act"] == "f32" else 2
    if case["op"] == "router":
        products = 2 if case["dx"] else 1
        return {"bytes": 8 * T * E + 12 * T * k + mask + products * b * T * d + (products - 1) * b * d * E + 4 * d * E + 8 * E + 12,
                "flops": 2 * products * T * d * E + 10 * T * E}
    kept = T * k * case["local"] / E
    return {"bytes": b * T * d + (2 if case["dy"] else 1) * b * kept * d + 12 * T * k, "flops": (3 if case["dy"] else 2) * kept * d}


# ---- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2 for g in s["grads"]))
        c = s["max_norm"] / norm if norm > s["max_norm"] else 1.0
        return dict(norm=torch.tensor([norm], dtype=torch.float64), out32=s["flat32"].double() * c,
                    out16=s["flat16"].double() * c)
    T, E, k = case["T"], case["E"], case["k"]
    keep = torch.ones(T, dtype=torch.bool, device=s["topk_idx"].device) if s["mask"] is None else s["mask"].bool()
    n = int(keep.sum())
    if case["op"] == "combine":
        pos = s["slot_pos"].view(T, k).long()
        dw, dy = torch.zeros(T, k, dtype=torch.float64, device=pos.device), None
        if case["dy"]:
            dy = torch.zeros(T * k, case["d"], dtype=torch.float64, device=pos.device)
        for i in range(k):
            t = (pos[:, i] >= 0).nonzero()[:, 0]
            do = s["dout"][t].double()
            dw[t, i] = torch.einsum("td,td->t", do, s["y"][pos[t, i]].double())
            if dy is not None:
                dy[pos[t, i]] = do * s["topk_w"][t, i, None].double()
        return dict(dtopk_w=dw, dy=dy) if case["dy"] else dict(dtopk_w=dw)
    logits = s["logits"].double().requires_grad_(True)
    rows, ids = logits[keep], s["topk_idx"][keep].long()
    counts = torch.histc(ids.double(), bins=E, min=-0.5, max=E - 0.5)
    if n:
        mean = torch.softmax(rows, dim=1).mean(dim=0)
        losses = torch.stack([E * (counts / (n * k) * mean).sum(), torch.logsumexp(rows, dim=1).pow(2).mean()])
    else:
        mean, losses = torch.zeros(E, dtype=torch.float64, device=ids.device), (rows.sum() * 0).repeat(2)
    if case["op"] == "balance":
        return dict(counts=counts.round().to(torch.int32), n_tokens=torch.tensor([n], dtype=torch.int32),
                    prob_mean=mean.detach(), losses=losses.detach())
    # the gates as a function of the chosen logits that has the value and the slope of a softmax with these gates
    w, g = s["topk_w"].double(), s["dtopk_w"].double()
    chosen = torch.gather(logits, 1, s["topk_idx"].long())
    step = chosen - chosen.detach()
    gates = w * (1 + step - (w * step).sum(dim=1, keepdim=True))
    total = (torch.where(keep[:, None], gates * g, 0.0)).sum() + (losses * s["dlosses"].double()).sum()
    dl, = torch.autograd.grad(total, logits)
    r = dict(dlogits=dl, dw_router=torch.mm(s["x"].double().t(), dl), dbias=torch.mv(dl.t(), torch.ones(T, dtype=torch.float64, device=dl.device)))
    if case["dx"]:
        r["dx"] = torch.mm(dl, s["w_router"].double().t())
    return r
