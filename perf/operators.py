"""The loss operators of a mixture-of-experts language model, as cases to measure.

Two operators, each with its forward and its backward pass:

* the linear cross entropy `gemm_bf16_nt_xent`: the loss of the logits X W^T
  of a language-model head, in pieces of the vocabulary, logits never kept;
* the routing step `router_topk`: softmax, top-k, per-expert counts, balance
  loss and z-loss on the router's FP32 logits.

`run` computes them in their plain form (32-bit torch operations), or with
`own` set through the package's entry points.
"""
import math

import torch

own = False

F32 = torch.float32
F64 = torch.float64

# The most multiply-adds M * V * K of a drawn linear cross entropy, and the
# most logits of a drawn routing step: those of the largest listed ones.
MOST_MACS = 4096 * 131072 * 4096
MOST_LOGITS = 65536 * 256


def listed():
    return [
        # scoring one token: streams the head's weights once
        {"name": "xent_fwd_one_token", "op": "xent_fwd", "M": 1, "V": 32768, "K": 2048},
        # scoring a small batch with a ragged vocabulary
        {"name": "xent_fwd_100x50001x1024", "op": "xent_fwd", "M": 100, "V": 50001, "K": 1024},
        # one sequence of the fine-tuning length, odd sizes everywhere
        {"name": "xent_fwd_1016x32003x2056", "op": "xent_fwd", "M": 1016, "V": 32003, "K": 2056},
        # a training batch on a large vocabulary
        {"name": "xent_fwd_8192x65536x4096", "op": "xent_fwd", "M": 8192, "V": 65536, "K": 4096},
        # gradients of a few rows: every weight is read and its gradient written
        {"name": "xent_bwd_37x32768x2048", "op": "xent_bwd", "M": 37, "V": 32768, "K": 2048, "dx": True, "dw": True},
        # one sequence, odd sizes
        {"name": "xent_bwd_1016x32003x2056", "op": "xent_bwd", "M": 1016, "V": 32003, "K": 2056, "dx": True, "dw": True},
        # adapters are trained and the head is frozen: only the rows' gradient
        {"name": "xent_bwd_dx_2048x65536x7168", "op": "xent_bwd", "M": 2048, "V": 65536, "K": 7168, "dx": True, "dw": False},
        # a training batch on a large vocabulary, both gradients
        {"name": "xent_bwd_4096x131072x4096", "op": "xent_bwd", "M": 4096, "V": 131072, "K": 4096, "dx": True, "dw": True},
        # routing of one decoded token
        {"name": "route_fwd_1x256_top8", "op": "route_fwd", "M": 1, "E": 256, "k": 8, "norm": True, "holes": False},
        # routing of the repository's router workload, with padding tokens and closed experts
        {"name": "route_fwd_4510x256_top8", "op": "route_fwd", "M": 4510, "E": 256, "k": 8, "norm": True, "holes": True},
        # few experts, odd counts, bf16 gradient for the router's weight product
        {"name": "route_bwd_4093x60_top4", "op": "route_bwd", "M": 4093, "E": 60, "k": 4, "norm": False, "holes": True, "bf16": True},
        # a large training batch
        {"name": "route_bwd_65536x256_top8", "op": "route_bwd", "M": 65536, "E": 256, "k": 8, "norm": True, "holes": True, "bf16": False},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["xent_fwd", "xent_bwd", "route_fwd", "route_bwd"])
    while op.startswith("xent"):
        M, V, K = _log_between(rng, 1, 8192), _log_between(rng, 1000, 131072), 8 * _log_between(rng, 32, 896)
        if M * V * K > MOST_MACS:
            continue
        case = {"op": op, "M": M, "V": V, "K": K}
        if op == "xent_bwd":
            case["dx"], case["dw"] = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        return case
    while True:
        M, E = _log_between(rng, 1, 65536), _log_between(rng, 4, 512)
        if M * E <= MOST_LOGITS:
            break
    case = {"op": op, "M": M, "E": E, "k": rng.randint(1, min(E, 16)), "norm": rng.random() < 0.5, "holes": rng.random() < 0.5}
    if op == "route_bwd":
        case["bf16"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs
def _prepare_xent(case, gen):
    M, V, K = case["M"], case["V"], case["K"]
    dev = gen.device
    W = (torch.randn(V, K, generator=gen, device=dev) * (2.0 / math.sqrt(K))).bfloat16()
    target = torch.randint(0, V, (M,), generator=gen, device=dev)
    # rows from unlearned to well learned: their target's probability runs from 1/V to nearly 1
    learned = torch.rand(M, 1, generator=gen, device=dev) * 4.5
    X = (torch.randn(M, K, generator=gen, device=dev) + learned * W[target].float()).bfloat16()
    # padding and prompt rows carry no loss; a single row does
    skip = torch.rand(M, generator=gen, device=dev) < (0.1 if M > 1 else 0.0)
    target[skip] = -100
    state = {"X": X, "W": W, "target": target}
    if case["op"] == "xent_bwd":
        live = (target >= 0).sum().clamp(min=1)
        state["dloss"] = (0.5 + torch.rand(M, generator=gen, device=dev)) / live
        state["lse"] = torch.logsumexp(X.float() @ W.float().T, dim=1)
    return state


def _prepare_route(case, gen):
    M, E, k = case["M"], case["E"], case["k"]
    dev = gen.device
    # per-expert offsets make the load uneven; a coarse grid of values makes ties
    logits = 1.5 * torch.randn(M, E, generator=gen, device=dev) + 0.7 * torch.randn(E, generator=gen, device=dev)
    tied = torch.rand(M, 1, generator=gen, device=dev) < 0.25
    logits = torch.where(tied, torch.round(logits * 8) / 8, logits)
    valid = torch.ones(M, dtype=torch.uint8, device=dev)
    if case["holes"]:
        closed = (torch.rand(M, E, generator=gen, device=dev) < 0.3) & (torch.rand(M, 1, generator=gen, device=dev) < 0.5)
        closed |= torch.rand(M, 1, generator=gen, device=dev) < 0.01  # rows with no expert left
        logits = torch.where(closed, torch.full_like(logits, -math.inf), logits)
        valid = (torch.rand(M, generator=gen, device=dev) >= 0.1).to(torch.uint8)
    state = {"logits": logits, "valid": valid}
    if case["op"] == "route_bwd":
        _, experts, lse, counts, _, _ = _route_fwd(logits, valid, k, case["norm"])
        state.update(experts=experts, lse=lse, counts=counts)
        state["dweights"] = torch.randn(M, k, generator=gen, device=dev) / M
        state["dlosses"] = torch.tensor([1e-2, 1e-3], device=dev)  # the two losses' coefficients
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = (_prepare_xent if case["op"].startswith("xent") else _prepare_route)(case, gen)
    state["case"] = dict(case)
    return state


# ------------------------------------------------------------------ plain forms
def _xent_fwd(X, W, target):
    logits = X.float() @ W.float().T
    top = logits.amax(dim=1)
    lse = top + torch.log(torch.exp(logits - top[:, None]).sum(dim=1))
    picked = logits.gather(1, target.clamp(min=0)[:, None])[:, 0]
    loss = torch.where(target >= 0, lse - picked, torch.zeros_like(lse))
    return loss, lse


def _xent_bwd(X, W, target, lse, dloss, dx, dw):
    x, w = X.float(), W.float()
    g = torch.exp(x @ w.T - lse[:, None])
    g.scatter_add_(1, target.clamp(min=0)[:, None], torch.full_like(lse, -1.0)[:, None])
    g *= torch.where(target >= 0, dloss, torch.zeros_like(dloss))[:, None]
    dX = (g @ w).bfloat16() if dx else None
    dW = (g.T @ x).bfloat16() if dw else None
    return [t for t in (dX, dW) if t is not None]


def _route_fwd(logits, valid, k, norm):
    M, E = logits.shape
    top = logits.amax(dim=1)
    live = (valid != 0) & (top > -math.inf)
    shift = torch.where(top > -math.inf, top, torch.zeros_like(top))
    lse = shift + torch.log(torch.exp(logits - shift[:, None]).sum(dim=1))
    p = torch.where(live[:, None], torch.exp(logits - torch.where(live, lse, shift)[:, None]), torch.zeros_like(logits))
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    best, idx = order.values[:, :k], order.indices[:, :k]
    taken = live[:, None] & (best > -math.inf)
    w = torch.where(taken, p.gather(1, idx), torch.zeros_like(best))
    if norm:
        s = w.sum(dim=1, keepdim=True)
        w = torch.where(taken, w / torch.where(live[:, None], s, torch.ones_like(s)), w)
    experts = torch.where(taken, idx, torch.full_like(idx, -1)).to(torch.int32)
    n = live.sum()
    slot = torch.where(taken, idx, torch.full_like(idx, E)).reshape(-1)
    hits = torch.zeros(E + 1, dtype=torch.int64, device=logits.device).scatter_add_(0, slot, torch.ones_like(slot))[:E]
    counts = torch.cat([hits, n[None]]).to(torch.int32)
    t = n.clamp(min=1).float()
    prob = p.sum(dim=0) / t
    balance = E * (hits.float() / (k * t) * prob).sum()
    z = torch.where(live, lse * lse, torch.zeros_like(lse)).sum() / t
    return w, experts, lse, counts, prob, torch.stack([balance, z])


def _route_bwd(logits, experts, lse, counts, dweights, dlosses, norm, bf16):
    M, E = logits.shape
    k = experts.shape[1]
    live = experts[:, :1] >= 0
    t = counts[E].clamp(min=1).float()
    p = torch.where(live, torch.exp(logits - torch.where(live, lse[:, None], torch.full_like(live, math.inf, dtype=F32))), torch.zeros_like(logits))
    idx = experts.clamp(min=0).long()
    taken = experts >= 0
    dwt = torch.where(taken, dweights, torch.zeros_like(dweights))
    if norm:
        q = torch.where(taken, p.gather(1, idx), torch.zeros_like(dwt))
        s = torch.where(live, q.sum(dim=1, keepdim=True), torch.ones_like(dwt[:, :1]))
        w = q / s
        dwt = torch.where(taken, (dwt - (dwt * w).sum(dim=1, keepdim=True)) / s, torch.zeros_like(dwt))
    dp = (dlosses[0] * E * counts[:E].float() / (k * t * t))[None, :].repeat(M, 1)
    dp = dp.scatter_add(1, idx, dwt)
    dl = p * (dp - (p * dp).sum(dim=1, keepdim=True))
    dl = dl + p * torch.where(live, 2.0 * dlosses[1] * lse[:, None] / t, torch.zeros_like(dl[:, :1]))
    return dl.bfloat16() if bf16 else dl


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import nvfp4_block_scaled_tcgen05_gb300 as g
        if op == "xent_fwd":
            return list(g.gemm_bf16_nt_xent(state["X"], state["W"], state["target"]))
        if op == "xent_bwd":
            out = g.gemm_bf16_nt_xent_backward(state["X"], state["W"], state["target"], state["lse"], state["dloss"],
                                               need_dx=case["dx"], need_dw=case["dw"])
            return [t for t in out if t is not None]
        if op == "route_fwd":
            return list(g.router_topk(state["logits"], case["k"], valid=state["valid"], normalize=case["norm"]))
        return g.router_topk_backward(state["logits"], state["experts"], state["lse"], state["counts"], dweights=state["dweights"],
                                      dlosses=state["dlosses"], normalize=case["norm"], dtype=torch.bfloat16 if case["bf16"] else F32)
    if op == "xent_fwd":
        return list(_xent_fwd(state["X"], state["W"], state["target"]))
    if op == "xent_bwd":
        return _xent_bwd(state["X"], state["W"], state["target"], state["lse"], state["dloss"], case["dx"], case["dw"])
    if op == "route_fwd":
        return list(_route_fwd(state["logits"], state["valid"], case["k"], case["norm"]))
    return _route_bwd(state["logits"], state["experts"], state["lse"], state["counts"], state["dweights"], state["dlosses"],
                      case["norm"], case["bf16"])


def work(case):
    """Inputs read once, outputs written once; the products of a pass that
    keeps no logits (the backward pass forms them again)."""
    M = case["M"]
    if case["op"].startswith("xent"):
        V, K = case["V"], case["K"]
        both = 2 * (M * K + V * K)
        if case["op"] == "xent_fwd":
            return {"bytes": both + 8 * M + 8 * M, "flops": 2 * M * V * K}
        out = 2 * (M * K if case["dx"] else 0) + 2 * (V * K if case["dw"] else 0)
        return {"bytes": both + 16 * M + out, "flops": 2 * M * V * K * (1 + case["dx"] + case["dw"])}
    E, k = case["E"], case["k"]
    if case["op"] == "route_fwd":
        return {"bytes": 4 * M * E + M + 8 * M * k + 4 * M + 8 * E + 12, "flops": 6 * M * E}
    return {"bytes": 4 * M * E + (2 if case["bf16"] else 4) * M * E + 8 * M * k + 4 * M + 4 * E + 12, "flops": 8 * M * E}


# ------------------------------------------------------------------ 64 bits
def _exact_xent(case, s):
    V = case["V"]
    X, target = s["X"].to(F64), s["target"]
    keep = (target >= 0).to(F64)
    step = 16384
    if case["op"] == "xent_fwd":
        parts, picked = [], torch.zeros_like(keep)
        for v in range(0, V, step):
            z = X @ s["W"][v:v + step].to(F64).T
            parts.append(torch.logsumexp(z, dim=1))
            here = (target >= v) & (target < v + z.shape[1])
            picked = torch.where(here, z.gather(1, (target - v).clamp(0, z.shape[1] - 1)[:, None])[:, 0], picked)
        lse = torch.logsumexp(torch.stack(parts), dim=0)
        return [keep * (lse - picked), lse]
    lse, row = s["lse"].to(F64), s["dloss"].to(F64) * keep
    dX, dW = torch.zeros_like(X), []
    for v in range(0, V, step):
        w = s["W"][v:v + step].to(F64)
        p = torch.exp(X @ w.T - lse[:, None])
        p -= (torch.arange(v, v + w.shape[0], device=X.device)[None, :] == target[:, None]).to(F64)
        p *= row[:, None]
        if case["dx"]:
            dX += p @ w
        if case["dw"]:
            dW.append(p.T @ X)
    return ([dX] if case["dx"] else []) + ([torch.cat(dW)] if case["dw"] else [])


def _exact_route(case, s):
    l = s["logits"].to(F64)
    M, E = l.shape
    k = case["k"]
    some = torch.isfinite(l).any(dim=1)
    lse = torch.logsumexp(l, dim=1)
    if case["op"] == "route_fwd":
        live = some & (s["valid"] != 0)
        p = torch.nan_to_num(torch.softmax(l, dim=1)) * live[:, None]
        _, idx = torch.sort(l, dim=1, descending=True, stable=True)
        idx = idx[:, :k]
        used = live[:, None] & torch.isfinite(l.gather(1, idx))
        w = p.gather(1, idx) * used
        if case["norm"]:
            w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
        hits = torch.bincount(idx[used], minlength=E)
        t = max(1, int(live.sum()))
        mean = p.sum(dim=0) / t
        balance = E * (hits.to(F64) / (k * t) * mean).sum()
        z = (lse[live] ** 2).sum() / t
        return [w, None, lse, None, mean, torch.stack([balance, z])]
    ids = s["experts"].long()
    used = ids >= 0
    live = used[:, 0]
    t = max(1, int(s["counts"][E]))
    p = torch.nan_to_num(torch.exp(l - s["lse"].to(F64)[:, None])) * live[:, None]
    up = s["dweights"].to(F64) * used
    at = ids.clamp(min=0)
    if case["norm"]:
        q = p.gather(1, at) * used
        total = q.sum(dim=1, keepdim=True)
        total[~live] = 1.0
        up = (up - (up * q).sum(dim=1, keepdim=True) / total) / total * used
    c0, c1 = (float(v) for v in s["dlosses"])
    dp = (c0 * E / (k * t * t)) * s["counts"][:E].to(F64).expand(M, E)
    dp = dp.scatter_add(1, at, up)
    out = p * (dp - (p * dp).sum(dim=1, keepdim=True))
    zrow = 2.0 * c1 / t * torch.where(live, s["lse"].to(F64), torch.zeros_like(lse))
    return out + p * zrow[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_xent if case["op"].startswith("xent") else _exact_route)(case, s)
