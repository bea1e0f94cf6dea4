"""The operators of a language model's feed-forward block, as cases to measure.

Four operators, trained and decoded with:

* the gated projection `gemm_bf16_nt_gated`: H = act(X Wg^T) * (X Wu^T), and its
  backward pass, from the stored gates or from X alone;
* the weight gradient `gemm_bf16_tn`: A^T B, the down projection's gradient;
* the residual step `residual_norm`: the norm after a block, its gate and
  residual scale, and the norm before the next block, forward and backward;
* products of few tokens with 4-bit weights, `gemv_w4a16` and, for both gated
  projections at once, `gemv_w4a16_gated`.

`run` computes them in their plain form (32-bit torch operations), or with
`own` set through the package's entry points.
"""
import math

import torch

own = False

F32 = torch.float32
F64 = torch.float64
BF16 = torch.bfloat16

EPS = 1e-6
ROOT_2_OVER_PI = math.sqrt(2.0 / math.pi)

# The most work of a drawn case: that of the largest listed ones.
MOST_MACS = 5120 * 11008 * 2048
MOST_VALUES = 16384 * 4096
MOST_WEIGHTS = 16384 * 7168


def listed():
    return [
        # one decoded token: streams both projections' weights once
        {"name": "gated_fwd_one_token_11008x2048", "op": "gated_fwd", "M": 1, "F": 11008, "K": 2048, "act": "silu", "gates": False},
        # a prompt of the fine-tuning length, odd sizes everywhere
        {"name": "gated_fwd_1016x5512x2056", "op": "gated_fwd", "M": 1016, "F": 5512, "K": 2056, "act": "gelu_tanh", "gates": False},
        # a training batch of the repository's gate and up shape, gates kept for the backward pass
        {"name": "gated_fwd_5120x11008x2048", "op": "gated_fwd", "M": 5120, "F": 11008, "K": 2048, "act": "silu", "gates": True},
        # one sequence, odd sizes, gates formed again (activations are not kept)
        {"name": "gated_bwd_1016x5512x2056", "op": "gated_bwd", "M": 1016, "F": 5512, "K": 2056, "act": "gelu_tanh", "gates": False},
        # the training batch's gradients from the stored gates
        {"name": "gated_bwd_5120x11008x2048", "op": "gated_bwd", "M": 5120, "F": 11008, "K": 2048, "act": "silu", "gates": True},
        # the down projection's gradient of a short sequence, odd sizes
        {"name": "tn_2056x5512x1015", "op": "tn", "M": 2056, "N": 5512, "K": 1015},
        # and of the training batch
        {"name": "tn_2048x11008x5120", "op": "tn", "M": 2048, "N": 11008, "K": 5120},
        # the residual step of one decoded token
        {"name": "norm_fwd_one_token_4096", "op": "norm_fwd", "M": 1, "D": 4096, "f32": False, "post": True, "pre": True, "groups": 1},
        # a training batch with the stream held in 32 bits
        {"name": "norm_fwd_16384x4096_f32", "op": "norm_fwd", "M": 16384, "D": 4096, "f32": True, "post": True, "pre": True, "groups": 1},
        # a training batch of odd rows whose gates belong to its sequences, gradients of everything
        {"name": "norm_bwd_8128x4104", "op": "norm_bwd", "M": 8128, "D": 4104, "f32": False, "post": True, "pre": True, "groups": 8},
        # the down projection of one decoded token
        {"name": "w4_2048x11008_one_token", "op": "w4", "M": 1, "N": 2048, "K": 11008},
        # both projections of a small batch of decoded tokens
        {"name": "w4_gated_11x8192x7168", "op": "w4_gated", "M": 11, "N": 8192, "K": 7168, "act": "silu"},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated_fwd", "gated_fwd", "gated_bwd", "tn", "norm_fwd", "norm_bwd", "w4", "w4_gated"])
    act = rng.choice(["silu", "gelu_tanh"])
    while op.startswith("gated"):
        M, F, K = _log_between(rng, 1, 8192), 8 * _log_between(rng, 16, 1792), 8 * _log_between(rng, 16, 896)
        if M * F * K <= MOST_MACS:
            return {"op": op, "M": M, "F": F, "K": K, "act": act, "gates": rng.random() < 0.5}
    while op == "tn":
        M, N, K = 8 * _log_between(rng, 16, 896), 8 * _log_between(rng, 16, 1792), _log_between(rng, 1, 8192)
        if M * N * K <= MOST_MACS:
            return {"op": op, "M": M, "N": N, "K": K}
    while op.startswith("norm"):
        M, D = _log_between(rng, 1, 65536), 8 * _log_between(rng, 8, 1024)
        groups = rng.choice([0, 1, 1, 2, 8, M])
        if M * D > MOST_VALUES or (groups and M % groups):
            continue
        kind = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        return {"op": op, "M": M, "D": D, "f32": rng.random() < 0.5, "post": kind[0], "pre": kind[1], "groups": groups}
    while True:
        M, N, K = rng.randint(1, 16), _log_between(rng, 64, 16384), 256 * _log_between(rng, 1, 64)
        if N * K <= (MOST_WEIGHTS if op == "w4" else MOST_WEIGHTS // 2):
            break
    case = {"op": op, "M": M, "N": N, "K": K}
    if op == "w4_gated":
        case["act"] = act
    return case


# ------------------------------------------------------------------ inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=gen.device)


def _prepare_gated(case, gen):
    M, F, K = case["M"], case["F"], case["K"]
    # gates of about unit size, as behind a norm
    state = {"X": _randn(gen, M, K).bfloat16(),
             "Wg": (_randn(gen, F, K) * (1.5 / math.sqrt(K))).bfloat16(),
             "Wu": (_randn(gen, F, K) * (1.0 / math.sqrt(K))).bfloat16()}
    if case["op"] == "gated_bwd":
        state["dH"] = (_randn(gen, M, F) * (0.1 / math.sqrt(F))).bfloat16()
        if case["gates"]:
            x = state["X"].float()
            state["gates"] = torch.stack([x @ state["Wg"].float().T, x @ state["Wu"].float().T]).bfloat16()
    return state


def _prepare_tn(case, gen):
    return {"A": (_randn(gen, case["K"], case["M"]) * 0.02).bfloat16(), "B": _randn(gen, case["K"], case["N"]).bfloat16()}


def _prepare_norm(case, gen):
    M, D = case["M"], case["D"]
    # a stream with a few large channels, a block's output, weights about one, gates about a half
    wide = torch.exp(0.5 * _randn(gen, D))
    x = _randn(gen, M, D) * wide * 2.0
    state = {"x": x if case["f32"] else x.bfloat16(), "block": (_randn(gen, M, D) * 0.7).bfloat16(), "scale": 0.7}
    state["w_post"] = (1.0 + 0.2 * _randn(gen, D)).bfloat16() if case["post"] else None
    state["w_pre"] = (1.0 + 0.2 * _randn(gen, D)).bfloat16() if case["pre"] else None
    state["gate"] = (0.5 + 0.25 * _randn(gen, case["groups"], D)).bfloat16() if case["groups"] else None
    if case["op"] == "norm_bwd":
        y, _, rstd_post, rstd_pre = _norm_fwd(state["x"], state["block"], state["w_post"], state["gate"], state["w_pre"], state["scale"])
        dy = _randn(gen, M, D) * 1e-3
        state = {**state, "x": None, "y": y, "rstd_post": rstd_post, "rstd_pre": rstd_pre, "dy": dy if case["f32"] else dy.bfloat16()}
        state["dn"] = (_randn(gen, M, D) * 1e-3).bfloat16() if case["pre"] else None
    return state


def _prepare_w4(case, gen):
    M, N, K = case["M"], case["N"], case["K"]
    state = {"A": _randn(gen, M, K).bfloat16()}
    for which in ("g", "u") if case["op"] == "w4_gated" else ("",):
        state["b" + which] = torch.randint(0, 256, (N, K // 2), generator=gen, device=gen.device, dtype=torch.uint8)
        # block scales over the powers of two from 2^-5 to 2^4
        exponent = torch.randint(2, 12, (N, K // 16), generator=gen, device=gen.device, dtype=torch.uint8)
        mantissa = torch.randint(0, 8, (N, K // 16), generator=gen, device=gen.device, dtype=torch.uint8)
        state["sf" + which] = exponent * 8 + mantissa
        state["scale" + which] = float(1.0 / (16.0 * math.sqrt(K)) * (1.0 if which != "u" else 1.25))
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    make = _prepare_gated if op.startswith("gated") else _prepare_tn if op == "tn" else _prepare_norm if op.startswith("norm") else _prepare_w4
    return {**make(case, gen), "case": dict(case)}


# ------------------------------------------------------------------ plain forms
def _act(g, act):
    z = g if act == "silu" else (2.0 * ROOT_2_OVER_PI) * (g + 0.044715 * g * g * g)
    return g / (1.0 + torch.exp(-z))


def _act_slope(g, act):
    z = g if act == "silu" else (2.0 * ROOT_2_OVER_PI) * (g + 0.044715 * g * g * g)
    dz = torch.ones_like(g) if act == "silu" else (2.0 * ROOT_2_OVER_PI) * (1.0 + 3.0 * 0.044715 * g * g)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s + g * s * (1.0 - s) * dz


def _gated_fwd(X, Wg, Wu, act, keep):
    x = X.float()
    g, u = x @ Wg.float().T, x @ Wu.float().T
    H = (_act(g, act) * u).bfloat16()
    return [H, torch.stack([g, u]).bfloat16()] if keep else [H]


def _gated_bwd(X, Wg, Wu, dH, act, gates):
    x, wg, wu, dh = X.float(), Wg.float(), Wu.float(), dH.float()
    if gates is None:
        g, u = x @ wg.T, x @ wu.T
    else:
        g, u = gates[0].float(), gates[1].float()
    dg, du = dh * u * _act_slope(g, act), dh * _act(g, act)
    return [(dg @ wg + du @ wu).bfloat16(), (dg.T @ x).bfloat16(), (du.T @ x).bfloat16()]


def _tn(A, B):
    return (A.float().T @ B.float()).bfloat16()


def _rows(gate, M):
    """The gate of each row: its sequence's."""
    return gate.float().repeat_interleave(M // gate.shape[0], dim=0)


def _norm_fwd(x, block, w_post, gate, w_pre, scale):
    b = block.float()
    rstd_post = rstd_pre = n = None
    if w_post is not None:
        rstd_post = 1.0 / torch.sqrt((b * b).mean(dim=1) + EPS)
        b = b * rstd_post[:, None] * w_post.float()
    if gate is not None:
        b = b * _rows(gate, x.shape[0])
    y = (x.float() + scale * b).to(x.dtype)
    if w_pre is not None:
        # the norm of the stream as it is stored
        s = y.float()
        rstd_pre = 1.0 / torch.sqrt((s * s).mean(dim=1) + EPS)
        n = (s * rstd_pre[:, None] * w_pre.float()).bfloat16()
    return y, n, rstd_post, rstd_pre


def _norm_bwd(dy, dn, y, block, rstd_post, rstd_pre, w_post, gate, w_pre, scale):
    t = dy.float()
    dw_pre = dw_post = dgate = None
    if w_pre is not None:
        yhat, d = y.float() * rstd_pre[:, None], dn.float()
        dw_pre = (d * yhat).sum(dim=0)
        d = d * w_pre.float()
        t = t + rstd_pre[:, None] * (d - yhat * (d * yhat).mean(dim=1, keepdim=True))
    dc, c, bhat = scale * t, block.float(), None
    if w_post is not None:
        bhat = c * rstd_post[:, None]
        c = bhat * w_post.float()
    if gate is not None:
        dgate = (dc * c).reshape(gate.shape[0], -1, gate.shape[1]).sum(dim=1)
        dc = dc * _rows(gate, y.shape[0])
    db = dc
    if w_post is not None:
        dw_post = (dc * bhat).sum(dim=0)
        q = dc * w_post.float()
        db = rstd_post[:, None] * (q - bhat * (q * bhat).mean(dim=1, keepdim=True))
    return t.to(dy.dtype), db.bfloat16(), dw_pre, dw_post, dgate


def _weights(b, sf):
    """e2m1 codes (two a byte, the even element low) times their e4m3 scales."""
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=b.device)
    table = torch.cat([mag, -mag])
    codes = torch.stack([b & 15, b >> 4], dim=2).reshape(b.shape[0], -1)
    return table[codes.int()] * sf.view(torch.float8_e4m3fn).float().repeat_interleave(16, dim=1)


def _w4(A, b, sf, scale):
    return scale * (A.float() @ _weights(b, sf).T)


# ------------------------------------------------------------------ one pass
def _given(*tensors):
    return [t for t in tensors if t is not None]


def run(state):
    case = state["case"]
    op, s = case["op"], state
    if own:
        import nvfp4_block_scaled_tcgen05_gb300 as g
        if op == "gated_fwd":
            return _given(*g.gemm_bf16_nt_gated(s["X"], s["Wg"], s["Wu"], act=case["act"], save_gates=case["gates"]))
        if op == "gated_bwd":
            return list(g.gemm_bf16_nt_gated_backward(s["X"], s["Wg"], s["Wu"], s["dH"], act=case["act"], gates=s.get("gates")))
        if op == "tn":
            return g.gemm_bf16_tn(s["A"], s["B"])
        if op == "norm_fwd":
            return _given(*g.residual_norm(s["x"], s["block"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"], scale=s["scale"], eps=EPS))
        if op == "norm_bwd":
            return _given(*g.residual_norm_backward(s["dy"], s["dn"], s["y"], s["block"], s["rstd_post"], s["rstd_pre"], w_post=s["w_post"],
                                                    gate=s["gate"], w_pre=s["w_pre"], scale=s["scale"]))
        if op == "w4":
            return g.gemv_w4a16(s["A"], s["b"], s["sf"], s["scale"])
        return g.gemv_w4a16_gated(s["A"], s["bg"], s["sfg"], s["scaleg"], s["bu"], s["sfu"], s["scaleu"], act=case["act"])
    if op == "gated_fwd":
        return _gated_fwd(s["X"], s["Wg"], s["Wu"], case["act"], case["gates"])
    if op == "gated_bwd":
        return _gated_bwd(s["X"], s["Wg"], s["Wu"], s["dH"], case["act"], s.get("gates"))
    if op == "tn":
        return _tn(s["A"], s["B"])
    if op == "norm_fwd":
        return _given(*_norm_fwd(s["x"], s["block"], s["w_post"], s["gate"], s["w_pre"], s["scale"]))
    if op == "norm_bwd":
        return _given(*_norm_bwd(s["dy"], s["dn"], s["y"], s["block"], s["rstd_post"], s["rstd_pre"], s["w_post"], s["gate"], s["w_pre"], s["scale"]))
    if op == "w4":
        return _w4(s["A"], s["b"], s["sf"], s["scale"]).bfloat16()
    return (_act(_w4(s["A"], s["bg"], s["sfg"], s["scaleg"]), case["act"]) * _w4(s["A"], s["bu"], s["sfu"], s["scaleu"])).bfloat16()


def work(case):
    """Inputs read once, outputs written once, and the products that a pass
    cannot do without (a backward pass without gates forms them again)."""
    op, M = case["op"], case["M"]
    if op.startswith("gated"):
        F, K = case["F"], case["K"]
        kept = 4 * M * F if case["gates"] else 0
        reads = 2 * M * K + 4 * F * K
        if op == "gated_fwd":
            return {"bytes": reads + 2 * M * F + kept, "flops": 4 * M * F * K}
        return {"bytes": 2 * reads + 2 * M * F + kept, "flops": (8 if case["gates"] else 12) * M * F * K}
    if op == "tn":
        N, K = case["N"], case["K"]
        return {"bytes": 2 * (M * K + N * K + M * N), "flops": 2 * M * N * K}
    if op.startswith("norm"):
        D, G = case["D"], case["groups"]
        wide = 4 if case["f32"] else 2
        norms, w = case["post"] + case["pre"], (case["post"] + case["pre"] + G) * D
        if op == "norm_fwd":
            return {"bytes": M * D * (2 * wide + 2 + 2 * case["pre"]) + 2 * w + 4 * M * norms, "flops": M * D * (3 + 4 * norms)}
        # dy, the stream and dn where there is a norm before the next block, the block's output; dx and db
        return {"bytes": M * D * (2 * wide + 4 + (wide + 2) * case["pre"]) + 6 * w + 4 * M * norms, "flops": M * D * (4 + 9 * norms)}
    N, K, two = case["N"], case["K"], 2 if op == "w4_gated" else 1
    return {"bytes": two * N * (K // 2 + K // 16) + 2 * M * K + 2 * M * N, "flops": 2 * two * M * N * K}


# ------------------------------------------------------------------ 64 bits
def _exact_gate(g, act):
    """act and its derivative, through the hyperbolic tangent."""
    if act == "silu":
        t = torch.tanh(0.5 * g)
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.25 * g * (1.0 - t * t)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 0.134145 * g * g)


def _exact_gated(case, s):
    X, act = s["X"].to(F64), case["act"]
    parts = [[] for _ in range(4)]
    dX = torch.zeros_like(X)
    step = 2048
    for f in range(0, case["F"], step):
        wg, wu = s["Wg"][f:f + step].to(F64), s["Wu"][f:f + step].to(F64)
        if case["op"] == "gated_bwd" and case["gates"]:
            g, u = s["gates"][:, :, f:f + step].to(F64)
        else:
            g, u = torch.mm(X, wg.t()), torch.mm(X, wu.t())
        a, slope = _exact_gate(g, act)
        if case["op"] == "gated_fwd":
            for out, t in zip(parts, (a * u, g, u)):
                out.append(t)
            continue
        d = s["dH"][:, f:f + step].to(F64)
        dg, du = d * u * slope, d * a
        dX += torch.mm(dg, wg) + torch.mm(du, wu)
        parts[0].append(torch.mm(dg.t(), X))
        parts[1].append(torch.mm(du.t(), X))
    if case["op"] == "gated_bwd":
        return [dX, torch.cat(parts[0]), torch.cat(parts[1])]
    H = torch.cat(parts[0], dim=1)
    return [H, torch.stack([torch.cat(parts[1], dim=1), torch.cat(parts[2], dim=1)])] if case["gates"] else [H]


def _wide(t):
    return None if t is None else t.to(F64)


def _exact_norm(case, s):
    M, D, G = case["M"], case["D"], case["groups"]
    b, wo, wi, gate = s["block"].to(F64), _wide(s["w_post"]), _wide(s["w_pre"]), _wide(s["gate"])
    per_row = None if gate is None else gate[torch.arange(M, device=b.device) // (M // G)]
    if case["op"] == "norm_fwd":
        out = {}
        if wo is not None:
            out["rstd_post"] = torch.rsqrt(b.pow(2).sum(dim=1) / D + EPS)
            b = torch.einsum("md,m,d->md", b, out["rstd_post"], wo)
        if gate is not None:
            b = b * per_row
        y = s["x"].to(F64) + s["scale"] * b
        if wi is not None:
            stored = y.to(s["x"].dtype).to(F64)
            out["rstd_pre"] = torch.rsqrt(stored.pow(2).sum(dim=1) / D + EPS)
            out["n"] = torch.einsum("md,m,d->md", stored, out["rstd_pre"], wi)
        return [y] + [out[k] for k in ("n", "rstd_post", "rstd_pre") if k in out]
    t, out = s["dy"].to(F64), {}
    if wi is not None:
        r, d = s["rstd_pre"].to(F64)[:, None], s["dn"].to(F64)
        hat = s["y"].to(F64) * r
        out["dw_pre"] = torch.einsum("md,md->d", d, hat)
        t = t + r * (d * wi - hat * torch.einsum("md,md,d->m", d, hat, wi)[:, None] / D)
    r = None if wo is None else s["rstd_post"].to(F64)[:, None]
    c = b if wo is None else b * r * wo
    dc = s["scale"] * t
    if gate is not None:
        out["dgate"] = torch.zeros_like(gate).index_add_(0, torch.arange(M, device=b.device) // (M // G), dc * c)
        dc = dc * per_row
    db = dc
    if wo is not None:
        hat = b * r
        out["dw_post"] = torch.einsum("md,md->d", dc, hat)
        db = r * (dc * wo - hat * torch.einsum("md,md,d->m", dc, hat, wo)[:, None] / D)
    return [t, db] + [out[k] for k in ("dw_pre", "dw_post", "dgate") if k in out]


def _exact_w4(case, s):
    def product(which):
        b, parts = s["b" + which], []
        for n in range(0, case["N"], 2048):
            rows = b[n:n + 2048].long()
            nibbles = torch.empty(rows.shape[0], case["K"], dtype=torch.long, device=b.device)
            nibbles[:, 0::2], nibbles[:, 1::2] = rows % 16, rows // 16
            m, e, sign = nibbles % 2, (nibbles // 2) % 4, 1 - 2 * (nibbles // 8)
            value = sign.to(F64) * torch.where(e > 0, (2 + m).to(F64) * torch.exp2(e.to(F64) - 2.0), 0.5 * m.to(F64))
            f = s["sf" + which][n:n + 2048].long()
            fe, fm = f // 8, f % 8
            scales = torch.where(fe > 0, (8 + fm).to(F64) * torch.exp2(fe.to(F64) - 10.0), fm.to(F64) * 2.0 ** -9)
            w = (value.reshape(rows.shape[0], -1, 16) * scales[:, :, None]).reshape(rows.shape[0], -1)
            parts.append(torch.mm(s["A"].to(F64), w.t()))
        return s["scale" + which] * torch.cat(parts, dim=1)
    if case["op"] == "w4":
        return product("")
    return _exact_gate(product("g"), case["act"])[0] * product("u")


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tn":
        return torch.mm(s["A"].to(F64).t(), s["B"].to(F64))
    return (_exact_gated if op.startswith("gated") else _exact_norm if op.startswith("norm") else _exact_w4)(case, s)
