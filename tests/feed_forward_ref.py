"""64-bit references of the feed-forward block's operators, and error bounds
derived from the number formats (none is fitted to a result).

A rounding to BF16 is off by at most 2^-8 of the value (half a step), to FP32 by
2^-24.  The tensor core may truncate what it adds into the accumulator: 2^-23 of
the running sum per 16 products, and the running sum is at most the sum of the
products' magnitudes.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64
BF16_HALF = 2.0 ** -8


def act(g, kind):
    """(act(g), act'(g)) through the hyperbolic tangent."""
    if kind == "silu":
        t = torch.tanh(g / 2)
        return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) / 4
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) / 2 * c * (1 + 3 * 0.044715 * g * g)


# The activation's FP32 evaluation: the exponent's argument z (three roundings and
# a constant's) is off by 2^-21 |z|, which moves s(z) by s (1 - s) 2^-21 |z| <=
# 2^-21 * 0.23; the two special-function operations and the sum add 2^-21 of s.
# act = x s and act' = s + x s (1 - s) z' with (1 - s) |z| < 1.3 stay within
ACT_REL = 2.0 ** -18     # of |x| s, and of s + |x| s (1 - s) z'
SLOPE_MAX = 1.2          # |act'| of both kinds


def acc_bound(K, mags):
    """Error of an FP32 accumulation of K products whose magnitudes sum to mags."""
    return (K / 16 + 4) * 2.0 ** -23 * mags


def gated(X, Wg, Wu, kind):
    """(H, G, U) and their error bounds, before H's rounding is counted."""
    x, wg, wu = X.to(F64), Wg.to(F64), Wu.to(F64)
    G, U = x @ wg.T, x @ wu.T
    a, _ = act(G, kind)
    K = X.shape[1]
    eg, eu = acc_bound(K, x.abs() @ wg.abs().T), acc_bound(K, x.abs() @ wu.abs().T)
    H = a * U
    ea = SLOPE_MAX * eg + ACT_REL * G.abs()
    eh = ea * (U.abs() + eu) + a.abs() * eu
    return H, G, U, eh * (1 + BF16_HALF) + BF16_HALF * H.abs(), eg * (1 + BF16_HALF) + BF16_HALF * G.abs(), eu * (1 + BF16_HALF) + BF16_HALF * U.abs()


def gated_backward(X, Wg, Wu, dH, kind, gates=None):
    """(dX, dWg, dWu) and their error bounds."""
    x, wg, wu, dh = X.to(F64), Wg.to(F64), Wu.to(F64), dH.to(F64)
    M, K = X.shape
    F = Wg.shape[0]
    if gates is None:
        G, U = x @ wg.T, x @ wu.T
        eg, eu = acc_bound(K, x.abs() @ wg.abs().T), acc_bound(K, x.abs() @ wu.abs().T)
    else:
        G, U = gates[0].to(F64), gates[1].to(F64)
        eg = eu = torch.zeros_like(G)
    a, slope = act(G, kind)
    dG, dU = dh * U * slope, dh * a
    # the slope changes by at most 1.2 |dg| (its own derivative is below 1.2 for both kinds)
    e_slope = 1.2 * eg + ACT_REL * (1 + G.abs())
    e_act = SLOPE_MAX * eg + ACT_REL * G.abs()
    edG = dh.abs() * (e_slope * (U.abs() + eu) + slope.abs() * eu)
    edU = dh.abs() * e_act
    edG, edU = edG * (1 + BF16_HALF) + BF16_HALF * dG.abs(), edU * (1 + BF16_HALF) + BF16_HALF * dU.abs()
    dX, dWg, dWu = dG @ wg + dU @ wu, dG.T @ x, dU.T @ x

    def out(value, carried, mags, n):
        e = carried + acc_bound(n, mags + carried)
        return e * (1 + BF16_HALF) + BF16_HALF * value.abs()
    eX = out(dX, edG @ wg.abs() + edU @ wu.abs(), dG.abs() @ wg.abs() + dU.abs() @ wu.abs(), 2 * F)
    eWg = out(dWg, edG.T @ x.abs(), dG.abs().T @ x.abs(), M)
    eWu = out(dWu, edU.T @ x.abs(), dU.abs().T @ x.abs(), M)
    return (dX, dWg, dWu), (eX, eWg, eWu)


def check(got, want, bound, what):
    """Every element within its bound."""
    off = (got.to(F64) - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        at = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds; first {at}: "
                             f"{float(got[at])} instead of {float(want[at])}, allowed {float(bound[at])}")


# ------------------------------------------------------------------ residual step
# A row's sum: a thread adds at most 32 terms, a warp's tree 5, the warps 16, all
# FP32: below 2^-18 of the sum of magnitudes, products and a division included.
ROW_SUM = 2.0 ** -18


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rows_of(gate, M):
    g = gate.to(F64).reshape(-1, gate.shape[-1])
    return g.repeat_interleave(M // g.shape[0], dim=0)


def norm(x, block, w_post, gate, w_pre, scale, eps, stored):
    """y, n, rstd_post, rstd_pre and the bounds of y, n; n is of the stream as `stored`."""
    b, y, ey, r_post = None, x.to(F64), torch.zeros_like(x, dtype=F64), None
    if block is not None:
        c = block.to(F64)
        if w_post is not None:
            r_post = torch.rsqrt((c * c).mean(dim=1) + eps)
            c = c * r_post[:, None] * w_post.to(F64)
        if gate is not None:
            c = c * rows_of(gate, x.shape[0])
        # the norm's scale, then four products and a sum in FP32, then the stored type
        y = y + scale * c
        ey = (ROW_SUM + 2.0 ** -21) * (scale * c).abs() + (2.0 ** -24 + half_step(x.dtype)) * (y.abs() + (scale * c).abs() * 2.0 ** -17)
    n = en = r_pre = None
    if w_pre is not None:
        s = stored.to(F64)
        r_pre = torch.rsqrt((s * s).mean(dim=1) + eps)
        n = s * r_pre[:, None] * w_pre.to(F64)
        en = (ROW_SUM + 2.0 ** -22 + BF16_HALF) * n.abs()
    return y, n, r_post, r_pre, ey, en


def norm_backward(dy, dn, y, block, r_post, r_pre, w_post, gate, w_pre, scale, dtype):
    """{name: (value, bound)} of residual_norm_backward."""
    like = dy if dy is not None else y
    M, D = like.shape
    t = torch.zeros(M, D, dtype=F64, device=like.device) if dy is None else dy.to(F64)
    mag, et, out = t.abs(), torch.zeros_like(t), {}
    sums = (M / 300 + 64) * 2.0 ** -24  # rows of a run, the runs that a warp joins, the warps
    e, yh, m1 = torch.zeros_like(t), torch.zeros_like(t), torch.zeros_like(t[:, :1])
    abs_eyh = m1
    if w_pre is not None:
        r = r_pre.to(F64)[:, None]
        yh, d = y.to(F64) * r, dn.to(F64)
        out["dw_pre"] = ((d * yh).sum(dim=0), (sums + 2.0 ** -22) * (d * yh).abs().sum(dim=0))
        e = d * w_pre.to(F64)
        m1 = (e * yh).mean(dim=1, keepdim=True)
        abs_eyh = (e * yh).abs().mean(dim=1, keepdim=True)
        t = t + r * (e - yh * m1)
        mag = mag + r * e.abs()
        et = 2.0 ** -20 * (mag + r * (yh * m1).abs()) + r * yh.abs() * ROW_SUM * abs_eyh
        e, m1, abs_eyh = r * e, r * m1, r * abs_eyh
    out["dx"] = (t, et + half_step(dtype) * (t.abs() + et))
    if block is None:
        return out
    g = torch.ones_like(t) if gate is None else rows_of(gate, M)
    q = scale * g * t
    eq = (scale * g).abs() * et + 2.0 ** -21 * q.abs()
    bh, w = block.to(F64), torch.ones_like(t[0])
    if w_post is not None:
        r, w = r_post.to(F64)[:, None], w_post.to(F64)
        bh = bh * r
        p = (scale * g * w * bh).abs()
        m2 = (q * w * bh).mean(dim=1, keepdim=True)
        e_m2 = 2 * ROW_SUM * ((p * mag).mean(dim=1, keepdim=True) +
                              (m1.abs() + abs_eyh) * (p * yh.abs()).mean(dim=1, keepdim=True))
        db = r * (q * w - bh * m2)
        edb = r * (w.abs() * eq + bh.abs() * e_m2) + 2.0 ** -20 * r * ((q * w).abs() + (bh * m2).abs())
        out["dw_post"] = ((q * bh).sum(dim=0), (sums + 2.0 ** -21) * (q * bh).abs().sum(dim=0) + (bh.abs() * eq).sum(dim=0))
    else:
        db, edb = q, eq
    out["dblock"] = (db, edb + BF16_HALF * (db.abs() + edb))
    if gate is not None:
        c = bh * w
        groups = gate.reshape(-1, D).shape[0]
        shape = (groups, M // groups, D)
        v = scale * t * c
        ev = (sums + 2.0 ** -21) * v.abs() + abs(scale) * c.abs() * et
        # a group whole within a run: its rows are added one after the other
        ev = ev + M / groups * 2.0 ** -24 * v.abs() if groups > 1 else ev
        out["dgate"] = (v.reshape(shape).sum(dim=1).reshape(gate.shape), ev.reshape(shape).sum(dim=1).reshape(gate.shape))
    return out


# ------------------------------------------------------------------ 4-bit weights
def nvfp4_weights(b, sf):
    """e2m1 * e4m3 in 64 bits, decoded from the formats' fields."""
    codes = torch.stack([b % 16, b // 16], dim=2).reshape(b.shape[0], -1).long()
    m, e, s = codes % 2, codes // 2 % 4, 1 - 2 * (codes // 8)
    value = s.to(F64) * torch.where(e > 0, (1 + m.to(F64) / 2) * 2.0 ** (e.to(F64) - 1), m.to(F64) / 2)
    f = sf.long()
    fm, fe, fs = f % 8, f // 8 % 16, 1 - 2 * (f // 128)
    scale = fs.to(F64) * torch.where(fe > 0, (1 + fm.to(F64) / 8) * 2.0 ** (fe.to(F64) - 7), fm.to(F64) * 2.0 ** -9)
    scale = torch.where(f % 128 == 127, torch.full_like(scale, float("nan")), scale)
    return value * scale.repeat_interleave(16, dim=1)


def few_tokens(A, b, sf, scale2):
    """(scale2 A w^T, error bound of its FP32 form)."""
    w, a = nvfp4_weights(b, sf), A.to(F64)
    v = scale2 * (a @ w.T)
    # the accumulator, the halves and splits of K, the scale
    return v, acc_bound(A.shape[1] + 16 * 20, abs(scale2) * (a.abs() @ w.abs().T)) + 2.0 ** -23 * v.abs()


def few_tokens_gated(A, bg, sfg, s_g, bu, sfu, s_u, kind):
    (G, eg), (U, eu) = few_tokens(A, bg, sfg, s_g), few_tokens(A, bu, sfu, s_u)
    a, _ = act(G, kind)
    ea = SLOPE_MAX * eg + ACT_REL * G.abs()
    H = a * U
    eh = ea * (U.abs() + eu) + a.abs() * eu + 2.0 ** -23 * H.abs()
    return H, eh * (1 + BF16_HALF) + BF16_HALF * H.abs()
