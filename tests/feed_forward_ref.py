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
