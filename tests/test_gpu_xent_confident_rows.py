"""Accuracy of the linear cross entropy where its terms cancel: long K loops and
rows whose target is nearly certain, against 64 bits.

Inputs.  W's rows have norm about 2 and X's about 2 sqrt(K), so the other
logits spread by 4; each row of X then gets as much of its target's row of W as
brings the target's logit to 22..30, which leaves it 1 - p of about 1e-2 down
to 1e-6.

Tolerances.  The tensor core drops what falls below 2^-24 of its running sum, 16
products at a time.  Half of a unit is lost on average, and a unit is 0.72 of
2^-24 of the value on average over the binades, so a running sum that grows
evenly loses (steps / 2) (0.72 / 2) 2^-24 of its end value: with 4096 products
256 steps, 2.7e-6; with chunks of 1024, 64 steps, 6.9e-7; with chunks of 256,
16 steps, 1.7e-7.  Adding the chunks and storing lse round by 2^-25 of their
value each, at random: sqrt(chunks) 2^-25 at most, 1.2e-7 for 16.  lse may be
off by twice the sum of the two, root mean square over the rows.

Gradient.  The passes form the same logits, so of z - lse only lse's own
rounding is left: 2^-20 for lse < 32 (its storing), 2^-19 (fewer than 32
additions at or above 1 on the way to the sum, each off by 2^-24), 2^-19 (the
exponent's product below 64 is rounded, times log 2) and 2^-22 (the
exponential): `delta`.  The drift of
the logits moves p by p (1 - p) times twice (K / 16) 2^-23 of the largest
running sum, 40 (`zeta`, the worst case: it vanishes with 1 - p).  G's rounding
to BF16 (8 bits) is at most 2^-8 of its size, 1.01 with what it rounds, the
result's the same, and the products' sums are FP32.  Every bound is taken element by
element.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_tcgen05_gb300 as lib
    yield lib
    assert lib.gemm_get_device_status() == 0


def learned_rows(M, V, K, seed):
    """X, W, target on the CPU."""
    gen = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, K, generator=gen) * (2 / K ** 0.5)).bfloat16()
    X = 2 * torch.randn(M, K, generator=gen)
    t = torch.randint(0, V, (M,), generator=gen)
    w = W[t].float()
    goal = 22 + 8 * torch.rand(M, generator=gen)
    part = (goal - (X * w).sum(1)) / (w * w).sum(1)
    return (X + part[:, None] * w).bfloat16(), W, t


def exact(X, W, t):
    z = X.to(F64) @ W.to(F64).T
    lse = torch.logsumexp(z, dim=1)
    # 1 - p of the target without cancellation: the sum over the others
    others = z.scatter(1, t[:, None], float("-inf"))
    return z, lse, torch.exp(torch.logsumexp(others, dim=1) - lse)


CASES = [(48, 2000, 4096), (100, 1999, 4096), (300, 2000, 4096), (200, 1500, 7168)]


@pytest.mark.parametrize("M,V,K", CASES)
def test_lse(g, M, V, K):
    X, W, t = (a.cuda() for a in learned_rows(M, V, K, 7 + M))
    loss, lse = g.gemm_bf16_nt_xent(X, W, t)
    _, want, _ = exact(X, W, t)
    chunk = 256 if M <= 128 else 1024
    drift = chunk / 16 / 2 * 0.72 / 2 * 2.0 ** -24
    rounding = ((K + chunk - 1) // chunk) ** 0.5 * 2.0 ** -25
    err = ((lse.to(F64) - want) / want).square().mean().sqrt()
    assert err <= 2 * (drift + rounding)


@pytest.mark.parametrize("M,V,K", CASES)
def test_gradients(g, M, V, K):
    X, W, t = (a.cuda() for a in learned_rows(M, V, K, 7 + M))
    d = torch.linspace(0.5, 1.5, M, device="cuda")
    _, lse = g.gemm_bf16_nt_xent(X, W, t)
    dX, dW = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    z, want_lse, rest = exact(X, W, t)
    assert (want_lse < 32).all()
    # enough rows whose target's gradient d (p - 1) the error of p could swamp
    assert ((rest > 1e-5) & (rest < 1e-3)).sum() >= M // 4
    p = torch.exp(z - want_lse[:, None])
    at = torch.arange(M, device="cuda"), t
    coeff = p.clone()
    coeff[at] = -rest
    G = coeff * d.to(F64)[:, None]
    delta = 2.0 ** -20 + 2.0 ** -19 + 2.0 ** -19 + 2.0 ** -22
    zeta = 2 * (K / 16) * 2.0 ** -23 * 40
    q = 1 - p
    q[at] = rest
    err = d.to(F64)[:, None] * p * (delta + zeta * q) + 1.01 * 2.0 ** -8 * G.abs()
    x, w = X.to(F64), W.to(F64)
    for got, want, bound in (
            (dX, G @ w, err @ w.abs() + (V + 64) * 2.0 ** -23 * (G.abs() @ w.abs())),
            (dW, G.T @ x, err.T @ x.abs() + (M + 64) * 2.0 ** -23 * (G.abs().T @ x.abs()))):
        assert ((got.to(F64) - want).abs() <= bound + 1.01 * 2.0 ** -8 * want.abs() + 1e-30).all()
