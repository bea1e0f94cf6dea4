"""The gated projection's activation and slope far from zero, every kernel that forms them:
the negative tail relative to its own size, and finite gates of any size, where the slope is
1 or 0."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
HALF = 2.0 ** -8  # a rounding to BF16


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_tcgen05_gb300 as g
    yield g
    assert g.gemm_get_device_status() == 0


def act(x, kind):
    """act(x), act'(x) and bounds of their FP32 evaluation, from s(z) = 1 / (1 + exp(-z)).

    z (silu: a constant and a product; gelu: three constants, two squares' products, a sum and a
    product) is off by at most 2^-21 |z|, which moves s by (1 - s) of that, relative to s; the
    exponential is good to 2^-22 (and zero below 2^-126, infinite from 2^128), the sum and the
    reciprocal to 2^-22 together; they are exact where the exponential is below 2^-25.
    """
    if kind == "silu":
        z, dz = x, torch.ones_like(x)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        z, dz = c * (x + 0.044715 * x ** 3), c * (1 + 3 * 0.044715 * x * x)
    s, r = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))  # r = 1 - s
    part = torch.where(s * r == 0, 0.0, s * r * dz * x.abs())
    slope = s + torch.sign(x) * part
    es = torch.where(z > 18.1, 0.0, r * (z.abs() * 2.0 ** -21 + 2.0 ** -22) + 2.0 ** -22)
    es = torch.where(z.isinf() & (z < 0), 0.0, es)  # s is zero
    lost = 2.0 ** -125  # an s below the normal range
    e_act = x.abs() * s * (es + 2.0 ** -24) + torch.where(z < -80, x.abs().clamp(max=100) * lost, 0.0)
    # x s (1 - s) z': the errors of s, of 1 - s (absolute, s es and a rounding), and four more roundings
    dz_x = torch.where(s * r == 0, 0.0, x.abs() * dz * s)
    e_slope = s * (es + 2.0 ** -24) + part * (es + 2.0 ** -21) + dz_x * s * (es + 2.0 ** -24)
    e_slope = e_slope + torch.where(z < -80, (1 + (x.abs() * dz).clamp(max=1000)) * lost, 0.0)
    return x * s, slope, e_act, e_slope


TAIL = [-0.5, -1.0, -1.25, -2.0, -3.0, -4.0, -5.0, -6.0, -7.0, -8.0, -9.0, -10.0, -12.0, -16.0, -20.0, -24.0, -30.0, -40.0, -60.0, -80.0, -86.0, -90.0]
FAR = [0.0, 0.75, 3.0, 5.0, 8.0, 17.0, 30.0, 100.0, 1e4, 1e10, 1.5e19, 2e19, 1e30, 3e38]
VALUES = TAIL + FAR + [-v for v in FAR]


def inputs(M):
    """G[m, 0] = gate m, U[m, 0] = 1, zeros elsewhere, all exact; dH = 1."""
    gates = torch.tensor([VALUES[m % len(VALUES)] for m in range(M)], dtype=F64, device="cuda").to(BF16)
    X, Wg, Wu = (torch.zeros(n, 16, dtype=BF16, device="cuda") for n in (M, 24, 24))
    X[:, 0], X[:, 1] = gates, 1.0
    Wg[0, 0] = Wu[0, 1] = 1.0
    return gates.to(F64), X, Wg, Wu, torch.ones(M, 24, dtype=BF16, device="cuda")


def check(got, want, e, kind, gates, what):
    bound = e * (1 + HALF) + HALF * want.abs() + 2.0 ** -134
    bad = ~((got.to(F64) - want).abs() <= bound)
    assert not bad.any(), f"{what} {kind}: " + ", ".join(
        f"gate {float(gates[m])}: {float(got[m])} instead of {float(want[m])}" for m in torch.nonzero(bad)[:, 0].tolist()[:4])


# the kernels' limits: 16, 32 and 128 tokens (and with M = 300 every value in one call)
SIZES = [1, 8, 16, 17, 32, 33, 50, 64, 65, 100, 128, 129, 300]


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M", SIZES)
def test_forward(g, M, kind):
    for shift in range(0, len(VALUES), max(M, 1)):
        gates, X, Wg, Wu, _ = inputs(M + shift)
        gates, X = gates[shift:], X[shift:].contiguous()
        a, _, e, _ = act(gates, kind)
        H = g.gemm_bf16_nt_gated(X, Wg, Wu, act=kind)[0]
        assert (H[:, 1:] == 0).all()
        check(H[:, 0], a, e, kind, gates, "H")


@pytest.mark.parametrize("kept", [True, False], ids=["gates", "from_x"])
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M", SIZES)
def test_backward(g, M, kind, kept):
    for shift in range(0, len(VALUES), max(M, 1)):
        gates, X, Wg, Wu, dH = inputs(M + shift)
        gates, X, dH = gates[shift:], X[shift:].contiguous(), dH[shift:].contiguous()
        a, slope, ea, es = act(gates, kind)
        both = g.gemm_bf16_nt_gated(X, Wg, Wu, act=kind, save_gates=True)[1] if kept else None
        dX = g.gemm_bf16_nt_gated_backward(X, Wg, Wu, dH, act=kind, gates=both, need_dw=False)[0]
        # one product each: dG[m, 0] in column 0, dU[m, 0] in column 1
        check(dX[:, 0], slope, es, kind, gates, "dG")
        check(dX[:, 1], a, ea, kind, gates, "dU")
        assert (dX[:, 2:] == 0).all()


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_four_bit_weights(g, kind):
    """gemv_w4a16_gated: the gate through the tokens, factors of one."""
    K, F = 256, 8
    b = torch.zeros(2, F, K // 2, dtype=torch.uint8, device="cuda")
    b[0, 0, 0], b[1, 0, 0] = 0x02, 0x20  # 1.0 at k = 0, and at k = 1
    sf = torch.full((F, K // 16), 0x38, dtype=torch.uint8, device="cuda")
    for first in range(0, len(VALUES), 16):
        vals = torch.tensor(VALUES[first:first + 16], dtype=F64, device="cuda").to(BF16)
        A = torch.zeros(len(vals), K, dtype=BF16, device="cuda")
        A[:, 0], A[:, 1] = vals, 1.0
        gates = vals.to(F64)
        a, _, e, _ = act(gates, kind)
        H = g.gemv_w4a16_gated(A, b[0], sf, 1.0, b[1], sf, 1.0, act=kind)
        assert (H[:, 1:] == 0).all()
        check(H[:, 0], a, e, kind, gates, "H")
