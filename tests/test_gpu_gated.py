"""The gated projection H = act(X Wg^T) * (X Wu^T), its gradients, and the weight
gradient A^T B, against 64-bit references."""
from __future__ import annotations

import pytest
import torch

import feed_forward_ref as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_tcgen05_gb300 as g
    yield g
    assert g.gemm_get_device_status() == 0


def randn(seed, *shape, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(BF16)


def inputs(M, F, K, seed=0):
    return (randn(seed, M, K), randn(seed + 1, F, K, scale=2.0 / K ** 0.5),
            randn(seed + 2, F, K, scale=1.5 / K ** 0.5), randn(seed + 3, M, F, scale=0.1))


# one token, few, a tile's edges, odd sizes; K below, at and past a stage of 128
SIZES = [(1, 8, 8), (1, 136, 72), (5, 1032, 256), (33, 264, 2056), (64, 248, 640), (65, 504, 136), (127, 128, 64),
         (128, 264, 392), (129, 248, 136), (256, 256, 128), (300, 1032, 520), (513, 392, 1000), (1100, 2568, 264)]
# few tokens: warps with no step, part of a tile, whole tiles; every count of token groups;
# tokens that shared memory holds, and not; long runs with more than 16 tokens, and not
SIZES += [(2, 136, 1032), (3, 9736, 1096), (8, 2056, 520), (9, 16392, 264), (16, 264, 5816), (16, 264, 6008),
          (17, 136, 72), (20, 9736, 1096), (32, 1032, 2824), (32, 520, 3064)]


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F,K", SIZES)
def test_forward(g, M, F, K, kind):
    X, Wg, Wu, _ = inputs(M, F, K)
    H, G, U, eh, eg, eu = ref.gated(X, Wg, Wu, kind)
    got, none = g.gemm_bf16_nt_gated(X, Wg, Wu, act=kind)
    assert none is None and got.dtype == BF16
    ref.check(got, H, eh, "H")
    got2, gates = g.gemm_bf16_nt_gated(X, Wg, Wu, act=kind, save_gates=True)
    ref.check(got2, H, eh, "H beside the gates")
    ref.check(gates[0], G, eg, "gate")
    ref.check(gates[1], U, eu, "up")


@pytest.mark.parametrize("kept", [True, False], ids=["gates", "from_x"])
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F,K", SIZES)
def test_backward(g, M, F, K, kind, kept):
    X, Wg, Wu, dH = inputs(M, F, K, seed=10)
    gates = g.gemm_bf16_nt_gated(X, Wg, Wu, act=kind, save_gates=True)[1] if kept else None
    want, bound = ref.gated_backward(X, Wg, Wu, dH, kind, gates)
    got = g.gemm_bf16_nt_gated_backward(X, Wg, Wu, dH, act=kind, gates=gates)
    for t, w, e, name in zip(got, want, bound, ("dX", "dWg", "dWu")):
        ref.check(t, w, e, name)
    # one side alone gives the same bits
    dx = g.gemm_bf16_nt_gated_backward(X, Wg, Wu, dH, act=kind, gates=gates, need_dw=False)
    dw = g.gemm_bf16_nt_gated_backward(X, Wg, Wu, dH, act=kind, gates=gates, need_dx=False)
    assert dx[1] is None and dx[2] is None and dw[0] is None
    assert torch.equal(dx[0], got[0]) and torch.equal(dw[1], got[1]) and torch.equal(dw[2], got[2])


@pytest.mark.parametrize("M,N,K", [(8, 8, 1), (136, 72, 1), (128, 256, 3), (264, 520, 100), (256, 256, 128), (1000, 248, 129),
                                   (520, 2056, 777), (2048, 1032, 4096), (8, 16, 5000), (512, 520, 4097),
                                   (1024, 1288, 2500)])
def test_tn(g, M, N, K):
    A, B = randn(3, K, M), randn(4, K, N)
    want = A.to(ref.F64).T @ B.to(ref.F64)
    e = ref.acc_bound(K, A.to(ref.F64).abs().T @ B.to(ref.F64).abs())
    ref.check(g.gemm_bf16_tn(A, B), want, e * (1 + ref.BF16_HALF) + ref.BF16_HALF * want.abs(), "C")
