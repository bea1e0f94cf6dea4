"""Outputs whose last column block leaves some of an epilogue warp's store boxes
unused: the box that the next tile takes must not be one that a store still
reads.  Short K loops bring the next tile soon; every call is compared with the
first one bit for bit and with the product in 64 bits."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_tcgen05_gb300 as lib
    yield lib
    assert lib.gemm_get_device_status() == 0


def check(call, want, rows=512):
    first = call()
    # BF16 rounding of an FP32 sum of 64 products of order 1
    err = (first[:rows].double() - want[:rows]).abs()
    assert (err <= 2.0 ** -8 * want[:rows].abs() + 2.0 ** -16).all()
    for _ in range(15):
        assert torch.equal(call(), first)


# 3, 1 and 2 of the last block's four 64-column boxes; a block of 192 columns
@pytest.mark.parametrize("N", [952, 776, 872, 712])
@pytest.mark.parametrize("M", [40000, 20100])
def test_bf16_products(g, M, N):
    K = 64
    gen = torch.Generator(device="cuda").manual_seed(N)
    A = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    B = torch.randn(N, K, generator=gen, device="cuda").bfloat16()
    want = A[:512].double() @ B.double().T
    check(lambda: g.gemm_bf16_nt(A, B), want)
    Bt = B.T.contiguous()
    check(lambda: g.gemm_bf16_nn(A, Bt), want)
    check(lambda: g.gemm_bf16_nt_splitk(A, B, 1), want)


@pytest.mark.parametrize("M,V,K", [(300, 20000, 952), (247, 39280, 952), (140, 30000, 712), (600, 20000, 776)])
def test_xent_gradients(g, M, V, K):
    gen = torch.Generator(device="cuda").manual_seed(V)
    X = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    W = (torch.randn(V, K, generator=gen, device="cuda") * (2 / K ** 0.5)).bfloat16()
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    d = torch.rand(M, generator=gen, device="cuda")
    _, lse = g.gemm_bf16_nt_xent(X, W, t)
    dX, dW = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    for i in range(40):
        if i % 2:
            torch.randn(1 << 20, device="cuda")       # other work between the calls
        again = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
        assert torch.equal(again[0], dX) and torch.equal(again[1], dW)
