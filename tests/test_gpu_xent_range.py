"""Linear cross entropy of finite logits near the largest FP32 value, on either
side of the row count where the tokens change to the MMA's other side."""
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


ROWS = [7, 100, 128, 129, 300]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("top,others", [
    (1.6, 1.4),     # a maximum of 2.7e38, the others far below it
    (1.6, -1.6),    # the difference of two logits passes the FP32 range
    (-1.4, -1.6),   # every logit near the lowest value
    (1.6, 0.0),
])
def test_finite_logits_near_the_end_of_the_range(g, M, top, others):
    # one product per logit, exact in FP32: z = 2^127 w, w with BF16's 8 bits
    V, K, at = 300, 64, 211
    X = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    X[:, 3] = 2.0 ** 127
    W = torch.zeros(V, K, device="cuda", dtype=torch.bfloat16)
    W[:, 3] = others
    W[at, 3] = top
    t = torch.full((M,), at, device="cuda")
    t[0] = 5
    loss, lse = g.gemm_bf16_nt_xent(X, W, t)
    z = X.to(F64) @ W.to(F64).T
    assert (z.abs() < torch.finfo(torch.float32).max).all()
    want = z.amax(dim=1)                        # the others are further than any bit of it
    assert torch.equal(lse.to(F64), want)
    pick = z.gather(1, t[:, None])[:, 0]
    # the difference of lse and the target's logit, rounded to FP32
    assert torch.equal(loss, (want - pick).float())
    d = torch.linspace(0.5, 2.0, M, device="cuda")
    # G: d at the certain class minus d at the target, so rows but the first are 0
    dX, dW = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    assert (dX[1:] == 0).all()
    gx = d[0].to(F64) * (W[at].to(F64) - W[5].to(F64))
    assert ((dX[0].to(F64) - gx).abs() <= 2.0 ** -7 * (W[at].abs() + W[5].abs()).to(F64)).all()
    assert torch.isfinite(dW).all()
    cols = torch.arange(V, device="cuda")
    assert (dW[(cols != at) & (cols != 5)] == 0).all()
    assert dW[at, 3] > 0 and dW[5, 3] == -dW[at, 3]
