"""A row whose loss has gradient zero beside a logit that is not finite, on either
side of the row count where the tokens change to the MMA's other side."""
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


ROWS = [7, 100, 128, 129, 300]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_gradient_zero_beside_a_logit_that_is_not_finite(g, M, bad):
    # 0 times NaN: the row has a target, so its gradient is NaN as the formula's,
    # however many rows there are; a row without a target has none
    gen = torch.Generator(device="cuda").manual_seed(M)
    V, K = 500, 64
    X = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    W = (torch.randn(V, K, generator=gen, device="cuda") / 4).bfloat16()
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    d = torch.rand(M, generator=gen, device="cuda") + 0.5
    X[2, 5] = bad
    d[2] = d[4] = 0.0                           # row 4 is an ordinary one
    t[3] = -1
    X[3, 5] = bad
    _, lse = g.gemm_bf16_nt_xent(X, W, t)
    assert torch.isnan(lse[2])                  # both signs occur among its logits
    dX, _ = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d, need_dw=False)
    assert torch.isnan(dX[2]).all()
    assert (dX[3] == 0).all() and (dX[4] == 0).all()
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[2] = False
    assert torch.isfinite(dX[rest]).all()
