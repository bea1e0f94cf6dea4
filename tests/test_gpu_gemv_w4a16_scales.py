"""Products of few tokens whose tensor scale is large: what fits BF16 comes back, whatever
the magnitudes of the other tokens in the call."""
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


def case(M, N, K, top):
    """Token 0: 2^top where every weight is zero, else zeros; the others of about one."""
    gen = torch.Generator(device="cuda").manual_seed(K + M)
    A = torch.randn(M, K, generator=gen, device="cuda").to(BF16)
    b = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    sf = torch.randint(40, 72, (N, K // 16), generator=gen, device="cuda", dtype=torch.uint8)
    A[0], A[:, :2], b[:, 0] = 0, 0, 0
    A[0, 0] = 2.0 ** top
    return A, b, sf


# 2^scale times a sum of at most 2^12 stays within BF16's range; scales down to the least FP32 number
@pytest.mark.parametrize("top,scale", [(127, 80), (127, 110), (100, 100), (20, 110), (0, 110), (-120, 110), (127, -100), (127, -126), (127, -149)])
@pytest.mark.parametrize("M,N,K", [(1, 40, 256), (3, 40, 1024), (16, 33, 4096), (2, 2048, 2048)])
def test_plain(g, M, N, K, top, scale):
    A, b, sf = case(M, N, K, top)
    want, e = ref.few_tokens(A, b, sf, 2.0 ** scale)
    assert (want[0] == 0).all()
    # below the normal ranges: half of FP32's and of BF16's least steps
    ref.check(g.gemv_w4a16(A, b, sf, 2.0 ** scale), want, e * (1 + ref.BF16_HALF) + ref.BF16_HALF * want.abs() + 2.0 ** -133, "C")


@pytest.mark.parametrize("scale", [-149, -140, -100, 0, 100, 126])
@pytest.mark.parametrize("magnitude", [-126, -100, -40, -30, 5, 40, 100, 120])
def test_all_tokens_of_one_magnitude(g, magnitude, scale):
    """Scales against tokens: the result within the range, below it or beyond it."""
    M, N, K = 4, 40, 1024
    A, b, sf = case(M, N, K, 0)
    A = (A.float() * 2.0 ** magnitude).to(BF16)
    want, e = ref.few_tokens(A, b, sf, 2.0 ** scale)
    got = g.gemv_w4a16(A, b, sf, 2.0 ** scale)
    bound = e * (1 + ref.BF16_HALF) + ref.BF16_HALF * want.abs() + 2.0 ** -133
    # (parts of a sum that leave the range make an infinity or NaN of it)
    parts = 2.0 ** scale * (A.to(ref.F64).abs() @ ref.nvfp4_weights(b, sf).abs().T)
    near = parts >= 2.0 ** 127
    assert not got[want.abs() >= 2.0 ** 129].isfinite().any()
    ref.check(torch.where(near, 0, got), torch.where(near, 0, want), bound, "C")


@pytest.mark.parametrize("top,scale", [(127, 80), (120, 105), (-120, 105)])
@pytest.mark.parametrize("M,F,K", [(1, 40, 256), (5, 24, 1024), (16, 520, 2048)])
def test_gated_by_a_large_factor(g, M, F, K, top, scale):
    A, b, sf = case(M, F, K, top)
    _, b2, sf2 = case(M, F, K, top)
    s_g = 2.0 ** -6
    want, e = ref.few_tokens_gated(A, b, sf, s_g, b2, sf2, 2.0 ** scale, "silu")
    assert (want[0] == 0).all()
    ref.check(g.gemv_w4a16_gated(A, b, sf, s_g, b2, sf2, 2.0 ** scale), want, e + 2.0 ** -133, "H")
