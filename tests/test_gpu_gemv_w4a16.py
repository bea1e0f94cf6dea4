"""Products of 1 to 16 tokens with NVFP4 weights, plain and gated, against 64-bit
references and against gemm_w4a16."""
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


def weights(N, K, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    b = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    # every e4m3 value but NaN, both signs
    sf = torch.randint(0, 127, (N, K // 16), generator=gen, device="cuda", dtype=torch.uint8)
    sf += 128 * torch.randint(0, 2, (N, K // 16), generator=gen, device="cuda", dtype=torch.uint8)
    return b, sf


def tokens(M, K, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(M, K, generator=gen, device="cuda").to(BF16)


# rows: one, a tile's edges, several tiles to an SM, more than a block holds at a time;
# K: the least, odd multiples, more than a block's tokens
SIZES = [(1, 70001, 256), (16, 40003, 256), (1, 24, 131072), (3, 50, 98304), (16, 9, 65536), (1, 1, 256), (1, 8, 256), (2, 15, 512), (3, 16, 768), (5, 17, 256), (7, 63, 1280), (8, 64, 2048), (9, 65, 2304), (1, 2048, 11008),
         (16, 127, 16384), (11, 130, 3328), (15, 1000, 4096), (4, 10008, 512), (16, 20000, 768), (12, 33, 256)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_plain(g, M, N, K):
    A, (b, sf) = tokens(M, K, 1), weights(N, K, 2)
    want, e = ref.few_tokens(A, b, sf, 0.37)
    ref.check(g.gemv_w4a16(A, b, sf, 0.37), want, e * (1 + ref.BF16_HALF) + ref.BF16_HALF * want.abs(), "C")


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F,K", SIZES)
def test_gated(g, M, F, K, kind):
    A, (bg, sfg), (bu, sfu) = tokens(M, K, 3), weights(F, K, 4), weights(F, K, 5)
    s_g, s_u = 0.01 / K ** 0.5, -0.02 / K ** 0.5
    want, e = ref.few_tokens_gated(A, bg, sfg, s_g, bu, sfu, s_u, kind)
    ref.check(g.gemv_w4a16_gated(A, bg, sfg, s_g, bu, sfu, s_u, act=kind), want, e, "H")


@pytest.mark.parametrize("M", range(1, 17))
def test_exact_sums(g, M):
    """Small whole numbers: every sum is exact, so the result is the rounded one."""
    K, N = 1536, 200
    gen = torch.Generator(device="cuda").manual_seed(M)
    A = torch.randint(-4, 5, (M, K), generator=gen, device="cuda").to(BF16)
    b = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    sf = torch.randint(5, 9, (N, K // 16), generator=gen, device="cuda", dtype=torch.uint8) * 8  # 2^-2 .. 2
    want = (A.to(ref.F64) @ ref.nvfp4_weights(b, sf).T).to(torch.float32).to(BF16)
    got = g.gemv_w4a16(A, b, sf, 1.0)
    assert torch.equal(got, want)
    if N % 8 == 0:
        assert torch.equal(g.gemm_w4a16(A, b, sf, 1.0), want)


def test_nonfinite_values_stay_in_their_rows(g):
    A, (b, sf) = tokens(3, 512, 6), weights(40, 512, 7)
    clean = g.gemv_w4a16(A, b, sf, 1.0)
    A[1, 7] = float("inf")
    sf[5, 3] = 0x7F
    got = g.gemv_w4a16(A, b, sf, 1.0)
    assert got[:, 5].isnan().all()
    keep = [n for n in range(40) if n != 5]
    assert torch.equal(got[0, keep], clean[0, keep]) and torch.equal(got[2, keep], clean[2, keep])
    assert not got[1].isfinite().any()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K,spread", [(1, 40, 256, 30), (3, 40, 1024, 60), (9, 33, 2048, 120), (16, 100, 4096, 126), (2, 2048, 2048, 40)])
def test_tokens_of_any_magnitude(g, M, N, K, spread, gated):
    """Values from 2^-spread up to 2^spread in one row, some below the normal range: products stay exact."""
    gen = torch.Generator(device="cuda").manual_seed(K + spread)
    r = lambda *s: torch.rand(*s, generator=gen, device="cuda")
    A = ((1 + r(M, K)) * torch.exp2(torch.floor((2 * r(M, K) - 1) * spread)) * torch.where(r(M, K) < 0.5, -1.0, 1.0)).to(BF16)
    A[:, ::7] = 0
    A[0, 1] = 2.0 ** -130  # a subnormal
    (b, sf), (b2, sf2) = weights(N, K, 8), weights(N, K, 9)
    # the large values meet weights of zero in half of the rows: what is left is small
    big = A.abs().amax(dim=0) > 2.0 ** (spread / 3)
    codes = torch.stack([b % 16, b // 16], dim=2).reshape(N, K)
    codes[::2][:, big] = 0
    b = codes[:, ::2] + 16 * codes[:, 1::2]
    if gated:
        s = 2.0 ** -spread
        want, e = ref.few_tokens_gated(A, b, sf, s, b2, sf2, s * 2.0 ** -8, "silu")
        ref.check(g.gemv_w4a16_gated(A, b, sf, s, b2, sf2, s * 2.0 ** -8), want, e + 2.0 ** -130, "H")
    else:
        s = 2.0 ** -20  # results stay within BF16's range
        want, e = ref.few_tokens(A, b, sf, s)
        # below the normal ranges: half of FP32's and of BF16's least steps
        ref.check(g.gemv_w4a16(A, b, sf, s), want, e * (1 + ref.BF16_HALF) + ref.BF16_HALF * want.abs() + 2.0 ** -133, "C")


def test_all_zero_tokens(g):
    b, sf = weights(40, 512, 10)
    assert (g.gemv_w4a16(torch.zeros(4, 512, dtype=BF16, device="cuda"), b, sf, 1.0) == 0).all()
