"""The residual step with an infinite or NaN weight or gate value in any column: the row has
it in that column, as the formula does, and 1 / sqrt(inf) = 0 or NaN where its sum reaches,
whatever the place in the row."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_tcgen05_gb300 as g
    yield g
    assert g.gemm_get_device_status() == 0


def make(M, D, dtype, post, pre, groups):
    gen = torch.Generator(device="cuda").manual_seed(D)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    block = r(M, D)
    # no zeros, which an infinity turns into NaN
    block = torch.where(block.abs() < 0.1, 0.1, block)
    return dict(x=r(M, D).to(dtype), block=block.to(BF16), w_post=(1 + 0.1 * r(D)).to(BF16) if post else None,
                gate=None if groups is None else (1 + 0.1 * r(groups, D)).to(BF16), w_pre=(1 + 0.1 * r(D)).to(BF16) if pre else None)


def column_apart(out, clean, rows, col, value, block):
    """`rows` of y hold `value` times the block's sign in `col` (NaN for NaN), their n is NaN there
    and zero elsewhere (NaN for NaN); every other value has the bits of the call without it."""
    D = out.y.shape[1]
    others = [c for c in range(D) if c != col % D]
    assert torch.equal(out.y[:, others], clean.y[:, others])
    keep = [m for m in range(out.y.shape[0]) if m not in rows]
    assert torch.equal(out.y[keep], clean.y[keep])
    if clean.rstd_post is not None:
        assert torch.equal(out.rstd_post, clean.rstd_post)
    got = out.y[rows, col].float()
    if math.isnan(value):
        assert got.isnan().all()
    else:
        assert torch.equal(got, value * torch.sign(block[rows, col].float()))
    if out.n is None:
        return
    assert torch.equal(out.n[keep], clean.n[keep]) and torch.equal(out.rstd_pre[keep], clean.rstd_pre[keep])
    assert out.n[rows, col].isnan().all()
    if math.isnan(value):
        assert out.rstd_pre[rows].isnan().all() and out.n[rows].isnan().all()
    else:
        assert (out.rstd_pre[rows] == 0).all() and (out.n[rows][:, others] == 0).all()


# one piece of eight; rows whose last pieces end within a warp, a thread's pieces, at their end; the
# sizes of one to four pieces a thread
@pytest.mark.parametrize("D", [8, 72, 264, 520, 1032, 2056, 4096, 4104, 5000, 5120, 6008, 8192, 12296])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("col", [0, -8, -1])
def test_weight_after_the_block(g, D, dtype, value, col):
    s = make(5, D, dtype, True, True, None)
    clean = g.residual_norm(**s)
    s["w_post"][col] = value
    column_apart(g.residual_norm(**s), clean, list(range(5)), col, value, s["block"])


@pytest.mark.parametrize("D", [8, 264, 4096, 4104, 5120, 8192, 12296])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("groups", [1, 3, 6])
@pytest.mark.parametrize("col", [0, -1])
def test_gate(g, D, dtype, post, pre, groups, col):
    s = make(6, D, dtype, post, pre, groups)
    clean = g.residual_norm(**s)
    s["gate"][groups - 1, col] = INF
    rows = list(range(6 - 6 // groups, 6))
    column_apart(g.residual_norm(**s), clean, rows, col, INF, s["block"])


@pytest.mark.parametrize("D", [8, 264, 4104, 5120, 12296])
@pytest.mark.parametrize("col", [0, -1])
def test_weight_before_the_next_block(g, D, col):
    """An infinite w_pre reaches its own column of n alone."""
    s = make(5, D, BF16, True, True, None)
    clean = g.residual_norm(**s)
    s["w_pre"][col] = INF
    out = g.residual_norm(**s)
    others = [c for c in range(D) if c != col % D]
    assert torch.equal(out.y, clean.y) and torch.equal(out.rstd_pre, clean.rstd_pre) and torch.equal(out.n[:, others], clean.n[:, others])
    assert not out.n[:, col].isfinite().any()


@pytest.mark.parametrize("D", [264, 4104, 5120, 12296])
@pytest.mark.parametrize("col", [0, -1])
@pytest.mark.parametrize("name", ["w_post", "gate"])
def test_gradient(g, D, col, name):
    """Backward, from a forward pass without the infinity: dx does not see w_post or the gate."""
    s = make(6, D, BF16, True, True, 3)
    out = g.residual_norm(**s)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dy, dn = (torch.randn(6, D, generator=gen, device="cuda").to(BF16) for _ in range(2))
    back = lambda: g.residual_norm_backward(dy, dn, out.y, s["block"], out.rstd_post, out.rstd_pre, w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"])
    clean = back()
    if name == "gate":
        s["gate"][0, col] = INF
    else:
        s["w_post"][col] = INF
    got = back()
    assert torch.equal(got.dx, clean.dx) and torch.equal(got.dw_pre, clean.dw_pre)
    rows = slice(0, 2) if name == "gate" else slice(0, 6)
    # q w_post is infinite in one place, so the row's mean is, and with it every place
    assert not got.dblock[rows].isfinite().any()
    assert torch.equal(got.dblock[2:], clean.dblock[2:]) or name == "w_post"
