"""The residual step's gradient with numbers of gates that divide unevenly among the SMs: more
blocks than SMs, groups a little longer or shorter than a run, few whole groups to a block;
rows of more than 8192 values, several to a unit."""
from __future__ import annotations

import pytest
import torch

import feed_forward_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_tcgen05_gb300 as g
    yield g
    assert g.gemm_get_device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("M,D,groups", [(12800, 520, 16), (12800, 520, 32), (12800, 520, 64), (12798, 520, 9), (4864, 264, 256), (4864, 264, 304),
                                        (4864, 264, 152), (9728, 1032, 153 * 2 - 2), (2432, 4104, 16), (2448, 4104, 153), (460, 9000, 1), (460, 12296, 4),
                                        (480, 12296, 160), (330, 16384, 2), (330, 16384, 330)])
def test_gradient(g, M, D, groups, post, dtype):
    gen = torch.Generator(device="cuda").manual_seed(groups)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, block, dy, dn = (2 * r(M, D)).to(dtype), r(M, D).to(BF16), r(M, D).to(dtype), r(M, D).to(BF16)
    w_post, w_pre, gate = (1 + 0.3 * r(D)).to(BF16) if post else None, (1 + 0.3 * r(D)).to(BF16), r(groups, D).to(BF16)
    out = g.residual_norm(x, block, w_post=w_post, gate=gate, w_pre=w_pre, scale=0.6)
    y, n, _, _, ey, en = ref.norm(x, block, w_post, gate, w_pre, 0.6, 1e-6, out.y)
    ref.check(out.y, y, ey, "y")
    ref.check(out.n, n, en, "n")
    want = ref.norm_backward(dy, dn, out.y, block, out.rstd_post, out.rstd_pre, w_post, gate, w_pre, 0.6, dtype)
    back = lambda **kw: g.residual_norm_backward(dy, dn, out.y, block, out.rstd_post, out.rstd_pre, w_post=w_post, gate=gate, w_pre=w_pre, scale=0.6, **kw)
    got = back()
    for name in got._fields:
        assert (getattr(got, name) is None) == (name not in want), name
        if name in want:
            ref.check(getattr(got, name), *want[name], name)
    for a, b in zip(got, back()):
        assert (a is None and b is None) or torch.equal(a, b)
