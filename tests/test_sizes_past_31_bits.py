"""The C ABI takes sizes as 32-bit int: the binding refuses what does not fit,
instead of calling with the lower 32 bits."""
from __future__ import annotations

import pytest
import torch

from test_abi import lib  # noqa: F401  (the built library)

WRAPS = 1 << 32


def test_workspace_bytes_of_sizes_past_31_bits_are_zero(lib):  # noqa: F811
    import nvfp4_block_scaled_tcgen05_gb300 as g
    assert g.gemm_bf16_nt_xent_workspace_bytes(40, 200) > 0
    for wrong in (WRAPS + 40, -WRAPS + 40, 1 << 31):
        assert g.gemm_bf16_nt_xent_workspace_bytes(wrong, 200) == 0
        assert g.gemm_bf16_nt_xent_workspace_bytes(40, wrong) == 0
        assert g.gemm_bf16_nt_xent_backward_workspace_bytes(wrong, 200, 64) == 0
        assert g.gemm_bf16_nt_xent_backward_workspace_bytes(40, wrong, 64) == 0
        assert g.gemm_bf16_nt_xent_backward_workspace_bytes(40, 200, wrong) == 0
        assert g.router_topk_workspace_bytes(WRAPS + 1000, 64) == 0
        assert g.router_topk_workspace_bytes(1000, WRAPS + 64) == 0


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_tcgen05_gb300 as lib
    yield lib
    assert lib.gemm_get_device_status() == 0


@pytest.mark.gpu
def test_a_row_stride_past_31_bits_is_refused(g):
    ld = WRAPS + 16                       # its lower 32 bits are a valid stride of 16 columns
    buf = torch.empty(ld + 16, device="cuda")
    l = buf.as_strided((2, 16), (ld, 1))
    l.copy_(torch.arange(32.0, device="cuda").view(2, 16))
    small = l.contiguous()
    out = g.router_topk(small, 2)
    with pytest.raises(ValueError):
        g.router_topk(l, 2)
    with pytest.raises(ValueError):
        g.router_topk_backward(l, out.experts, out.lse, out.counts, dweights=torch.ones(2, 2, device="cuda"))
    # one row has no stride
    assert torch.equal(g.router_topk(l[1:], 2).experts, out.experts[1:])


@pytest.mark.gpu
def test_dimensions_past_31_bits_are_refused(g):
    # (no elements, so no memory)
    long = torch.empty(WRAPS + 40, 0, device="cuda", dtype=torch.bfloat16)
    short = torch.empty(8, 0, device="cuda", dtype=torch.bfloat16)
    t = torch.zeros(8, device="cuda", dtype=torch.int64)
    with pytest.raises(ValueError):
        g.gemm_bf16_nt_xent(short, long, t)
    with pytest.raises(ValueError):
        g.router_topk(torch.empty(0, WRAPS + 40, device="cuda"), 2)
    C = torch.empty(8, 0, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        g.gemm_bf16_nt(long, short, C)
