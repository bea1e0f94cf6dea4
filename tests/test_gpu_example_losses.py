"""The losses example: its gradients against plain PyTorch, and that it learns."""
from __future__ import annotations

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import moe_language_model_losses as m
    yield m
    assert m.g.gemm_get_device_status() == 0


def test_autograd_functions_against_plain_pytorch(ex):
    gen = torch.Generator(device="cuda").manual_seed(1)
    M, H, V, E, k = 200, 64, 515, 16, 3
    X, Wv, Wr = ((torch.randn(n, H, generator=gen, device="cuda") * s).bfloat16() for n, s in ((M, 1), (V, 0.2), (E, 0.3)))
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    t[::7] = -100
    valid = (t >= 0).to(torch.uint8)
    u = torch.randn(M, k, generator=gen, device="cuda")
    leaves = [a.clone().requires_grad_(True) for a in (X, Wv, Wr)]
    w, losses, experts, counts = ex.Route.apply(leaves[0], leaves[2], k, valid)
    total = ex.LinearCrossEntropy.apply(leaves[0], leaves[1], t) + (w * u).sum() / M + losses[0] + 0.1 * losses[1]
    total.backward()

    x, wv, wr = (a.double().requires_grad_(True) for a in (X, Wv, Wr))
    ce = torch.nn.functional.cross_entropy(x @ wv.T, t, ignore_index=-100)
    l = x @ wr.T
    p = torch.softmax(l, dim=1)
    q = p.gather(1, experts.clamp(min=0).long())
    live = valid.bool()
    T = live.sum()
    bal = E * (counts[:-1].double() / (k * T) * p[live].sum(0) / T).sum()
    z = (torch.logsumexp(l, 1)[live] ** 2).sum() / T
    want = ce + (q / q.sum(1, keepdim=True) * u)[live].sum() / M + bal + 0.1 * z
    want.backward()
    # FP32 sums of BF16 inputs, the ordered product's K = 64 roundings
    assert abs(total.item() - want.item()) <= 1e-5 * abs(want.item())
    # Gradients: BF16 terms (2^-8) summed and rounded to BF16, three BF16 results added
    for a, b in zip(leaves, (x, wv, wr)):
        assert (a.grad.double() - b.grad).norm() <= 2 ** -7 * b.grad.norm()


def test_it_learns(ex):
    h = ex.train(steps=40, rows=512, hidden=128, vocab=1021, experts=8, report=None)
    first, last = h[0], h[-1]
    assert last[0] < 0.5 * first[0]
    assert last[1] >= 0.99            # the balance loss has its minimum near 1
