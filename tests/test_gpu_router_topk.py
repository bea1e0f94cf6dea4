"""The routing step against its definition in 64 bits, on the GPU.

Tolerances.  A probability is exp(l - lse) in FP32: the difference carries
2^-24 (|l| + |lse|) twice and lse its own 2^-22, so its relative error is at
most `rel` = 2^-22 (|l| + |lse| + 2) per row (with room for the exponential's
own two units); sums of M such terms add M 2^-24 at most.  Chosen experts and
counts are exact.
"""
from __future__ import annotations

import math

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


def logits_of(M, E, seed, ties=True, closed=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    l = 2 * torch.randn(M, E, generator=gen, device="cuda")
    if ties:
        l = torch.where(torch.rand(M, 1, generator=gen, device="cuda") < 0.5, torch.round(l * 2) / 2, l)
    if closed:
        l = l.masked_fill(torch.rand(M, E, generator=gen, device="cuda") < closed, -math.inf)
    valid = (torch.rand(M, generator=gen, device="cuda") < 0.85).to(torch.uint8)
    return l, valid


def reference(l, k, valid, norm):
    """Everything in 64 bits; a row at a time in the choice, by (-logit, index)."""
    x = l.to(F64)
    M, E = x.shape
    live = (x > -math.inf).any(dim=1)
    if valid is not None:
        live &= valid != 0
    lse = torch.logsumexp(x, dim=1)
    p = torch.where(live[:, None], torch.exp(x - lse[:, None]), torch.zeros_like(x)).nan_to_num(0.0)
    order = torch.argsort(-x, dim=1, stable=True)[:, :k]
    ok = live[:, None] & (x.gather(1, order) > -math.inf)
    experts = torch.where(ok, order, torch.full_like(order, -1))
    w = torch.where(ok, p.gather(1, order), torch.zeros(1, 1, dtype=F64, device=l.device))
    if norm:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    counts = torch.bincount(order[ok], minlength=E)
    T = int(live.sum())
    t = max(T, 1)
    probs = p.sum(dim=0) / t
    bal = E * (counts.to(F64) / (k * t) * probs).sum()
    z = (lse[live] ** 2).sum() / t
    rel = 2.0 ** -22 * (torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(dim=1) +
                        lse.nan_to_num(0, 0, 0).abs() + 2)
    return dict(w=w, experts=experts, lse=lse, counts=counts, T=T, probs=probs, bal=bal, z=z,
                rel=rel, live=live, p=p)


def check_forward(out, r):
    assert torch.equal(out.experts.long(), r["experts"])
    assert torch.equal(out.counts[:-1].long(), r["counts"]) and int(out.counts[-1]) == r["T"]
    fin = torch.isfinite(r["lse"])
    assert ((out.lse.to(F64) - r["lse"])[fin].abs() <= r["rel"][fin]).all()
    assert (out.lse[~fin] == -math.inf).all()
    assert ((out.weights.to(F64) - r["w"]).abs() <= 3 * r["rel"][:, None] * r["w"] + 1e-37).all()
    top = float(r["rel"][r["live"]].max()) if r["T"] else 0.0
    M = r["w"].shape[0]
    tol = top + M * 2.0 ** -24 + 2.0 ** -20
    assert ((out.probs.to(F64) - r["probs"]).abs() <= tol * r["probs"] + 1e-37).all()
    assert abs(float(out.losses[0]) - float(r["bal"])) <= (tol + 2.0 ** -19) * float(r["bal"])
    assert abs(float(out.losses[1]) - float(r["z"])) <= (2 * top + M * 2.0 ** -24 + 2.0 ** -20) * max(float(r["z"]), 1e-3)


SHAPES = [
    (1, 1, 1), (1, 256, 8), (3, 7, 7), (5, 8, 2), (8, 32, 1), (9, 33, 32), (64, 64, 6), (100, 60, 4),
    (65, 65, 3), (1000, 128, 8), (257, 256, 8), (4510, 256, 8), (77, 257, 5), (300, 512, 16),
    (31, 1000, 32), (50, 1024, 10), (20011, 16, 2),
]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("M,E,k", SHAPES)
def test_forward(g, M, E, k, norm):
    l, valid = logits_of(M, E, M + E + k)
    check_forward(g.router_topk(l, k, normalize=norm), reference(l, k, None, norm))
    check_forward(g.router_topk(l, k, valid=valid, normalize=norm), reference(l, k, valid, norm))
    l, valid = logits_of(M, E, M + E + k, closed=0.6)
    l[M // 2] = -math.inf
    check_forward(g.router_topk(l, k, valid=valid, normalize=norm), reference(l, k, valid, norm))


def grad_reference(l, k, valid, norm, dw, dl, r):
    """Autograd through the definition in 64 bits, choice and counts fixed."""
    M, E = l.shape
    live = r["live"]
    x = l.to(F64)[live].requires_grad_(True)
    if x.numel() == 0:
        return torch.zeros(M, E, dtype=F64, device=l.device)
    lse = torch.logsumexp(x, dim=1)
    p = torch.exp(x - lse[:, None])
    ex = r["experts"][live]
    ok = (ex >= 0).to(F64)
    w = p.gather(1, ex.clamp(min=0)) * ok
    if norm:
        w = w / w.sum(dim=1, keepdim=True)
    t = r["T"]
    total = 0.0
    if dw is not None:
        total = total + (w * ok * dw.to(F64)[live]).sum()
    if dl is not None:
        bal = E * (r["counts"].to(F64) / (k * t) * p.sum(dim=0) / t).sum()
        total = total + float(dl[0]) * bal + float(dl[1]) * (lse ** 2).sum() / t
    out = torch.zeros(M, E, dtype=F64, device=l.device)
    if torch.is_tensor(total):
        out[live] = torch.autograd.grad(total, x)[0].nan_to_num(0.0)
    return out


def grad_bound(l, k, norm, dw, dl, r):
    """Error bound: every factor of dl = p (dp - sum p dp + shift) carries a few
    rel; dp's weight part grows by 1 / s (its sum) when normalised."""
    M, E = l.shape
    t = max(r["T"], 1)
    ex = r["experts"]
    ok = ex >= 0
    up = torch.zeros(M, E, dtype=F64, device=l.device)
    if dw is not None:
        u = torch.where(ok, dw.to(F64).abs(), torch.zeros(1, 1, dtype=F64, device=l.device))
        if norm:
            s = torch.where(ok, r["p"].gather(1, ex.clamp(min=0)), torch.zeros(1, 1, dtype=F64, device=l.device)).sum(dim=1, keepdim=True).clamp(min=1e-30)
            u = (u + u.amax(dim=1, keepdim=True)) / s * ok
        up.scatter_add_(1, ex.clamp(min=0), u)
    base = torch.zeros(M, E, dtype=F64, device=l.device)
    shift = torch.zeros(M, 1, dtype=F64, device=l.device)
    if dl is not None:
        base += abs(float(dl[0])) * E * r["counts"].to(F64)[None] / (k * t * t)
        shift = 2 * abs(float(dl[1])) * r["lse"].nan_to_num(0, 0, 0).abs()[:, None] / t
    dp = up + base
    size = r["p"] * (dp + (r["p"] * dp).sum(dim=1, keepdim=True) + shift)
    return 8 * r["rel"][:, None] * size + 1e-37


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("M,E,k", SHAPES)
def test_backward(g, M, E, k, norm):
    gen = torch.Generator(device="cuda").manual_seed(M * 7 + E)
    l, valid = logits_of(M, E, M + E + 2 * k, closed=0.3)
    l[M // 2] = -math.inf
    out = g.router_topk(l, k, valid=valid, normalize=norm)
    r = reference(l, k, valid, norm)
    dw = torch.randn(M, k, generator=gen, device="cuda")
    dl = torch.tensor([0.7, -0.3], device="cuda")
    for a, b in ((dw, dl), (dw, None), (None, dl), (None, None)):
        want = grad_reference(l, k, valid, norm, a, b, r)
        tol = grad_bound(l, k, norm, a, b, r)
        got = g.router_topk_backward(l, out.experts, out.lse, out.counts, dweights=a, dlosses=b, normalize=norm)
        assert got.dtype == torch.float32
        assert ((got.to(F64) - want).abs() <= tol).all()
        assert (got[~r["live"]] == 0).all()
        half = g.router_topk_backward(l, out.experts, out.lse, out.counts, dweights=a, dlosses=b,
                                      normalize=norm, dtype=torch.bfloat16)
        assert torch.equal(half, got.bfloat16())       # the same value, rounded once


@pytest.mark.parametrize("norm", [False, True])
def test_backward_against_differences(g, norm):
    M, E, k, h = 40, 24, 3, 1e-5
    l, valid = logits_of(M, E, 5, ties=False)
    out = g.router_topk(l, k, valid=valid, normalize=norm)
    r = reference(l, k, valid, norm)
    gen = torch.Generator(device="cuda").manual_seed(8)
    dw = torch.randn(M, k, generator=gen, device="cuda")
    dl = torch.tensor([3.0, 0.5], device="cuda")
    got = g.router_topk_backward(l, out.experts, out.lse, out.counts, dweights=dw, dlosses=dl, normalize=norm)
    tol = grad_bound(l, k, norm, dw, dl, r)

    def total(x):
        q = reference(x, k, valid, norm)
        assert torch.equal(q["experts"], r["experts"])   # the step is small enough
        return (q["w"] * dw.to(F64)).sum() + 3.0 * q["bal"] + 0.5 * q["z"]

    for _ in range(4):
        u = torch.randn(M, E, generator=gen, device="cuda", dtype=F64)
        num = (total(l.to(F64) + h * u) - total(l.to(F64) - h * u)) / (2 * h)
        assert (num - (got.to(F64) * u).sum()).abs() <= (tol * u.abs()).sum() + 1e-6


@pytest.mark.parametrize("E,k", [(256, 8), (64, 32), (1024, 5), (33, 33 - 1)])
def test_all_equal_logits_take_the_lowest_indices(g, E, k):
    # every value is a candidate: more than 32 of them go the long way
    l = torch.full((70, E), 0.25, device="cuda")
    out = g.router_topk(l, k, normalize=True)
    assert (out.experts == torch.arange(k, device="cuda")).all()
    assert ((out.weights.to(F64) - 1 / k).abs() <= 1e-6 / k).all()
    assert (out.counts[:k] == 70).all() and (out.counts[k:-1] == 0).all()
    l[:, E - 1] = 1.0                      # one value above the ties
    out = g.router_topk(l, k)
    assert (out.experts[:, 0] == E - 1).all()
    assert (out.experts[:, 1:] == torch.arange(k - 1, device="cuda")).all()


def test_row_stride(g):
    l, valid = logits_of(333, 48, 3, closed=0.2)
    wide = torch.full((333, 131), float("nan"), device="cuda")
    view = wide[:, 17:65]
    view.copy_(l)
    a, b = g.router_topk(l, 5, valid=valid), g.router_topk(view, 5, valid=valid)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    dw = torch.randn(333, 5, device="cuda")
    assert torch.equal(g.router_topk_backward(l, a.experts, a.lse, a.counts, dweights=dw),
                       g.router_topk_backward(view, a.experts, a.lse, a.counts, dweights=dw))


def test_bool_mask_and_no_live_row(g):
    l, valid = logits_of(100, 16, 3)
    a, b = g.router_topk(l, 2, valid=valid), g.router_topk(l, 2, valid=valid.bool())
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    for x, v in ((l, torch.zeros(100, dtype=torch.uint8, device="cuda")), (torch.full_like(l, -math.inf), None)):
        out = g.router_topk(x, 2, valid=v, normalize=True)
        assert (out.experts == -1).all() and (out.weights == 0).all() and (out.counts == 0).all()
        assert (out.probs == 0).all() and (out.losses == 0).all()
        d = g.router_topk_backward(x, out.experts, out.lse, out.counts, dweights=torch.ones(100, 2, device="cuda"),
                                   dlosses=torch.ones(2, device="cuda"), normalize=True)
        assert (d == 0).all()


def test_lowest_values_infinities_and_nan(g):
    low = torch.finfo(torch.float32).min
    l = torch.zeros(6, 8, device="cuda")
    l[0] = low                    # a finite mask everywhere: uniform
    l[1] = low
    l[1, 3] = 0.0                 # one open expert, the rest of weight 0
    l[2] = -math.inf
    l[2, 5] = -2.0                # one expert left for k = 2
    l[3, 2] = math.nan
    l[4, 0], l[4, 1] = -0.0, 0.0  # equal: the lower index first
    l[5, 6] = math.inf
    out = g.router_topk(l, 2, normalize=False)
    ex = out.experts.tolist()
    assert ex[0] == [0, 1] and ex[1] == [3, 0] and ex[2] == [5, -1] and ex[4] == [0, 1]
    assert ex[3][0] == 2 and ex[5][0] == 6
    w = out.weights
    assert torch.allclose(w[0], torch.full((2,), 0.125, device="cuda"), rtol=1e-6)
    assert w[1].tolist() == [1.0, 0.0] and w[2].tolist() == [1.0, 0.0]
    assert torch.isnan(w[3]).all() and torch.isnan(out.lse[3]) and torch.isnan(out.losses).all()
    assert torch.isnan(out.lse[5])
    assert int(out.counts[-1]) == 6
    # NaN in rows that take no part stays there
    out = g.router_topk(l, 2, valid=torch.tensor([1, 1, 1, 0, 1, 0], dtype=torch.uint8, device="cuda"))
    assert torch.isfinite(out.losses[0]) and torch.isfinite(out.probs).all() and (out.experts[3] == -1).all()
    assert out.losses[1] == math.inf     # lse^2 of the rows of lowest values


def test_repeats_bit_for_bit_on_another_stream_and_from_a_graph(g):
    l, valid = logits_of(30011, 128, 4)
    a = g.router_topk(l, 6, valid=valid, normalize=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = g.router_topk(l, 6, valid=valid, normalize=True, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = g.router_topk(l, 6, valid=valid, normalize=True)
    for _ in range(3):
        for x in c:
            x.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, c))


def test_offsets_past_32_bits(g):
    # rows 70001 floats apart: the last row starts past 2^31 elements
    M, E, ld = 31000, 16, 70001
    buf = torch.empty(M * ld, device="cuda")
    view = buf.as_strided((M, E), (ld, 1))
    l, _ = logits_of(M, E, 6)
    view.copy_(l)
    a, b = g.router_topk(l, 2), g.router_topk(view, 2)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals(g):
    l, valid = logits_of(10, 16, 1)
    for bad in (l.double(), l.bfloat16()):
        with pytest.raises(TypeError):
            g.router_topk(bad, 2)
    with pytest.raises(ValueError):
        g.router_topk(l.T, 2)
    with pytest.raises(ValueError):
        g.router_topk(l, 17)
    with pytest.raises(ValueError):
        g.router_topk(l, 0)
    with pytest.raises(ValueError):
        g.router_topk(l, 2, valid=valid[:9])
    with pytest.raises(ValueError):
        g.router_topk(l.cpu(), 2)
    with pytest.raises(ValueError):
        g.router_topk(torch.zeros(1, 16, device="cuda").expand(10, 16), 2)
    wide = torch.zeros(4, 1025, device="cuda")
    with pytest.raises(g.GemmError):
        g.router_topk(wide, 2)
    with pytest.raises(g.GemmError):
        g.router_topk(torch.zeros(4, 64, device="cuda"), 33)
    out = g.router_topk(l, 2)
    with pytest.raises(ValueError):
        g.router_topk_backward(l, out.experts, out.lse, out.counts[:-1])
    with pytest.raises(TypeError):
        g.router_topk_backward(l, out.experts.long(), out.lse, out.counts)
    with pytest.raises(TypeError):
        g.router_topk_backward(l, out.experts, out.lse, out.counts, dtype=torch.float16)
    with pytest.raises(g.GemmError):
        g.router_topk_backward(l, out.experts, out.lse, out.counts, dlogits=l)
