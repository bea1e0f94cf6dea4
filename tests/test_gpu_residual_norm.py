"""The residual step (norm after a block, gate, residual scale, norm before the next
block) and its gradients, against 64-bit references."""
from __future__ import annotations

import pytest
import torch

import feed_forward_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_tcgen05_gb300 as g
    yield g
    assert g.gemm_get_device_status() == 0


def make(M, D, dtype, post, pre, groups, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    return dict(x=(2 * r(M, D)).to(dtype), block=r(M, D).to(BF16),
                w_post=(1 + 0.3 * r(D)).to(BF16) if post else None,
                gate=None if groups is None else (r(D) if groups == 0 else r(groups, D)).to(BF16),
                w_pre=(1 + 0.3 * r(D)).to(BF16) if pre else None), dict(dy=r(M, D).to(dtype), dn=r(M, D).to(BF16) if pre else None)


# rows: one, fewer and more than the grid; D: one piece, a warp's edge, odd, the most
SHAPES = [(1, 8), (1, 4096), (3, 248), (7, 256), (33, 264), (130, 2056), (40, 5120), (25, 6008), (304, 1032), (305, 8), (701, 4104), (16, 8192), (12, 12296), (9, 16384)]
# with a gate: none (None), one vector (0), groups
KINDS = [(True, True, 0), (True, True, 1), (True, False, None), (False, True, None), (False, True, 0), (False, False, 1)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("post,pre,groups", KINDS)
@pytest.mark.parametrize("M,D", SHAPES)
def test_forward_and_backward(g, M, D, post, pre, groups, dtype):
    run(g, M, D, post, pre, groups, dtype)


# groups that lie within a run, hold several runs, or are rows
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D,groups", [(12, 264, 12), (12, 264, 3), (1000, 72, 500), (1000, 72, 8), (1000, 72, 1000), (2432, 40, 2), (3648, 16, 304),
                                        (460, 1032, 460), (500, 4104, 500), (320, 2056, 160), (701, 3592, 701), (33, 5120, 33),
                                        (40, 8192, 40), (40, 6008, 20), (20, 12296, 20)])
def test_gate_groups(g, M, D, groups, dtype):
    run(g, M, D, True, True, groups, dtype)
    run(g, M, D, False, True, groups, dtype)


def run(g, M, D, post, pre, groups, dtype):
    s, grads = make(M, D, dtype, post, pre, groups)
    scale, eps = 0.6, 1e-5
    out = g.residual_norm(**s, scale=scale, eps=eps)
    y, n, r_post, r_pre, ey, en = ref.norm(**s, scale=scale, eps=eps, stored=out.y)
    assert out.y.dtype == dtype
    ref.check(out.y, y, ey, "y")
    for got, want, e, name in ((out.n, n, en, "n"), (out.rstd_post, r_post, None, "rstd_post"), (out.rstd_pre, r_pre, None, "rstd_pre")):
        assert (got is None) == (want is None), name
        if want is not None:
            ref.check(got, want, ref.ROW_SUM * want.abs() if e is None else e, name)
    for dy in (grads["dy"], None) if pre else (grads["dy"],):
        want = ref.norm_backward(dy, grads["dn"], out.y, s["block"], out.rstd_post, out.rstd_pre, s["w_post"], s["gate"], s["w_pre"], scale, dtype)
        got = g.residual_norm_backward(dy, grads["dn"], out.y, s["block"], out.rstd_post, out.rstd_pre, w_post=s["w_post"],
                                       gate=s["gate"], w_pre=s["w_pre"], scale=scale)
        for name in got._fields:
            assert (getattr(got, name) is None) == (name not in want), name
            if name in want:
                assert getattr(got, name).shape == want[name][0].shape
                ref.check(getattr(got, name), *want[name], name)
        # without the weights' gradients the others keep their bits
        less = g.residual_norm_backward(dy, grads["dn"], out.y, s["block"], out.rstd_post, out.rstd_pre, w_post=s["w_post"],
                                        gate=s["gate"], w_pre=s["w_pre"], scale=scale, need_dw=False)
        assert less.dw_pre is None and less.dw_post is None and less.dgate is None
        assert torch.equal(less.dx, got.dx) and torch.equal(less.dblock, got.dblock)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_first_norm_without_a_block(g, dtype):
    s, grads = make(50, 520, dtype, False, True, None)
    out = g.residual_norm(s["x"], w_pre=s["w_pre"])
    assert out.y is s["x"] and out.rstd_post is None
    _, n, _, r_pre, _, en = ref.norm(s["x"], None, None, None, s["w_pre"], 1.0, 1e-6, s["x"])
    ref.check(out.n, n, en, "n")
    for dy in (grads["dy"], None):
        want = ref.norm_backward(dy, grads["dn"], s["x"], None, None, out.rstd_pre, None, None, s["w_pre"], 1.0, dtype)
        got = g.residual_norm_backward(dy, grads["dn"], s["x"], rstd_pre=out.rstd_pre, w_pre=s["w_pre"])
        assert got.dblock is None and got.dw_post is None
        ref.check(got.dx, *want["dx"], "dx")
        ref.check(got.dw_pre, *want["dw_pre"], "dw_pre")


@pytest.mark.parametrize("kind", [(True, True), (True, False), (False, True)])
def test_without_what_the_gradient_needs(g, kind):
    s, _ = make(9, 264, BF16, *kind, 0)
    out, less = g.residual_norm(**s), g.residual_norm(**s, need_rstd=False)
    assert less.rstd_post is None and less.rstd_pre is None
    assert torch.equal(less.y, out.y) and (out.n is None) == (less.n is None)
    assert out.n is None or torch.equal(less.n, out.n)


def test_in_place(g):
    s, grads = make(77, 1032, BF16, True, True, 0)
    out = g.residual_norm(**s)
    x = s["x"].clone()
    again = g.residual_norm(**{**s, "x": x}, y=x)
    assert again.y is x and torch.equal(x, out.y) and torch.equal(again.n, out.n)
    back = lambda dy, **kw: g.residual_norm_backward(dy, grads["dn"], out.y, s["block"], out.rstd_post, out.rstd_pre, w_post=s["w_post"],
                                                     gate=s["gate"], w_pre=s["w_pre"], **kw)
    want, dy = back(grads["dy"]), grads["dy"].clone()
    got = back(dy, dx=dy)
    assert got.dx is dy
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_rows_with_nan_inf_and_zeros_stay_apart(g):
    s, grads = make(6, 264, BF16, True, True, None)
    clean = g.residual_norm(**s)
    s["block"][1, 3] = float("nan")
    s["x"][2, 5] = float("inf")
    s["block"][3] = 0
    s["x"][4], s["block"][4] = 0, 0
    out = g.residual_norm(**s)
    assert out.y[1].isnan().all() and out.n[1].isnan().all()
    assert out.y[2].isinf().sum() == 1 and out.rstd_pre[2] == 0 and out.n[2].isnan().sum() == 1
    assert torch.equal(out.y[3], s["x"][3])  # a norm of zeros is zeros
    # 1 / sqrt(1e-6): eps in FP32 is off by 2^-24 of it (half of that in the root), the root and the quotient round once each
    assert (out.n[4] == 0).all()
    assert abs(float(out.rstd_post[4]) - 1000) <= 1000 * 2.0 ** -22 and out.rstd_post[4] == out.rstd_pre[4]
    for row in (0, 5):
        assert torch.equal(out.y[row], clean.y[row]) and torch.equal(out.n[row], clean.n[row])


@pytest.mark.parametrize("D", [8, 264, 520, 4104, 5000])
@pytest.mark.parametrize("where", [0, -1])
def test_infinite_and_nan_gradients_as_the_formula_has_them(g, D, where):
    """A row with an infinity in its first or last place: the same places are infinite, of the
    same sign, and NaN as in the formula; the other rows keep their bits."""
    s, grads = make(3, D, F32, True, True, None)
    out = g.residual_norm(**s)
    back = lambda: g.residual_norm_backward(grads["dy"], grads["dn"], out.y, s["block"], out.rstd_post, out.rstd_pre, w_post=s["w_post"],
                                            w_pre=s["w_pre"], need_dw=False)
    clean = back()
    for value in (float("inf"), float("nan")):
        for name in ("dy", "dn"):
            keep = grads[name].clone()
            grads[name][1, where] = value
            got = back()
            grads[name].copy_(keep)
            assert torch.equal(got.dx[::2], clean.dx[::2]) and torch.equal(got.dblock[::2], clean.dblock[::2])
            # t is infinite or NaN where dy is; an infinite mean reaches every place of the row
            if name == "dy":
                assert not got.dx[1, where].isfinite() and int((~got.dx[1].isfinite()).sum()) == 1
            elif value == float("inf"):
                yhat = out.y[1].double() * out.rstd_pre[1].double()
                e = float(s["w_pre"][where]) * float("inf")
                want = -yhat * (e * float(yhat[where]))
                want[where] = float("nan") if float(yhat[where]) ** 2 > 0 else e
                fine = torch.isinf(got.dx[1]) & (torch.sign(got.dx[1]) == torch.sign(want))
                assert bool(fine[torch.arange(D, device="cuda") != where % D].all())
            else:
                assert got.dx[1].isnan().all()


def test_against_differences(g):
    """The gradients against central differences of the forward formula in 64 bits."""
    s, grads = make(4, 16, F32, True, True, 2, seed=5)
    out = g.residual_norm(**s, scale=0.6)
    got = g.residual_norm_backward(grads["dy"], grads["dn"], out.y, s["block"], out.rstd_post, out.rstd_pre, w_post=s["w_post"],
                                   gate=s["gate"], w_pre=s["w_pre"], scale=0.6)

    def loss(**kw):
        a = {k: kw.get(k, v).to(F64) for k, v in s.items()}
        c = a["block"] * torch.rsqrt((a["block"] ** 2).mean(1, keepdim=True) + 1e-6) * a["w_post"]
        y = a["x"] + 0.6 * a["gate"].repeat_interleave(2, 0) * c
        n = y * torch.rsqrt((y ** 2).mean(1, keepdim=True) + 1e-6) * a["w_pre"]
        return (grads["dy"].to(F64) * y).sum() + (grads["dn"].to(F64) * n).sum()

    h = 1e-4
    for name, grad in (("x", got.dx), ("block", got.dblock), ("w_pre", got.dw_pre), ("w_post", got.dw_post), ("gate", got.dgate)):
        base = s[name].to(F64)
        for i in range(0, base.numel(), 7):
            step = torch.zeros_like(base).reshape(-1)
            step[i] = h
            d = (loss(**{name: base + step.reshape(base.shape)}) - loss(**{name: base - step.reshape(base.shape)})) / (2 * h)
            v = float(grad.reshape(-1)[i])
            # truncation h^2 / 6 times a third derivative of order 10, the BF16 rounding of dblock, FP32 sums
            assert abs(v - float(d)) <= 1e-6 + (2.0 ** -8 if name == "block" else 2.0 ** -16) * (abs(float(d)) + 1), (name, i)
