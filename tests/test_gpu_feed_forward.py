"""The feed-forward block's operators as they are used together: a block's forward and
backward pass, a decoded token, captured graphs, other streams and threads, and what
they leave alone."""
from __future__ import annotations

import threading

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


def randn(gen, *shape, scale=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


class Block:
    """x -> norm -> gated projection -> down projection -> norm, gate, scale -> x, twice."""

    def __init__(self, D, F, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.w_pre, self.w_post, self.w_next = ((1 + 0.2 * randn(gen, D, dtype=F32)).to(BF16) for _ in range(3))
        self.gate = (0.5 + 0.2 * randn(gen, D, dtype=F32)).to(BF16)
        self.Wg, self.Wu = randn(gen, F, D, scale=1.5 / D ** 0.5), randn(gen, F, D, scale=1 / D ** 0.5)
        self.Wd = randn(gen, D, F, scale=1 / F ** 0.5)
        self.scale = 0.7

    def forward(self, g, x, act):
        first = g.residual_norm(x, w_pre=self.w_pre)
        H, gates = g.gemm_bf16_nt_gated(first.n, self.Wg, self.Wu, act=act, save_gates=True)
        out = g.gemm_bf16_nt(H, self.Wd)
        last = g.residual_norm(x, out, w_post=self.w_post, gate=self.gate, w_pre=self.w_next, scale=self.scale)
        return first, H, gates, out, last

    def backward(self, g, x, act, saved, dy, dn):
        first, H, gates, out, last = saved
        end = g.residual_norm_backward(dy, dn, last.y, out, last.rstd_post, last.rstd_pre, w_post=self.w_post, gate=self.gate,
                                       w_pre=self.w_next, scale=self.scale)
        dH = g.gemm_bf16_nn(end.dblock, self.Wd)
        dWd = g.gemm_bf16_tn(end.dblock, H)
        dn0, dWg, dWu = g.gemm_bf16_nt_gated_backward(first.n, self.Wg, self.Wu, dH, act=act, gates=gates)
        begin = g.residual_norm_backward(end.dx, dn0, x, rstd_pre=first.rstd_pre, w_pre=self.w_pre)
        return begin.dx, begin.dw_pre, dWg, dWu, dWd, end.dw_post, end.dgate, end.dw_pre

    def exact(self, x, act):
        """The same in 64 bits, differentiable."""
        p = {k: getattr(self, k).to(F64).requires_grad_() for k in ("w_pre", "w_post", "w_next", "gate", "Wg", "Wu", "Wd")}
        x = x.to(F64).requires_grad_()
        r = lambda v: torch.rsqrt((v * v).mean(dim=1, keepdim=True) + 1e-6)
        n = x * r(x) * p["w_pre"]
        h = ref.act(n @ p["Wg"].T, act)[0] * (n @ p["Wu"].T)
        out = h @ p["Wd"].T
        y = x + self.scale * p["gate"] * (out * r(out) * p["w_post"])
        return x, p, y, y * r(y) * p["w_next"]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,D,F,dtype", [(1, 256, 512, BF16), (200, 264, 520, F32), (333, 1024, 1032, BF16)])
def test_block_forward_and_backward(g, M, D, F, dtype, act):
    b, gen = Block(D, F), torch.Generator(device="cuda").manual_seed(1)
    x, dy, dn = randn(gen, M, D, dtype=dtype), randn(gen, M, D, dtype=dtype), randn(gen, M, D)
    saved = b.forward(g, x, act)
    grads = b.backward(g, x, act, saved, dy, dn)
    x64, p, y, n = b.exact(x, act)
    # A chain of at most six BF16 roundings (2^-8 each at most, independent) before a value; the
    # norm of their sum is that of one times sqrt(6) if they are independent, 6 at most.
    bound = 6 * 2.0 ** -8
    rel = lambda got, want: float((got.to(F64) - want).norm() / want.norm())
    assert rel(saved[4].y, y) <= bound and rel(saved[4].n, n) <= bound
    torch.autograd.backward([y, n], [dy.to(F64), dn.to(F64)])
    want = (x64.grad, p["w_pre"].grad, p["Wg"].grad, p["Wu"].grad, p["Wd"].grad, p["w_post"].grad, p["gate"].grad, p["w_next"].grad)
    for name, got, w in zip(("x", "w_pre", "Wg", "Wu", "Wd", "w_post", "gate", "w_next"), grads, want):
        # the backward pass carries the forward pass's roundings and as many of its own
        assert rel(got, w) <= 2 * bound, name


def quantize(gen, N, K):
    b = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    sf = torch.randint(40, 64, (N, K // 16), generator=gen, device="cuda", dtype=torch.uint8)
    return b, sf


@pytest.mark.parametrize("M", [1, 5, 16])
def test_decoded_tokens_with_4_bit_weights(g, M):
    """norm -> both projections -> down projection -> norm, on NVFP4 weights; the prompt's
    kernels give the same block within their roundings."""
    D, F, gen = 512, 1280, torch.Generator(device="cuda").manual_seed(M)
    (bg, sg), (bu, su), (bd, sd) = quantize(gen, F, D), quantize(gen, F, D), quantize(gen, D, F)
    w, x = (1 + 0.2 * randn(gen, D, dtype=F32)).to(BF16), randn(gen, M, D)
    s = [0.3 / D ** 0.5, 0.3 / D ** 0.5, 0.3 / F ** 0.5]
    n = g.residual_norm(x, w_pre=w).n
    H = g.gemv_w4a16_gated(n, bg, sg, s[0], bu, su, s[1])
    want, e = ref.few_tokens_gated(n, bg, sg, s[0], bu, su, s[1], "silu")
    ref.check(H, want, e, "H")
    out = g.gemv_w4a16(H, bd, sd, s[2])
    want, e = ref.few_tokens(H, bd, sd, s[2])
    ref.check(out, want, e * (1 + ref.BF16_HALF) + ref.BF16_HALF * want.abs(), "out")
    # gemm_w4a16 sums in another order: both are within the bound of the same value
    ref.check(g.gemm_w4a16(H, bd, sd, s[2]), want, e * (1 + ref.BF16_HALF) + ref.BF16_HALF * want.abs(), "gemm_w4a16")
    step = g.residual_norm(x, out, w_post=w, w_pre=w, y=x)
    assert step.y is x


def calls(g, seed=0):
    """(name, inputs that may be replaced, call) of every operator."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    X, Wg, Wu, dH = randn(gen, 70, 264), randn(gen, 520, 264, scale=0.1), randn(gen, 520, 264, scale=0.1), randn(gen, 70, 520)
    X2, dH2 = randn(gen, 200, 264), randn(gen, 200, 520)
    x, blk, w, gate = randn(gen, 90, 520), randn(gen, 90, 520), randn(gen, 520), randn(gen, 3, 520)
    r = torch.rand(90, generator=gen, device="cuda") + 0.5
    A, (b, sf), (b2, sf2) = randn(gen, 11, 512), quantize(gen, 300, 512), quantize(gen, 300, 512)
    yield "gated, few", [X], lambda: g.gemm_bf16_nt_gated(X, Wg, Wu, save_gates=True)
    yield "gated", [X2], lambda: g.gemm_bf16_nt_gated(X2, Wg, Wu, act="gelu_tanh")[:1]
    yield "gated backward", [X2, dH2], lambda: g.gemm_bf16_nt_gated_backward(X2, Wg, Wu, dH2)
    yield "gated backward, gates", [dH], lambda: g.gemm_bf16_nt_gated_backward(X, Wg, Wu, dH, gates=gates)
    yield "tn", [dH], lambda: [g.gemm_bf16_tn(dH, X)]
    yield "norm", [x, blk], lambda: g.residual_norm(x, blk, w_post=w, gate=gate, w_pre=w)
    yield "norm backward", [x, blk], lambda: g.residual_norm_backward(x, blk, x, blk, r, r, w_post=w, gate=gate, w_pre=w)
    X3, dH3, row_gate = randn(gen, 11, 264), randn(gen, 11, 520), randn(gen, 90, 520)
    yield "gated, fewer", [X3], lambda: g.gemm_bf16_nt_gated(X3, Wg, Wu, act="gelu_tanh", save_gates=True)
    yield "gated backward, fewer", [X3, dH3], lambda: g.gemm_bf16_nt_gated_backward(X3, Wg, Wu, dH3)
    yield "norm, a gate per row", [x, blk], lambda: g.residual_norm(x, blk, w_post=w, gate=row_gate, w_pre=w)
    yield "norm backward, a gate per row", [x, blk], lambda: g.residual_norm_backward(x, blk, x, blk, r, r, w_post=w, gate=row_gate, w_pre=w)
    yield "gemv", [A], lambda: [g.gemv_w4a16(A, b, sf, 0.1)]
    yield "gemv gated", [A], lambda: [g.gemv_w4a16_gated(A, b, sf, 0.01, b2, sf2, 0.02)]


gates = None


@pytest.fixture(scope="module")
def ops(g):
    global gates
    gates = torch.randn(2, 70, 520, device="cuda").to(BF16)
    return list(calls(g))


def same(a, b):
    assert len(a) == len(b)
    for s, t in zip(a, b):
        assert (s is None) == (t is None)
        if s is not None:
            assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))


def test_results_repeat_bit_for_bit(g, ops):
    for name, _, call in ops:
        first = [t.clone() for t in call()]
        for _ in range(3):
            same(first, call())


def test_captured_and_replayed_with_new_inputs(g, ops):
    for name, inputs, call in ops:
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        for k in range(3):
            for t in inputs:
                t.copy_(torch.randn_like(t.float()))
            want = [t.clone() for t in call()]
            for t in out:
                t.view(torch.uint8).fill_(0x5A)
            graph.replay()
            torch.cuda.synchronize()
            same(want, out)


def test_a_given_stream_and_threads(g, ops):
    want = {name: [t.clone() for t in call()] for name, _, call in ops}
    torch.cuda.synchronize()
    errors = []

    def work(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(10):
                    for name, _, call in ops:
                        out = call()
                        stream.synchronize()
                        same(want[name], out)
        except Exception as e:  # noqa: BLE001
            errors.append((k, e))
    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]


def test_stream_argument(g):
    gen = torch.Generator(device="cuda").manual_seed(0)
    X, W, x = randn(gen, 40, 64), randn(gen, 72, 64), randn(gen, 40, 264)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    H = g.gemm_bf16_nt_gated(X, W, W, stream=s)[0]
    d = g.gemm_bf16_nt_gated_backward(X, W, W, H, stream=s)
    C = g.gemm_bf16_tn(X, H, stream=s)
    n = g.residual_norm(x, w_pre=x[0].contiguous(), stream=s.cuda_stream)
    s.synchronize()
    same([H], g.gemm_bf16_nt_gated(X, W, W)[:1])
    same(d, g.gemm_bf16_nt_gated_backward(X, W, W, H))
    same([C], [g.gemm_bf16_tn(X, H)])
    same([n.n, n.rstd_pre], [g.residual_norm(x, w_pre=x[0].contiguous())[i] for i in (1, 3)])


def guarded(shape, dtype, fill):
    """A tensor inside a larger buffer, and the buffer."""
    n = 1
    for s in shape:
        n *= s
    size = torch.empty(0, dtype=dtype).element_size()
    pad = 4096 // size
    buf = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    return buf[pad:pad + n].view(shape), buf, pad


@pytest.mark.parametrize("M", [1, 20, 65, 130, 257])
def test_nothing_outside_the_outputs_is_written(g, M):
    gen = torch.Generator(device="cuda").manual_seed(M)
    X, Wg, Wu, dH = randn(gen, M, 136), randn(gen, 264, 136), randn(gen, 264, 136), randn(gen, M, 264)
    x, w = randn(gen, M, 264), randn(gen, 264)
    r = torch.rand(M, generator=gen, device="cuda")
    A, (b, sf) = randn(gen, min(M, 16), 256), quantize(gen, 33, 256)
    T = lambda *s, dtype=BF16: guarded(s, dtype, 7.0)
    outs = {k: T(*s) for k, s in dict(H=(M, 264), gates=(2, M, 264), dX=(M, 136), dWg=(264, 136), dWu=(264, 136), C=(264, 136), y=(M, 264),
                                      n=(M, 264), dx=(M, 264), db=(M, 264), c=(min(M, 16), 33), h=(min(M, 16), 33)).items()}
    o = {k: v[0] for k, v in outs.items()}
    g.gemm_bf16_nt_gated(X, Wg, Wu, H=o["H"], gates=o["gates"])
    g.gemm_bf16_nt_gated_backward(X, Wg, Wu, dH, dX=o["dX"], dWg=o["dWg"], dWu=o["dWu"])
    g.gemm_bf16_tn(dH, X, C=o["C"])
    g.residual_norm(x, x, w_post=w, w_pre=w, y=o["y"], n=o["n"])
    g.residual_norm_backward(x, x, x, x, r, r, w_post=w, w_pre=w, dx=o["dx"], dblock=o["db"])
    g.gemv_w4a16(A, b, sf, 1.0, C=o["c"])
    g.gemv_w4a16_gated(A, b, sf, 1.0, b, sf, 1.0, H=o["h"])
    for name, (t, buf, pad) in outs.items():
        assert (buf[:pad] == 7.0).all() and (buf[-pad:] == 7.0).all(), name
        assert not (t == 7.0).all(), name


def test_weights_as_halves_of_one_matrix_and_shared(g):
    gen = torch.Generator(device="cuda").manual_seed(2)
    X, W = randn(gen, 140, 128), randn(gen, 2 * 264, 128)
    a = g.gemm_bf16_nt_gated(X, W[:264], W[264:])[0]
    same([a], [g.gemm_bf16_nt_gated(X, W[:264].clone(), W[264:].clone())[0]])
    H, G, U, eh, _, _ = ref.gated(X, W[:264], W[:264], "silu")
    ref.check(g.gemm_bf16_nt_gated(X, W[:264], W[:264])[0], H, eh, "one matrix twice")


def test_large_and_infinite_gates(g):
    """Gates far out on both sides, infinities and NaN: as the formula has them, and in
    their own row."""
    X = torch.zeros(130, 8, dtype=BF16, device="cuda")
    vals = [0.0, 1.0, -1.0, 80.0, -80.0, 1e4, -1e4, 3e38, -3e38, float("inf"), float("-inf"), float("nan")]
    X[: len(vals), 0] = torch.tensor(vals).to(BF16)
    X[:, 1] = 1.0
    Wg, Wu = torch.zeros(8, 8, dtype=BF16, device="cuda"), torch.zeros(8, 8, dtype=BF16, device="cuda")
    Wg[:, 0], Wu[:, 1] = 1.0, 2.0
    for M in (len(vals), 130):
        for kind in ("silu", "gelu_tanh"):
            H = g.gemm_bf16_nt_gated(X[:M].contiguous(), Wg, Wu, act=kind)[0].float()
            assert (H[0] == 0).all()
            # (an infinity or NaN meets the zeros of the weights: NaN in the whole row, as in gemm_bf16_nt)
            assert H[9].isnan().all() and H[10].isnan().all() and H[11].isnan().all()
            assert (H[5] == 2 * X[5, 0].float()).all() and H[7].isfinite().all() | H[7].isinf().all()
            assert (H[6].abs() <= 1e-30).all() and (H[8].abs() <= 1e-30).all()
            if M == 130:
                assert (H[12:] == 0).all()
    # stored gates: infinite ones through the gradient
    gates = torch.zeros(2, 2, 8, dtype=BF16, device="cuda")
    gates[0, 0], gates[1] = float("inf"), 1.0
    dX = g.gemm_bf16_nt_gated_backward(X[:2].contiguous(), Wg, Wu, torch.ones(2, 8, dtype=BF16, device="cuda"), gates=gates, need_dw=False)[0]
    assert not dX[0].isfinite().all() and dX[1].isfinite().all()


def test_python_refusals(g):
    gen = torch.Generator(device="cuda").manual_seed(0)
    X, W, x, w = randn(gen, 4, 64), randn(gen, 72, 64), randn(gen, 6, 64), randn(gen, 64)
    H = randn(gen, 4, 72)
    bad = [
        lambda: g.gemm_bf16_nt_gated(X.float(), W, W), lambda: g.gemm_bf16_nt_gated(X, W, W[:64]), lambda: g.gemm_bf16_nt_gated(X, W, W.cpu()),
        lambda: g.gemm_bf16_nt_gated(X, W, W, act="relu"), lambda: g.gemm_bf16_nt_gated(X[:, ::2], W, W), lambda: g.gemm_bf16_nt_gated(X, W, W, H=H[:3]),
        lambda: g.gemm_bf16_nt_gated_backward(X, W, W, H[:, :64].contiguous()), lambda: g.gemm_bf16_nt_gated_backward(X, W, W, H, dWg=W),
        lambda: g.gemm_bf16_nt_gated_backward(X, W, W, H, need_dx=False, need_dw=False), lambda: g.gemm_bf16_nt_gated_backward(X, W, W, H, gates=H),
        lambda: g.gemm_bf16_tn(X, H[:3]), lambda: g.gemm_bf16_tn(X, H.float()), lambda: g.gemm_bf16_tn(X, H, C=H),
        lambda: g.residual_norm(x), lambda: g.residual_norm(x, w_post=w), lambda: g.residual_norm(x, x, gate=randn(gen, 4, 64)),
        lambda: g.residual_norm(x.half(), w_pre=w), lambda: g.residual_norm(x, w_pre=w[:56]), lambda: g.residual_norm(x, w_pre=w.float()),
        lambda: g.residual_norm(x, w_pre=w, y=x), lambda: g.residual_norm(x, x, n=x), lambda: g.residual_norm(x.t(), w_pre=w[:6]),
        lambda: g.residual_norm_backward(None, None, x), lambda: g.residual_norm_backward(x, x, x), lambda: g.residual_norm_backward(x, None, x),
        lambda: g.residual_norm_backward(x, x, x.float(), rstd_pre=torch.ones(6, device="cuda"), w_pre=w),
        lambda: g.residual_norm_backward(x, x, x, w_pre=w), lambda: g.residual_norm_backward(x, None, None, x, w_post=w),
        lambda: g.gemv_w4a16(randn(gen, 17, 256), *quantize(gen, 8, 256), 1.0), lambda: g.gemv_w4a16(randn(gen, 2, 128), *quantize(gen, 8, 128), 1.0),
        lambda: g.gemv_w4a16(randn(gen, 2, 256), quantize(gen, 8, 256)[0], quantize(gen, 9, 256)[1], 1.0),
        lambda: g.gemv_w4a16_gated(randn(gen, 2, 256), *quantize(gen, 8, 256), 1.0, *quantize(gen, 16, 256), 1.0),
        lambda: g.gemv_w4a16(randn(gen, 0, 256), *quantize(gen, 8, 256), 1.0),
    ]
    for k, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError)):
            call()
            raise AssertionError(f"call {k} was accepted")
    # what only the library knows: alignment, overlap, empty, a short workspace
    for call in (lambda: g.gemm_bf16_nt_gated(X, W[:70].contiguous(), W[:70].contiguous()), lambda: g.gemm_bf16_nt_gated(X[:0], W, W),
                 lambda: g.gemm_bf16_nt_gated(X, W, W, H=W.view(-1)[:4 * 72].view(4, 72)), lambda: g.residual_norm(randn(gen, 3, 60), w_pre=randn(gen, 60)),
                 lambda: g.residual_norm(x, w_pre=w, n=x), lambda: g.gemm_bf16_tn(X[:0], H[:0]),
                 lambda: g.gemm_bf16_nt_gated_backward(X, W, W, H, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(g.GemmError):
            call()


def test_past_32_bit_offsets(g):
    """Outputs and weights of more than 2^31 elements and 2^32 bytes: rows near the end."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    rows = 140000
    pick = torch.tensor([0, 1, 65535, 131072, rows - 1], device="cuda")
    X, W = randn(gen, rows, 64), randn(gen, 16384, 64, scale=0.2)
    H = g.gemm_bf16_nt_gated(X, W, W)[0]  # 2.3e9 elements
    want, _, _, e, _, _ = ref.gated(X[pick], W, W, "silu")
    ref.check(H[pick], want, e, "H")
    dW = g.gemm_bf16_tn(H[:, :8].contiguous(), X)
    ref_dW = H[:, :8].to(F64).T @ X.to(F64)
    mags = H[:, :8].to(F64).abs().T @ X.to(F64).abs()
    ref.check(dW, ref_dW, ref.acc_bound(rows, mags) * 1.01 + ref.BF16_HALF * ref_dW.abs(), "tn over many rows")
    dX = g.gemm_bf16_nt_gated_backward(X, W, W, H, need_dw=False)[0]
    (wx, _, _), (ex, _, _) = ref.gated_backward(X[pick], W, W, H[pick], "silu")
    ref.check(dX[pick], wx, ex, "dX")
    del dX
    w = randn(gen, 16384)
    out = g.residual_norm(H, H, w_post=w, w_pre=w)
    y, n, _, _, ey, en = ref.norm(H[pick], H[pick], w, None, w, 1.0, 1e-6, out.y[pick])
    ref.check(out.y[pick], y, ey, "y")
    ref.check(out.n[pick], n, en, "n")
    back = g.residual_norm_backward(H, out.n, out.y, H, out.rstd_post, out.rstd_pre, w_post=w, w_pre=w, need_dw=False)
    want = ref.norm_backward(H[pick], out.n[pick], out.y[pick], H[pick], out.rstd_post[pick], out.rstd_pre[pick], w, None, w, 1.0, BF16)
    ref.check(back.dx[pick], *want["dx"], "dx")
    ref.check(back.dblock[pick], *want["dblock"], "dblock")
    del H, out, back
    F, K = 300000, 8192  # 2.5e9 weights
    Wg, X = torch.empty(F, K, dtype=BF16, device="cuda"), randn(gen, 3, K)
    Wg.view(-1).view(torch.int16).random_(0x3C00, 0x3D00, generator=gen)  # 2^-7 to 2^-5
    at = torch.tensor([0, 131071, 262144, F - 1], device="cuda")
    want, _, _, e, _, _ = ref.gated(X, Wg[at], Wg[at], "silu")
    ref.check(g.gemm_bf16_nt_gated(X, Wg, Wg)[0][:, at], want, e, "H of few tokens")
    del Wg
    N, K = 560000, 8192  # 2.3e9 code bytes
    b = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=torch.uint8)
    sf = torch.full((N, K // 16), 56, device="cuda", dtype=torch.uint8)
    A = randn(gen, 2, K)
    at = torch.tensor([0, 262143, 524288, N - 1], device="cuda")
    want, e = ref.few_tokens(A, b[at], sf[at], 0.01)
    ref.check(g.gemv_w4a16(A, b, sf, 0.01)[:, at], want, e * 1.01 + ref.BF16_HALF * want.abs(), "gemv")
