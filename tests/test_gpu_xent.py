"""Linear cross entropy against its definition in 64 bits, on the GPU.

Tolerances.  A logit is a sum of K FP32-accumulated products: its error is at
most (K + 8) 2^-23 times the row's sum of |x||w| (`dz` below; 2^-23 allows for
truncating adders).  The loss and lse then carry dz (2 dz for the loss), the
exponential's 2^-21 and the sums' rounding.  A gradient term
g = d (exp(z - lse) - [target]) carries |d| p (dz + error of lse + 2^-20) and
its rounding to BF16, 2^-8 |g| (one unit in the last place covers both
neighbours); the products add FP32 summation error and the result's own
rounding.  Every bound is evaluated element by element in 64 bits.
"""
from __future__ import annotations

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


def problem(M, V, K, seed, scale=2.0, ignored=0.2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    W = (torch.randn(V, K, generator=gen, device="cuda") * (scale / K ** 0.5)).bfloat16()
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    if M > 2:
        t[torch.rand(M, generator=gen, device="cuda") < ignored] = -100
        t[0], t[M - 1] = V - 1, 0     # the first and the last column are targets
    d = torch.rand(M, generator=gen, device="cuda") * 2 - 0.5
    return X, W, t, d


def reference(X, W, t):
    x, w = X.to(F64), W.to(F64)
    z = x @ w.T
    lse = torch.logsumexp(z, dim=1)
    pick = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    loss = torch.where(t >= 0, lse - pick, torch.zeros_like(lse))
    K = X.shape[1]
    dz = ((K + 8) * 2.0 ** -23) * (x.abs() @ w.abs().T).amax(dim=1)
    V = W.shape[0]
    dlse = dz + 2.0 ** -20 + (V / 256 + 80) * 2.0 ** -24 + lse.abs() * 2.0 ** -22
    return z, lse, loss, dz, dlse


def check_forward(loss, lse, ref):
    z, rlse, rloss, dz, dlse = ref
    assert ((lse.to(F64) - rlse).abs() <= dlse).all()
    assert ((loss.to(F64) - rloss).abs() <= dlse + dz + 2.0 ** -22 * rlse.abs()).all()


def gradients(X, W, t, lse, d):
    """Reference gradients and the bounds of their errors."""
    x, w = X.to(F64), W.to(F64)
    K, (M, V) = X.shape[1], (X.shape[0], W.shape[0])
    z = x @ w.T
    dz = ((K + 8) * 2.0 ** -23) * (x.abs() @ w.abs().T).amax(dim=1, keepdim=True)
    p = torch.exp(z - lse.to(F64)[:, None])
    live = (t >= 0)[:, None]
    dd = torch.where(live, d.to(F64)[:, None], torch.zeros(1, 1, dtype=F64, device=X.device))
    G = p.clone()
    G.scatter_add_(1, t.clamp(min=0)[:, None], -torch.ones(M, 1, dtype=F64, device=X.device))
    G = G * dd
    err = dd.abs() * p * (dz + 2.0 ** -20) + 2.0 ** -8 * G.abs() + 2.0 ** -130
    dX, dW = G @ w, G.T @ x
    eX = err @ w.abs() + (V + 64) * 2.0 ** -23 * (G.abs() @ w.abs()) + 2.0 ** -8 * dX.abs()
    eW = err.T @ x.abs() + (M + 64) * 2.0 ** -23 * (G.abs().T @ x.abs()) + 2.0 ** -8 * dW.abs()
    return dX, dW, eX, eW


SHAPES = [
    (1, 1, 8),            # one class: loss 0
    (1, 1000, 64),        # one token
    (2, 255, 8),          # a column short of a tile
    (37, 257, 72),        # one column past a tile, K tail
    (128, 4096, 256),     # single-CTA limit
    (129, 777, 264),      # first pair size, ragged everywhere
    (300, 2049, 200),     # two row blocks
    (640, 512, 1024),     # exact multiples
    (513, 33, 40),        # fewer classes than a 64-column chunk
    (1000, 5003, 520),    # split dX sums with a ragged K
]


@pytest.mark.parametrize("M,V,K", SHAPES)
def test_forward_and_backward(g, M, V, K):
    X, W, t, d = problem(M, V, K, 1000 + M + V + K)
    loss, lse = g.gemm_bf16_nt_xent(X, W, t)
    ref = reference(X, W, t)
    check_forward(loss, lse, ref)
    dX, dW = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    rX, rW, eX, eW = gradients(X, W, t, lse, d)
    assert ((dX.to(F64) - rX).abs() <= eX).all()
    assert ((dW.to(F64) - rW).abs() <= eW).all()
    # one gradient alone is the same gradient
    only_x, none = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d, need_dw=False)
    assert none is None and torch.equal(only_x, dX)
    none, only_w = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d, need_dx=False)
    assert none is None and torch.equal(only_w, dW)


@pytest.mark.parametrize("M,V,K", [
    (16411, 9001, 72),    # three pieces of the vocabulary, the last one short
    (20000, 12345, 2056), # pieces, K tail, several tiles of dX
])
def test_pieces_of_the_vocabulary(g, M, V, K):
    X, W, t, d = problem(M, V, K, 5)
    loss, lse = g.gemm_bf16_nt_xent(X, W, t)
    dX, dW = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    check_forward(loss, lse, reference(X, W, t))
    rX, rW, eX, eW = gradients(X, W, t, lse, d)
    assert ((dX.to(F64) - rX).abs() <= eX).all()
    assert ((dW.to(F64) - rW).abs() <= eW).all()
    again = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dW)   # fixed order of sums


@pytest.mark.parametrize("M,V,K", [
    (1, 1849, 72), (64, 1849, 328),       # tiles of 64 vocabulary rows
    (3, 4902, 136), (64, 4865, 40),       # of 128
    (17, 23300, 64), (128, 9000, 264),    # of 192
    (33, 32769, 24), (100, 19456, 1032),  # of 256
])
def test_tile_heights_of_few_tokens(g, M, V, K):
    X, W, t, d = problem(M, V, K, 31 + V)
    loss, lse = g.gemm_bf16_nt_xent(X, W, t)
    check_forward(loss, lse, reference(X, W, t))
    dX, dW = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    rX, rW, eX, eW = gradients(X, W, t, lse, d)
    assert ((dX.to(F64) - rX).abs() <= eX).all()
    assert ((dW.to(F64) - rW).abs() <= eW).all()


@pytest.mark.parametrize("M,V,K", [
    (1000, 20000, 520),    # dW's first clusters take more tiles than the others
    (300, 30011, 1032),    # many parts of dX, more than one round of dW
    (16411, 20001, 72),    # six pieces, whose G grids start early too
    (128, 530001, 40),     # few tokens in two pieces
])
def test_grids_that_start_early(g, M, V, K):
    X, W, t, d = problem(M, V, K, 37)
    loss, lse = g.gemm_bf16_nt_xent(X, W, t)
    dX, dW = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    rX, rW, eX, eW = gradients(X, W, t, lse, d)
    assert ((dX.to(F64) - rX).abs() <= eX).all()
    assert ((dW.to(F64) - rW).abs() <= eW).all()
    for _ in range(5):
        again = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
        assert torch.equal(again[0], dX) and torch.equal(again[1], dW)


def test_concurrent_streams_and_threads(g):
    # two host threads, a stream and a workspace each, on the same weights
    import threading
    cases = [problem(M, 6000, 256, 41 + M) for M in (50, 300)]
    want = []
    for X, W, t, d in cases:
        loss, lse = g.gemm_bf16_nt_xent(X, W, t)
        want.append((loss, lse, *g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)))
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            X, W, t, d = cases[i]
            s = torch.cuda.Stream()
            for _ in range(20):
                loss, lse = g.gemm_bf16_nt_xent(X, W, t, stream=s)
                got[i].append((loss, lse, *g.gemm_bf16_nt_xent_backward(X, W, t, lse, d, stream=s)))
            s.synchronize()
        except Exception as e:  # noqa: BLE001 (reported by the main thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors
    for i in range(2):
        assert len(got[i]) == 20
        for res in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(res, want[i]))


@pytest.mark.parametrize("M", [100, 300])
def test_gradients_against_differences(g, M):
    V, K = 600, 64
    X, W, t, d = problem(M, V, K, 77)
    _, lse = g.gemm_bf16_nt_xent(X, W, t)
    dX, dW = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    _, _, eX, eW = gradients(X, W, t, lse, d)
    gen = torch.Generator(device="cuda").manual_seed(3)

    def total(x, w):
        z = x @ w.T
        l = torch.logsumexp(z, dim=1) - z.gather(1, t.clamp(min=0)[:, None])[:, 0]
        return (d.to(F64) * torch.where(t >= 0, l, torch.zeros_like(l))).sum()

    x, w, h = X.to(F64), W.to(F64), 1e-4
    for _ in range(4):
        ux = torch.randn(M, K, generator=gen, device="cuda", dtype=F64)
        uw = torch.randn(V, K, generator=gen, device="cuda", dtype=F64)
        num = (total(x + h * ux, w) - total(x - h * ux, w)) / (2 * h)
        # third derivative of a row's loss along u: at most 8 max|u.w|^3
        rest = h * h / 6 * (d.abs() * 8 * (ux @ w.T).abs().amax(dim=1) ** 3).sum() + 1e-9
        assert (num - (dX.to(F64) * ux).sum()).abs() <= (eX * ux.abs()).sum() + rest
        num = (total(x, w + h * uw) - total(x, w - h * uw)) / (2 * h)
        rest = h * h / 6 * (d.abs() * 8 * (x @ uw.T).abs().amax(dim=1) ** 3).sum() + 1e-9
        assert (num - (dW.to(F64) * uw).sum()).abs() <= (eW * uw.abs()).sum() + rest


@pytest.mark.parametrize("M", [5, 200])
def test_rows_without_a_loss(g, M):
    X, W, t, d = problem(M, 300, 64, 9)
    t[:] = -1
    loss, lse = g.gemm_bf16_nt_xent(X, W, t)
    assert (loss == 0).all() and torch.isfinite(lse).all()
    d[:] = float("nan")                        # not used in such rows
    dX, dW = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    assert (dX == 0).all() and (dW == 0).all()


@pytest.mark.parametrize("M", [7, 300])
def test_target_past_the_vocabulary_is_loud(g, M):
    V = 300
    X, W, t, d = problem(M, V, 64, 11, ignored=0.0)
    bad = M // 2
    t[bad] = V
    loss, lse = g.gemm_bf16_nt_xent(X, W, t)
    assert torch.isnan(loss[bad]) and torch.isfinite(lse).all()
    ok = torch.arange(M, device="cuda") != bad
    assert torch.isfinite(loss[ok]).all()
    dX, dW = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    assert torch.isnan(dX[bad]).all() and torch.isfinite(dX[ok]).all() and torch.isnan(dW).all()
    t[bad] = 2 ** 40                           # past 32 bits
    assert torch.isnan(g.gemm_bf16_nt_xent(X, W, t)[0][bad])
    t[bad] = -2 ** 40
    assert g.gemm_bf16_nt_xent(X, W, t)[0][bad] == 0


@pytest.mark.parametrize("M", [7, 300])
def test_non_finite_rows_stay_in_their_row(g, M):
    V = 700
    X, W, t, d = problem(M, V, 64, 13, ignored=0.0)
    clean = g.gemm_bf16_nt_xent(X, W, t)
    X2 = X.clone()
    X2[2, 5] = float("nan")
    X2[3, 5] = float("inf")
    loss, lse = g.gemm_bf16_nt_xent(X2, W, t)
    assert torch.isnan(loss[2:4]).all() and torch.isnan(lse[2:4]).all()
    ok = torch.ones(M, dtype=torch.bool, device="cuda")
    ok[2:4] = False
    assert torch.equal(loss[ok], clean[0][ok]) and torch.equal(lse[ok], clean[1][ok])
    # the same rows without a loss: their gradient is zero, the others' untouched
    t[2:4] = -100
    dX0, _ = g.gemm_bf16_nt_xent_backward(X, W, t, clean[1], d, need_dw=False)
    dX, _ = g.gemm_bf16_nt_xent_backward(X2, W, t, lse, d, need_dw=False)
    assert (dX[2:4] == 0).all() and torch.equal(dX[ok], dX0[ok])


def test_extreme_logits(g):
    # logits of +-3e4: the maximum is subtracted before any exponential
    M, V, K = 150, 400, 64
    X = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    W = torch.zeros(V, K, device="cuda", dtype=torch.bfloat16)
    X[:, 0] = 256
    W[:, 0] = torch.arange(V, device="cuda") - 200.0
    t = torch.arange(M, device="cuda") + 250
    loss, lse = g.gemm_bf16_nt_xent(X, W, t)
    z = X.to(F64) @ W.to(F64).T
    want = torch.logsumexp(z, dim=1)
    assert ((lse.to(F64) - want).abs() <= 2.0 ** -20 * want.abs()).all()
    assert ((loss.to(F64) - (want - z[torch.arange(M), t])).abs() <= 2.0 ** -20 * want.abs()).all()


@pytest.mark.parametrize("M,V,K", [(64, 1000, 128), (300, 1000, 128)])
def test_outputs_stay_inside_their_buffers(g, M, V, K):
    X, W, t, d = problem(M, V, K, 15)
    pad = 512

    def framed(n, dtype):
        buf = torch.full((n + 2 * pad,), 7.0, device="cuda", dtype=dtype)
        return buf, buf[pad:pad + n]

    bl, loss = framed(M, torch.float32)
    bs, lse = framed(M, torch.float32)
    need = g.gemm_bf16_nt_xent_workspace_bytes(M, V)
    wbuf = torch.full((need + 2 * pad,), 7, device="cuda", dtype=torch.uint8)
    g.gemm_bf16_nt_xent(X, W, t, loss=loss, lse=lse, workspace=wbuf[pad:pad + need])
    bx, dx = framed(M * K, torch.bfloat16)
    bw, dw = framed(V * K, torch.bfloat16)
    need = g.gemm_bf16_nt_xent_backward_workspace_bytes(M, V, K)
    w2 = torch.full((need + 2 * pad,), 7, device="cuda", dtype=torch.uint8)
    g.gemm_bf16_nt_xent_backward(X, W, t, lse, d, dX=dx.view(M, K), dW=dw.view(V, K),
                                 workspace=w2[pad:pad + need])
    for b in (bl, bs, bx, bw, wbuf, w2):
        assert (b[:pad] == 7).all() and (b[-pad:] == 7).all()
    want = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    assert torch.equal(dx.view(M, K), want[0]) and torch.equal(dw.view(V, K), want[1])


def test_another_stream_and_graph_replay(g):
    M, V, K = 300, 3001, 256
    X, W, t, d = problem(M, V, K, 17)
    loss, lse = g.gemm_bf16_nt_xent(X, W, t)
    dX, dW = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    l2, s2 = g.gemm_bf16_nt_xent(X, W, t, stream=s)
    x2, w2 = g.gemm_bf16_nt_xent_backward(X, W, t, s2, d, stream=s)
    s.synchronize()
    assert torch.equal(l2, loss) and torch.equal(x2, dX) and torch.equal(w2, dW)
    graph = torch.cuda.CUDAGraph()
    l3, s3 = torch.empty_like(loss), torch.empty_like(lse)
    x3, w3 = torch.empty_like(dX), torch.empty_like(dW)
    ws = torch.empty(g.gemm_bf16_nt_xent_workspace_bytes(M, V), dtype=torch.uint8, device="cuda")
    wb = torch.empty(g.gemm_bf16_nt_xent_backward_workspace_bytes(M, V, K), dtype=torch.uint8,
                     device="cuda")
    with torch.cuda.graph(graph):
        g.gemm_bf16_nt_xent(X, W, t, loss=l3, lse=s3, workspace=ws)
        g.gemm_bf16_nt_xent_backward(X, W, t, s3, d, dX=x3, dW=w3, workspace=wb)
    for _ in range(3):
        for b in (l3, s3, x3, w3):
            b.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(l3, loss) and torch.equal(x3, dX) and torch.equal(w3, dW)


def test_calls_in_a_row_share_a_workspace(g):
    # the next call starts while the last grids of the previous one run
    cases = [problem(M, V, K, 19 + M) for M, V, K in ((300, 3001, 256), (100, 2000, 64), (700, 900, 512))]
    want = []
    for X, W, t, d in cases:
        _, lse = g.gemm_bf16_nt_xent(X, W, t)
        want.append((lse, *g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)))
    torch.cuda.synchronize()
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(5):
        for X, W, t, d in cases:
            _, lse = g.gemm_bf16_nt_xent(X, W, t, workspace=ws)
            got.append((lse, *g.gemm_bf16_nt_xent_backward(X, W, t, lse, d, workspace=ws)))
    torch.cuda.synchronize()
    for i, res in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(res, want[i % 3]))


@pytest.mark.parametrize("M,V,K", [
    (40, 530000, 4104),      # W and dW past 2^32 bytes and 2^31 elements
    (530000, 300, 4104),     # X and dX past them
])
def test_offsets_past_32_bits(g, M, V, K):
    gen = torch.Generator(device="cuda").manual_seed(23)
    X = torch.randn(M, K, generator=gen, device="cuda", dtype=torch.bfloat16)
    W = torch.randn(V, K, generator=gen, device="cuda", dtype=torch.bfloat16) * (2 / K ** 0.5)
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    t[0], t[-1] = V - 1, V - 2
    d = torch.ones(M, device="cuda")
    loss, lse = g.gemm_bf16_nt_xent(X, W, t)
    dX, dW = g.gemm_bf16_nt_xent_backward(X, W, t, lse, d)
    rows = torch.cat([torch.arange(0, min(M, 16)), torch.arange(max(0, M - 16), M)]).unique().cuda()
    cols = torch.cat([torch.arange(0, 16), torch.arange(V - 16, V)]).unique().cuda()
    step = 8192
    x = X[rows].to(F64)
    z = torch.cat([x @ W[v:v + step].to(F64).T for v in range(0, V, step)], dim=1)
    want = torch.logsumexp(z, dim=1)
    dz = (K + 8) * 2.0 ** -23 * (x.abs() @ W[:4096].to(F64).abs().T).amax() * 1.5
    assert ((lse[rows].to(F64) - want).abs() <= dz + 2.0 ** -20 + (V / 256 + 80) * 2.0 ** -24).all()
    G = torch.exp(z - lse[rows].to(F64)[:, None])
    G[torch.arange(len(rows)), t[rows]] -= 1
    gx = sum(G[:, v:v + step] @ W[v:v + step].to(F64) for v in range(0, V, step))
    ga = sum(G[:, v:v + step].abs() @ W[v:v + step].to(F64).abs() for v in range(0, V, step))
    assert ((dX[rows].to(F64) - gx).abs() <= (2.0 ** -8 + 2 * dz) * ga + 2.0 ** -8 * gx.abs()).all()
    gw = torch.zeros(len(cols), K, dtype=F64, device="cuda")
    aw = torch.zeros_like(gw)
    w = W[cols].to(F64)
    for m in range(0, M, step):
        xm = X[m:m + step].to(F64)
        q = torch.exp(xm @ w.T - lse[m:m + step].to(F64)[:, None])
        q -= (t[m:m + step][:, None] == cols[None, :]).to(F64)
        gw += q.T @ xm
        aw += q.abs().T @ xm.abs()
    assert ((dW[cols].to(F64) - gw).abs() <=
            (2.0 ** -8 + 2 * dz + (M + 64) * 2.0 ** -23) * aw + 2.0 ** -8 * gw.abs()).all()


def test_refusals(g):
    X, W, t, d = problem(40, 200, 64, 29)
    loss, lse = g.gemm_bf16_nt_xent(X, W, t)
    with pytest.raises(TypeError):
        g.gemm_bf16_nt_xent(X.float(), W, t)
    with pytest.raises(TypeError):
        g.gemm_bf16_nt_xent(X, W, t.int())
    with pytest.raises(ValueError):
        g.gemm_bf16_nt_xent(X, W[:, :32].contiguous(), t)
    with pytest.raises(ValueError):
        g.gemm_bf16_nt_xent(X, W, t[:39])
    with pytest.raises(ValueError):
        g.gemm_bf16_nt_xent(X[:, ::2], W[:, ::2], t)
    with pytest.raises(ValueError):
        g.gemm_bf16_nt_xent(X, W, t.cpu())
    with pytest.raises(g.GemmError):                       # K % 8
        g.gemm_bf16_nt_xent(X[:, :60].contiguous(), W[:, :60].contiguous(), t)
    with pytest.raises(g.GemmError):                       # workspace too small
        g.gemm_bf16_nt_xent(X, W, t, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(g.GemmError):                       # loss on lse
        g.gemm_bf16_nt_xent(X, W, t, loss=lse, lse=lse)
    with pytest.raises(ValueError):
        g.gemm_bf16_nt_xent_backward(X, W, t, lse, d, need_dx=False, need_dw=False)
    with pytest.raises(ValueError):
        g.gemm_bf16_nt_xent_backward(X, W, t, lse, d[:39])
    with pytest.raises(ValueError):
        g.gemm_bf16_nt_xent_backward(X, W, t, lse, d, dX=torch.empty_like(W))
    with pytest.raises(g.GemmError):                       # dX in X
        g.gemm_bf16_nt_xent_backward(X, W, t, lse, d, dX=X)
