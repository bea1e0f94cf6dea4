"""Host-side checks of the C entry points of a feed-forward block's operators: bad
arguments are refused before anything touches a device."""
from __future__ import annotations

import pytest

from test_abi import lib  # noqa: F401  (the built library)

P = 0x1000000  # 16-byte aligned fake addresses, 16 MB apart; never dereferenced
BIG = 1 << 23


def gated(lib, **kw):
    a = dict(X=P, Wg=2 * P, Wu=3 * P, H=4 * P, gates=5 * P, act=0, M=40, F=200, K=64)
    a.update(kw)
    return lib.gemm_bf16_nt_gated(a["X"], a["Wg"], a["Wu"], a["H"], a["gates"], a["act"], a["M"], a["F"], a["K"], None)


@pytest.mark.parametrize("kw,expect", [
    ({"X": 0}, 1), ({"Wg": 0}, 1), ({"Wu": 0}, 1), ({"H": 0}, 1),
    ({"M": 0}, 2), ({"F": -8}, 2), ({"K": 0}, 2), ({"act": 2}, 2), ({"act": -1}, 2), ({"M": (1 << 30) + 1}, 2),
    ({"F": (1 << 29) + 8}, 2), ({"M": 1 << 30, "F": 1 << 29}, 2),
    ({"X": P + 8}, 3), ({"Wg": 2 * P + 2}, 3), ({"Wu": 3 * P + 4}, 3), ({"H": 4 * P + 8}, 3), ({"gates": 5 * P + 8}, 3),
    ({"F": 204}, 3), ({"K": 60}, 3),
    ({"H": P}, 4), ({"H": 2 * P + 16}, 4), ({"gates": 3 * P}, 4), ({"gates": 4 * P + 16}, 4), ({"gates": 4 * P - 2 * 40 * 200 * 2 + 16}, 4),
])
def test_gated_rejects_bad_arguments(lib, kw, expect):  # noqa: F811
    assert gated(lib, **kw) == expect


def gated_backward(lib, **kw):
    a = dict(X=P, Wg=2 * P, Wu=3 * P, dH=4 * P, gates=5 * P, dX=6 * P, dWg=7 * P, dWu=8 * P, ws=9 * P, n=BIG, act=1, M=40, F=200, K=64)
    a.update(kw)
    return lib.gemm_bf16_nt_gated_backward(a["X"], a["Wg"], a["Wu"], a["dH"], a["gates"], a["dX"], a["dWg"], a["dWu"], a["ws"], a["n"],
                                           a["act"], a["M"], a["F"], a["K"], None)


@pytest.mark.parametrize("kw,expect", [
    ({"X": 0}, 1), ({"Wg": 0}, 1), ({"Wu": 0}, 1), ({"dH": 0}, 1), ({"ws": 0}, 1), ({"dWg": 0}, 1), ({"dWu": 0}, 1),
    ({"dX": 0, "dWg": 0, "dWu": 0}, 1),
    ({"M": -1}, 2), ({"act": 7}, 2), ({"n": 40 * 200 * 4 - 1}, 2),
    ({"F": 100}, 3), ({"dH": 4 * P + 8}, 3), ({"dX": 6 * P + 2}, 3), ({"dWg": 7 * P + 8}, 3), ({"dWu": 8 * P + 4}, 3), ({"ws": 9 * P + 8}, 3),
    ({"gates": 5 * P + 2}, 3),
    ({"dX": P}, 4), ({"dWg": 3 * P}, 4), ({"dWu": 7 * P + 16}, 4), ({"ws": 5 * P}, 4), ({"dX": 4 * P}, 4), ({"ws": 8 * P}, 4),
    ({"gates": 0, "ws": 4 * P}, 4),
])
def test_gated_backward_rejects_bad_arguments(lib, kw, expect):  # noqa: F811
    assert gated_backward(lib, **kw) == expect


def tn(lib, **kw):
    a = dict(A=P, B=2 * P, C=3 * P, ws=4 * P, n=BIG, M=64, N=72, K=4096)
    a.update(kw)
    return lib.gemm_bf16_tn(a["A"], a["B"], a["C"], a["ws"], a["n"], a["M"], a["N"], a["K"], None)


@pytest.mark.parametrize("kw,expect", [
    ({"A": 0}, 1), ({"B": 0}, 1), ({"C": 0}, 1), ({"ws": 0}, 1),
    ({"M": 0}, 2), ({"N": -8}, 2), ({"K": 0}, 2), ({"M": 1 << 30, "N": 1 << 30}, 2), ({"n": 64 * 72 * 4}, 2),
    ({"A": P + 8}, 3), ({"B": 2 * P + 2}, 3), ({"C": 3 * P + 4}, 3), ({"ws": 4 * P + 8}, 3), ({"M": 60}, 3), ({"N": 76}, 3),
    ({"C": P + 16}, 4), ({"C": 2 * P}, 4), ({"ws": P}, 4), ({"ws": 3 * P + 16}, 4),
])
def test_tn_rejects_bad_arguments(lib, kw, expect):  # noqa: F811
    assert tn(lib, **kw) == expect


def norm(lib, **kw):
    a = dict(x=P, b=2 * P, wo=3 * P, g=4 * P, wi=5 * P, y=6 * P, n=7 * P, ro=8 * P, ri=9 * P, eps=1e-6, f32=0, M=40, D=64, rows=20)
    a.update(kw)
    return lib.residual_norm(a["x"], a["b"], a["wo"], a["g"], a["wi"], a["y"], a["n"], a["ro"], a["ri"], 1.0, a["eps"], a["f32"], a["M"], a["D"],
                             a["rows"], None)


@pytest.mark.parametrize("kw,expect", [
    ({"x": 0}, 1), ({"y": 0}, 1), ({"n": 0}, 1), ({"b": 0}, 1), ({"b": 0, "y": 0}, 1), ({"b": 0, "y": 0, "wo": 0}, 1),
    ({"wi": 0}, 1), ({"wi": 0, "n": 0}, 1), ({"wo": 0}, 1),
    ({"b": 0, "y": 0, "wo": 0, "g": 0, "ro": 0, "wi": 0, "n": 0, "ri": 0}, 1),
    ({"M": 0}, 2), ({"D": 0}, 2), ({"D": 16392}, 2), ({"rows": 0}, 2), ({"rows": 13}, 2), ({"rows": 80}, 2), ({"eps": -1e-6}, 2), ({"eps": float("nan")}, 2),
    ({"D": 60}, 3), ({"x": P + 8}, 3), ({"g": 4 * P + 2}, 3), ({"n": 7 * P + 4}, 3), ({"ro": 8 * P + 2}, 3), ({"ri": 9 * P + 1}, 3),
    ({"y": P + 16}, 4), ({"y": 2 * P}, 4), ({"n": P}, 4), ({"n": 6 * P}, 4), ({"ro": 3 * P}, 4), ({"ri": 4 * P + 240}, 4),
])
def test_residual_norm_rejects_bad_arguments(lib, kw, expect):  # noqa: F811
    assert norm(lib, **kw) == expect


def norm_backward(lib, **kw):
    a = dict(dy=P, dn=2 * P, y=3 * P, b=4 * P, ro=5 * P, ri=6 * P, wo=7 * P, g=8 * P, wi=9 * P, dx=10 * P, db=11 * P, dwo=12 * P, dg=13 * P, dwi=14 * P,
             ws=15 * P, bytes=BIG, f32=1, M=40, D=64, rows=20)
    a.update(kw)
    return lib.residual_norm_backward(a["dy"], a["dn"], a["y"], a["b"], a["ro"], a["ri"], a["wo"], a["g"], a["wi"], a["dx"], a["db"], a["dwo"], a["dg"],
                                      a["dwi"], a["ws"], a["bytes"], 1.0, a["f32"], a["M"], a["D"], a["rows"], None)


@pytest.mark.parametrize("kw,expect", [
    ({"dx": 0}, 1), ({"dy": 0, "dn": 0, "wi": 0, "dwi": 0}, 1), ({"dn": 0}, 1), ({"y": 0}, 1), ({"ri": 0}, 1), ({"ro": 0}, 1), ({"db": 0}, 1), ({"b": 0}, 1),
    ({"wi": 0}, 1), ({"wo": 0}, 1), ({"g": 0}, 1), ({"ws": 0}, 1), ({"b": 0, "db": 0}, 1),
    ({"M": -3}, 2), ({"D": 16384 + 8}, 2), ({"rows": 7}, 2), ({"bytes": 64}, 2),
    ({"D": 12}, 3), ({"dx": 10 * P + 8}, 3), ({"dwo": 12 * P + 4}, 3), ({"ws": 15 * P + 8}, 3), ({"ri": 6 * P + 2}, 3),
    ({"dx": P + 16}, 4), ({"dx": 2 * P}, 4), ({"db": 4 * P}, 4), ({"dwi": 12 * P + 16}, 4), ({"dg": 9 * P}, 4), ({"ws": 10 * P}, 4),
])
def test_residual_norm_backward_rejects_bad_arguments(lib, kw, expect):  # noqa: F811
    assert norm_backward(lib, **kw) == expect


def gemv(lib, **kw):
    a = dict(A=P, b=2 * P, sf=3 * P, C=4 * P, M=3, N=40, K=512)
    a.update(kw)
    return lib.gemv_w4a16(a["A"], a["b"], a["sf"], 1.0, a["C"], a["M"], a["N"], a["K"], None)


@pytest.mark.parametrize("kw,expect", [
    ({"A": 0}, 1), ({"b": 0}, 1), ({"sf": 0}, 1), ({"C": 0}, 1),
    ({"M": 0}, 2), ({"M": 17}, 2), ({"N": 0}, 2), ({"K": -256}, 2), ({"N": (1 << 30) + 1}, 2),
    ({"K": 128}, 3), ({"A": P + 8}, 3), ({"b": 2 * P + 4}, 3), ({"sf": 3 * P + 8}, 3), ({"C": 4 * P + 1}, 3),
    ({"C": P}, 4), ({"C": 2 * P + 1024}, 4), ({"C": 3 * P + 2}, 4),
])
def test_gemv_rejects_bad_arguments(lib, kw, expect):  # noqa: F811
    assert gemv(lib, **kw) == expect


def gemv_gated(lib, **kw):
    a = dict(A=P, bg=2 * P, sg=3 * P, bu=4 * P, su=5 * P, H=6 * P, act=0, M=3, F=40, K=512)
    a.update(kw)
    return lib.gemv_w4a16_gated(a["A"], a["bg"], a["sg"], 1.0, a["bu"], a["su"], 1.0, a["H"], a["act"], a["M"], a["F"], a["K"], None)


@pytest.mark.parametrize("kw,expect", [
    ({"A": 0}, 1), ({"bg": 0}, 1), ({"sg": 0}, 1), ({"bu": 0}, 1), ({"su": 0}, 1), ({"H": 0}, 1),
    ({"M": 17}, 2), ({"F": 0}, 2), ({"act": 2}, 2), ({"K": 300}, 3), ({"bu": 4 * P + 8}, 3), ({"su": 5 * P + 2}, 3),
    ({"H": 4 * P}, 4), ({"H": 5 * P}, 4), ({"H": 3 * P}, 4),
])
def test_gemv_gated_rejects_bad_arguments(lib, kw, expect):  # noqa: F811
    assert gemv_gated(lib, **kw) == expect


def test_workspace_sizes(lib):  # noqa: F811
    f = lib.gemm_bf16_nt_gated_backward_workspace_bytes
    assert f(0, 8, 8) == 0 and f(8, -8, 8) == 0 and f(8, (1 << 29) + 8, 8) == 0
    assert f(5120, 11008, 2048) >= 5120 * 11008 * 4
    # dX of few tokens is summed from parts of a long K loop
    assert f(1, 11008, 2048) > 11008 * 4 + 2048 * 4
    t = lib.gemm_bf16_tn_workspace_bytes
    assert t(0, 8, 8) == 0 and t(2048, 11008, 5120) == 0   # tiles enough
    assert t(64, 72, 4096) >= 2 * 64 * 72 * 4              # one tile, a long K
    n = lib.residual_norm_backward_workspace_bytes
    assert n(100, 64, 100, 0, 0) == 0                            # no gradient of a weight: none
    assert n(100, 60, 100, 1, 0) == 0 and n(100, 64, 30, 1, 1) == 0  # invalid
    assert 0 < n(100000, 8192, 100000, 2, 1) < 32 << 20          # by the blocks, not by the rows
