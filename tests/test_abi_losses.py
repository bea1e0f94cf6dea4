"""Host-side checks of the loss operators' C entry points: bad arguments are
refused before anything touches a device."""
from __future__ import annotations

import pytest

from test_abi import lib  # noqa: F401  (the built library)

P = 0x1000000  # 16-byte aligned fake addresses, 16 MB apart; never dereferenced
BIG = 1 << 23


def xent(lib, **kw):
    a = dict(X=P, W=2 * P, target=3 * P, loss=4 * P, lse=5 * P, ws=6 * P, n=BIG, M=40, V=200, K=64)
    a.update(kw)
    return lib.gemm_bf16_nt_xent(a["X"], a["W"], a["target"], a["loss"], a["lse"], a["ws"], a["n"],
                                 a["M"], a["V"], a["K"], None)


@pytest.mark.parametrize("kw,expect", [
    ({"X": 0}, 1), ({"W": 0}, 1), ({"target": 0}, 1), ({"loss": 0}, 1), ({"lse": 0}, 1), ({"ws": 0}, 1),
    ({"M": 0}, 2), ({"V": -1}, 2), ({"K": 0}, 2), ({"M": (1 << 30) + 1}, 2), ({"V": 0x7FFFFFFF}, 2),
    ({"M": 1 << 30, "V": 1 << 30}, 2),             # too many tiles
    ({"n": 40 * 8 - 1}, 2),                        # workspace a byte short
    ({"K": 60}, 3), ({"X": P + 8}, 3), ({"W": 2 * P + 2}, 3), ({"target": 3 * P + 4}, 3),
    ({"loss": 4 * P + 2}, 3), ({"lse": 5 * P + 1}, 3), ({"ws": 6 * P + 8}, 3),
    ({"loss": P}, 4), ({"lse": 4 * P + 8}, 4), ({"ws": 2 * P + 64}, 4), ({"loss": 3 * P}, 4), ({"ws": 5 * P}, 4),
])
def test_xent_rejects_bad_arguments(lib, kw, expect):  # noqa: F811
    assert xent(lib, **kw) == expect


def xent_backward(lib, **kw):
    a = dict(X=P, W=2 * P, target=3 * P, lse=4 * P, dloss=5 * P, dX=6 * P, dW=7 * P, ws=8 * P, n=BIG, M=40, V=200, K=64)
    a.update(kw)
    return lib.gemm_bf16_nt_xent_backward(a["X"], a["W"], a["target"], a["lse"], a["dloss"], a["dX"], a["dW"],
                                          a["ws"], a["n"], a["M"], a["V"], a["K"], None)


@pytest.mark.parametrize("kw,expect", [
    ({"X": 0}, 1), ({"target": 0}, 1), ({"lse": 0}, 1), ({"dloss": 0}, 1), ({"ws": 0}, 1), ({"dX": 0, "dW": 0}, 1),
    ({"M": 0}, 2), ({"K": -8}, 2), ({"n": 16}, 2),
    ({"K": 12}, 3), ({"dX": 6 * P + 8}, 3), ({"dW": 7 * P + 8}, 3), ({"dloss": 5 * P + 2}, 3), ({"lse": 4 * P + 3}, 3),
    ({"dX": P + 16}, 4), ({"dW": 6 * P + 16}, 4), ({"ws": 7 * P + 16}, 4), ({"dX": 5 * P - 16}, 4),
    ({"dX": 0, "ws": 7 * P}, 4),
])
def test_xent_backward_rejects_bad_arguments(lib, kw, expect):  # noqa: F811
    assert xent_backward(lib, **kw) == expect


def route(lib, **kw):
    a = dict(l=P, v=2 * P, w=3 * P, e=4 * P, s=5 * P, c=6 * P, p=7 * P, o=8 * P, ws=9 * P, n=BIG, M=1000, E=60, ld=60, k=4)
    a.update(kw)
    return lib.router_topk(a["l"], a["v"], a["w"], a["e"], a["s"], a["c"], a["p"], a["o"], a["ws"], a["n"],
                           a["M"], a["E"], a["ld"], a["k"], 1, None)


@pytest.mark.parametrize("kw,expect", [
    ({"l": 0}, 1), ({"w": 0}, 1), ({"e": 0}, 1), ({"s": 0}, 1), ({"c": 0}, 1), ({"p": 0}, 1), ({"o": 0}, 1), ({"ws": 0}, 1),
    ({"M": 0}, 2), ({"E": 0}, 2), ({"E": 1025, "ld": 1025}, 2), ({"ld": 59}, 2), ({"k": 0}, 2), ({"k": 33}, 2),
    ({"E": 3, "k": 4}, 2), ({"n": 16}, 2), ({"M": 0x7FFFFFFF}, 2),
    ({"l": P + 2}, 3), ({"w": 3 * P + 1}, 3), ({"ws": 9 * P + 4}, 3), ({"o": 8 * P + 2}, 3),
    ({"w": P + 400}, 4), ({"e": 3 * P + 64}, 4), ({"s": 2 * P}, 4), ({"c": 5 * P}, 4), ({"ws": 7 * P}, 4),
])
def test_router_topk_rejects_bad_arguments(lib, kw, expect):  # noqa: F811
    assert route(lib, **kw) == expect


def route_backward(lib, **kw):
    a = dict(l=P, e=2 * P, s=3 * P, c=4 * P, dw=5 * P, dl=6 * P, out=7 * P, bf16=0, M=1000, E=60, ld=60, k=4)
    a.update(kw)
    return lib.router_topk_backward(a["l"], a["e"], a["s"], a["c"], a["dw"], a["dl"], a["out"], a["bf16"],
                                    a["M"], a["E"], a["ld"], a["k"], 0, None)


@pytest.mark.parametrize("kw,expect", [
    ({"l": 0}, 1), ({"e": 0}, 1), ({"s": 0}, 1), ({"c": 0}, 1), ({"out": 0}, 1),
    ({"M": -1}, 2), ({"E": 2000, "ld": 2000}, 2), ({"ld": 1}, 2), ({"k": 61}, 2),
    ({"out": 7 * P + 2}, 3), ({"bf16": 1, "out": 7 * P + 1}, 3), ({"dw": 5 * P + 2}, 3), ({"dl": 6 * P + 1}, 3),
    ({"out": P}, 4), ({"out": 5 * P}, 4), ({"out": 6 * P}, 4),
])
def test_router_topk_backward_rejects_bad_arguments(lib, kw, expect):  # noqa: F811
    assert route_backward(lib, **kw) == expect


def test_workspace_sizes(lib):  # noqa: F811
    assert lib.gemm_bf16_nt_xent_workspace_bytes(0, 8) == 0
    assert lib.gemm_bf16_nt_xent_workspace_bytes(40, 200) > 0
    assert lib.gemm_bf16_nt_xent_backward_workspace_bytes(40, 0, 8) == 0
    # bounded by the pieces, not by the logits: 64 Ki x 128 Ki logits would be 16 GiB in BF16
    big = lib.gemm_bf16_nt_xent_backward_workspace_bytes(65536, 131072, 4096)
    assert 0 < big < 4 << 30
    assert lib.router_topk_workspace_bytes(1, 256) == 0      # one block needs none
    assert lib.router_topk_workspace_bytes(100, 2000) == 0   # invalid
    assert lib.router_topk_workspace_bytes(1 << 20, 256) <= 1 << 20
