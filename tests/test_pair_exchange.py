"""The exchange between two epilogue warps of few tokens' gated tiles (csrc/pair_exchange.cuh):
every interleaving of two warps of two lanes, with an mbarrier's parity waits."""
from __future__ import annotations

import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_block_scaled_tcgen05_gb300", "csrc")
EXCHANGES, LANES = 5, 2
WRITE, SYNC, ARRIVE, WAIT, VOTE, READ, DONE = range(7)


class Protocol:
    def __init__(self, arrivals, arrive_at, wait_at, parity, half):
        self.arrivals, self.arrive_at, self.wait_at, self.parity, self.half = arrivals, arrive_at, wait_at, parity, half


def explore(p, first):
    """States reachable by warps `first` and first + 2; raises at a wrong read, returns the number
    of states, or None where one has no way on."""
    warps = (first, first ^ 2)
    bars = sorted({f(e) for e in warps for f in (p.arrive_at, p.wait_at)})
    at = {b: i for i, b in enumerate(bars)}
    # per warp: (n, each lane's step); per barrier: (arrivals still due, parity of its phase);
    # per warp: what each lane wrote last in each half
    start = (tuple((0, (WRITE,) * LANES) for _ in warps), ((p.arrivals, 0),) * len(bars), (((-1,) * LANES,) * 2,) * 2)
    todo, seen, stuck = [start], {start}, False
    while todo:
        lanes, phases, boxes = todo.pop()
        after = []

        def go(w, n, steps, phases=phases, boxes=boxes):
            if all(s == DONE for s in steps) and n + 1 < EXCHANGES:
                n, steps = n + 1, (WRITE,) * LANES
            after.append((tuple((n, tuple(steps)) if i == w else lanes[i] for i in range(2)), phases, boxes))

        for w in range(2):
            n, steps = lanes[w]
            # steps that the whole warp takes
            for step, then in ((SYNC, ARRIVE), (VOTE, READ)):
                if all(s == step for s in steps):
                    go(w, n, (then,) * LANES)
            for k, s in enumerate(steps):
                def to(then):
                    return tuple(then if i == k else x for i, x in enumerate(steps))
                if s == WRITE:
                    halves = list(boxes[w])
                    h = p.half(n)
                    halves[h] = tuple(n if i == k else x for i, x in enumerate(halves[h]))
                    go(w, n, to(SYNC), boxes=tuple(tuple(halves) if i == w else boxes[i] for i in range(2)))
                elif s == ARRIVE and k == 0:
                    b = at[p.arrive_at(warps[w])]
                    due, phase = phases[b]
                    new = (due - 1, phase) if due > 1 else (p.arrivals, phase ^ 1)
                    go(w, n, to(WAIT), phases=tuple(new if i == b else x for i, x in enumerate(phases)))
                elif s == ARRIVE:
                    go(w, n, to(WAIT))
                elif s == WAIT:
                    # a wait for parity x ends while the current phase has the other parity
                    if phases[at[p.wait_at(warps[w])]][1] != p.parity(n):
                        go(w, n, to(VOTE))
                elif s == READ:
                    got = boxes[1 - w][p.half(n)][k]
                    assert got == n, f"warp {warps[w]} read exchange {got} instead of {n}"
                    go(w, n, to(DONE))
        if not after and any(s != DONE for _, steps in lanes for s in steps):
            stuck = True
        for x in after:
            if x not in seen:
                seen.add(x)
                todo.append(x)
    return None if stuck else len(seen)


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """The protocol that the kernel uses, from its header."""
    d = tmp_path_factory.mktemp("pair_exchange")
    src, exe = d / "p.cpp", d / "p"
    src.write_text('#include <cstdio>\n#include "pair_exchange.cuh"\nusing P = gb300::PairExchange;\n'
                   'int main() {\n  std::printf("%d", P::kArrivals);\n  for (int e = 0; e < 4; ++e) std::printf(" %d", P::bar(e));\n'
                   f'  for (unsigned n = 0; n < {EXCHANGES}; ++n) std::printf(" %u %u", P::parity(n), P::half(n));\n}}\n')
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-x", "c++", str(src), "-o", str(exe)], check=True)
    v = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    bar, rest = v[1:5], v[5:]
    return Protocol(v[0], bar.__getitem__, bar.__getitem__, rest[::2].__getitem__, rest[1::2].__getitem__)


def test_every_interleaving_ends_and_reads_its_own_exchange(kernels):
    for first in (0, 1):
        assert explore(kernels, first) > 100
    assert kernels.wait_at(0) != kernels.wait_at(1), "the pairs' barriers"


def test_the_model_finds_planted_mistakes():
    low = lambda n: n & 1
    # a barrier of each warp's own, at which the other arrives: it can run ahead of a waiting lane
    assert explore(Protocol(1, lambda e: e ^ 2, lambda e: e, low, low), 0) is None
    # one arrival to the shared barrier: a wait ends before the other warp has written
    with pytest.raises(AssertionError, match="read exchange"):
        assert explore(Protocol(1, lambda e: e & 1, lambda e: e & 1, low, low), 0) is not None
    # one half for all exchanges: written again before the other has read it
    with pytest.raises(AssertionError, match="read exchange"):
        explore(Protocol(2, lambda e: e & 1, lambda e: e & 1, low, lambda n: 0), 0)
