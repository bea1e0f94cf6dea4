"""The routing step called by host threads at the same time with numbers of
experts that need different amounts of shared memory of one kernel: no call is
refused, and every result is that of the call made alone."""
from __future__ import annotations

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_tcgen05_gb300 as lib
    yield lib
    assert lib.gemm_get_device_status() == 0


# forward: 257..512 and 513..1024 experts are one kernel each; backward: 513..1024
@pytest.mark.parametrize("experts", [(300, 512), (700, 1024)])
def test_two_numbers_of_experts_at_once(g, experts):
    M, k, calls = 20, 4, 20000
    lib = g.load()
    gen = torch.Generator(device="cuda").manual_seed(experts[0])
    work = []                 # two threads per number of experts
    for E in experts * 2:
        l = torch.randn(M, E, generator=gen, device="cuda")
        dw = torch.randn(M, k, generator=gen, device="cuda")
        r = g.router_topk(l, k)
        d = g.router_topk_backward(l, r.experts, r.lse, r.counts, dweights=dw)
        out, dl = [torch.empty_like(t) for t in r], torch.empty_like(d)
        work.append((E, l, dw, r, d, out, dl, torch.cuda.Stream()))
    torch.cuda.synchronize()
    refused = [0] * len(work)
    start = threading.Barrier(len(work))

    def loop(i):
        # the C entry points themselves: the interpreter's lock is free while
        # one runs, and little time passes between two
        E, l, dw, r, _, out, dl, s = work[i]
        ptrs = [t.data_ptr() for t in out]
        forward = (l.data_ptr(), None, *ptrs, None, 0, M, E, E, k, 0, s.cuda_stream)
        backward = (l.data_ptr(), r.experts.data_ptr(), r.lse.data_ptr(), r.counts.data_ptr(),
                    dw.data_ptr(), None, dl.data_ptr(), 0, M, E, E, k, 0, s.cuda_stream)
        start.wait()
        for _ in range(calls):
            refused[i] += lib.router_topk(*forward) != 0
            refused[i] += lib.router_topk_backward(*backward) != 0
        s.synchronize()

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(work))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert refused == [0] * len(work)
    for _, _, _, r, d, out, dl, _ in work:
        assert all(torch.equal(a, b) for a, b in zip(out, r)) and torch.equal(dl, d)
