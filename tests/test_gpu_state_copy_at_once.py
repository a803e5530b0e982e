"""state_copy called at once from several host threads, and captured, with very different numbers
of entries: each call needs another amount of shared memory of one kernel."""
import sys
import threading

import pytest
import torch

from kimi_delta_attention_17_gb300 import _lib, build, state_copy

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def entries(n):
    """A rotation of n slots."""
    i = torch.arange(n, dtype=torch.int32, device="cuda")
    return torch.roll(i, 1), i


@pytest.mark.parametrize("sizes", [(1, 1024), (1025, 4096), (1, 1, 1024, 700, 4096, 1025)])
def test_host_threads(sizes):
    """The C entry in tight loops: threads meet between a kernel's limit and its launch."""
    calls, copy = 10000, _lib.lib().kda_state_copy
    pools = [torch.arange(n, dtype=torch.int64, device="cuda").repeat_interleave(2).view(n, 2) for n in sizes]
    lists = [entries(n) for n in sizes]
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    refused, start, interval = [], threading.Barrier(len(sizes)), sys.getswitchinterval()

    def work(pool, src, dst, stream):
        n = src.shape[0]
        args = (None, 0, pool.data_ptr(), n, src.data_ptr(), dst.data_ptr(), n, 1, 16, stream.cuda_stream)
        start.wait(60)
        for _ in range(calls):
            status = copy(*args)
            if status:
                refused.append((n, status))

    threads = [threading.Thread(target=work, args=(p, *l, s)) for p, l, s in zip(pools, lists, streams)]
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    assert not refused, "%d calls refused, first %r" % (len(refused), refused[0])
    for n, pool in zip(sizes, pools):
        want = (torch.arange(n, device="cuda") - calls) % n
        assert torch.equal(pool[:, 0], want) and torch.equal(pool[:, 1], want)


def test_one_capture_of_several_sizes():
    sizes = (1024, 1, 300, 4096, 1025)
    pools = [torch.arange(2 * n, dtype=torch.int64, device="cuda").view(n, 2) for n in sizes]
    lists = [entries(n) for n in sizes]
    want = [torch.roll(p, 1, 0) for p in pools]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for p, (src, dst) in zip(pools, lists):
            state_copy(p, src, dst)
    state_copy(torch.zeros(2, 2, dtype=torch.int64, device="cuda"), *entries(2))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, w) for p, w in zip(pools, want))
