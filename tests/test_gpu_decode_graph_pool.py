"""A graph of decode steps over a pool of states: what it costs to build, and what it keeps."""
import gc
import weakref

import pytest
import torch

from kimi_delta_attention_17_gb300 import DecodeGraph, build, decode_step
from tests.test_gpu_state_pool import decode_inputs, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def inputs(N, H, d, steps):
    per = [decode_inputs(N, H, d, torch.bfloat16, {}, seed=s) for s in range(steps)]
    return [torch.stack([p[i] for p in per]) for i in range(5)]


def test_building_makes_no_copy_of_the_pool():
    N, H, d, P = 2, 4, 128, 4096
    stacked, slots = inputs(N, H, d, 2), i32([P - 1, 3])
    pool = torch.zeros(P, H, d, d, device="cuda")                 # 1 GiB
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    graph = DecodeGraph(*stacked, d ** -0.5, pool, slots=slots)
    assert torch.cuda.max_memory_allocated() - before < pool.numel() * 4 // 8
    assert not pool.any() and slots.tolist() == [P - 1, 3]        # no step has run
    graph.replay()
    torch.cuda.synchronize()
    assert pool[3].any() and pool[P - 1].any() and not pool[4:P - 1].any()


def test_keeps_what_its_steps_read():
    """Tensors that the caller lets go stay alive with the graph."""
    N, H, d, P = 2, 2, 64, 5
    stacked, slots = inputs(N, H, d, 2), i32([4, 1])
    pool = torch.zeros(P, H, d, d, device="cuda")
    want = pool.clone()
    outs = [decode_step(*[t[s] for t in stacked], d ** -0.5, want, slots=slots) for s in range(2)]
    graph = DecodeGraph(*stacked, d ** -0.5, pool, slots=slots)
    alive = [weakref.ref(t) for t in stacked + [slots]]
    del stacked, slots
    gc.collect()
    assert all(r() is not None for r in alive)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(pool, want) and torch.equal(graph.out, torch.stack(outs))
    del graph
    gc.collect()
    assert all(r() is None for r in alive)
