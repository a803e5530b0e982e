"""The pool of recurrent states: copies, compaction, and the steps that address
it by slot, alone and as a serving loop runs them."""
import random

import numpy as np
import pytest
import torch

from kimi_delta_attention_17_gb300 import (DecodeGraph, build, chunk_fwd, decode_step, gated_scan_fwd,
                                           gated_scan_step, state_compact, state_copy)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def pool_of(L, P, floats, seed=0):
    return torch.randn(L, P, floats, generator=torch.Generator().manual_seed(seed))


def assigned(pool, src, dst, source=None):
    """The assignment entry by entry, on the values before it."""
    before = pool if source is None else source
    after = pool.clone()
    for s, d in zip(src, dst):
        if 0 <= d < pool.shape[1] and s < before.shape[1]:
            after[:, d] = before[:, s] if s >= 0 else 0.0
    return after


def check_copy(pool, src, dst, source=None):
    dev = pool.cuda()
    kept = None if source is None else source.cuda()
    got = state_copy(dev, i32(src), i32(dst), source=kept, slot_dim=1)
    assert got is dev
    assert torch.equal(dev.cpu(), assigned(pool, src, dst, source))
    if source is not None:
        assert torch.equal(kept.cpu(), source)


@pytest.mark.parametrize("floats", [4, 12, 260, 4096, 20000])
@pytest.mark.parametrize("src,dst", [
    ([], []), ([3], [3]), ([1], [0]), ([0, 1], [1, 0]),                     # nothing, itself, a move, a swap
    ([1, 2, 3, 0], [0, 1, 2, 3]), ([0, 1, 2, 3, 4], [1, 2, 3, 4, 5]),        # a cycle, a shift
    ([5, 5, 5, 5], [0, 1, 2, 5]), ([2, 0, 0], [0, 1, 2]),                    # a fork, one through a moved slot
    ([-1, 4, -1], [4, 5, 0]), ([-1, -1, -1], [0, 1, 2]),                     # clears, one of a source
    ([0, 1, 2], [3, 3, 3]), ([0, 4, -1], [4, 4, 4]), ([1, 3], [3, 3]),       # the last of one destination holds
    ([0, 1, 2], [-1, 6, 5]), ([6, 2, 7, 1], [0, 1, 2, 3]), ([0, 0], [2 ** 31 - 1, -2 ** 31])])
def test_copy_within_a_pool(src, dst, floats):
    check_copy(pool_of(2, 6, floats), src, dst)


@pytest.mark.parametrize("seed", range(6))
def test_copy_random(seed):
    rng = random.Random(seed)
    P, L, floats = rng.choice([7, 64, 300]), rng.randint(1, 3), 4 * rng.choice([1, 3, 33, 512])
    n = rng.choice([1, P // 2, 2 * P])
    src = [rng.randrange(-2, P + 2) for _ in range(n)]
    dst = [rng.randrange(-2, P + 2) for _ in range(n)]
    check_copy(pool_of(L, P, floats, seed), src, dst)


@pytest.mark.parametrize("n", [1024, 1025, 4096])
def test_copy_many_entries(n):
    rng = random.Random(n)
    perm = list(range(5000))
    rng.shuffle(perm)
    check_copy(pool_of(1, 5000, 20), perm[:n], sorted(perm[:n]))


def test_copy_from_another_pool():
    pool, source = pool_of(3, 9, 40), pool_of(3, 4, 40, seed=1)
    check_copy(pool, [0, 3, 3, -1, 4, 1], [8, 0, 1, 2, 3, -1], source)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int64, torch.uint8])
def test_copy_any_type_and_flat_pool(dtype):
    pool = (torch.arange(5 * 48).reshape(5, 3, 16) % 251).to(dtype)
    dev = pool.cuda()
    state_copy(dev, i32([4, 0]), i32([0, 2]))
    want = pool.clone()
    want[0], want[2] = pool[4], pool[0]
    assert torch.equal(dev.cpu(), want)
    same = pool.cuda()
    state_copy(same, i32([4, 0]), i32([0, 2]), source=same)
    assert torch.equal(same.cpu(), want)


def compacted(pool, live):
    after, n = pool.clone(), int(sum(live))
    to = [i if alive else -1 for i, alive in enumerate(live)]
    holes = iter([i for i in range(n) if not live[i]])
    for i in range(n, len(live)):
        if live[i]:
            to[i] = next(holes)
            after[:, to[i]] = pool[:, i]
    return after, to, n


@pytest.mark.parametrize("P,share", [(1, 0.0), (1, 1.0), (2, 0.5), (33, 0.0), (33, 1.0), (40, 0.3), (1024, 0.6),
                                     (1025, 0.5), (4096, 0.5), (4096, 0.9), (4097, 0.5), (5000, 0.2)])
@pytest.mark.parametrize("L,floats", [(1, 4), (2, 516)])
def test_compact(P, share, L, floats):
    rng = random.Random(P)
    pool = pool_of(L, P, floats)
    live = [rng.random() < share for _ in range(P)]
    want, to, n = compacted(pool, live)
    for kind in (torch.bool, torch.uint8):
        dev, mask = pool.cuda(), torch.tensor(live).to(kind).cuda()
        if kind == torch.uint8:
            mask *= 7  # any value but zero
        new_slot, count = state_compact(dev, mask, slot_dim=1)
        assert torch.equal(dev.cpu(), want) and new_slot.tolist() == to and count.tolist() == [n]


def test_compact_large_slots_and_given_outputs():
    pool = pool_of(1, 7, 40000)
    live = [False, True, False, True, False, True, True]
    want, to, n = compacted(pool, live)
    dev = pool.cuda()
    new_slot, count = torch.empty(7, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    got = state_compact(dev[0], torch.tensor(live).cuda(), new_slot=new_slot, count=count)
    assert got[0] is new_slot and got[1] is count
    assert torch.equal(dev.cpu(), want) and new_slot.tolist() == to and count.tolist() == [n]


DECODE = [dict(), dict(gate="logsigmoid", l2norm_qk=True), dict(gate="bounded"), dict(decay="scalar"),
          dict(decay="none", l2norm_qk=True)]


def decode_inputs(N, H, d, dtype, options, seed=0):
    gen = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(N, H, d, generator=gen) for _ in range(3))
    q, k = (torch.nn.functional.normalize(t, dim=-1) for t in (q, k))
    decay = options.get("decay", "channel")
    g = None if decay == "none" else -torch.rand((N, H, d) if decay == "channel" else (N, H), generator=gen)
    return [t if t is None else t.cuda() for t in (q.to(dtype), k.to(dtype), v.to(dtype), g,
                                                   torch.rand(N, H, generator=gen))]


@pytest.mark.parametrize("options", DECODE)
@pytest.mark.parametrize("H,d,dtype", [(3, 64, torch.bfloat16), (2, 128, torch.bfloat16), (1, 64, torch.float32),
                                       (5, 128, torch.float32)])
def test_decode_by_slot_equals_dense_decode(H, d, dtype, options):
    """Bit for bit, on the gathered states; padding rows give zeros, other slots stay."""
    P, slots = 9, [7, -1, 0, 3, P_OUT, 8]
    args = decode_inputs(len(slots), H, d, dtype, options)
    pool0 = torch.randn(P, H, d, d, generator=torch.Generator().manual_seed(1)).cuda() * 0.1
    pool = pool0.clone()
    out = decode_step(*args, d ** -0.5, pool, slots=i32(slots), **options)
    rows = [n for n, s in enumerate(slots) if 0 <= s < P]
    at = [slots[n] for n in rows]
    state = pool0[at].clone()
    dense = decode_step(*[t if t is None else t[rows].contiguous() for t in args], d ** -0.5, state, **options)
    want = pool0.clone()
    want[at] = state
    assert torch.equal(out[rows], dense) and torch.equal(pool, want)
    assert (out[[n for n in range(len(slots)) if n not in rows]] == 0).all()


P_OUT = 9


def test_decode_more_rows_than_a_grid_dimension():
    N, d = 66001, 64
    args = [t if t is None else t.cuda() for t in decode_inputs(N, 1, d, torch.bfloat16, {})]
    pool = torch.randn(N, 1, d, d, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) * 0.1
    slots = torch.randperm(N, device="cuda").int()
    state = pool[slots.long()]
    dense = decode_step(*args, d ** -0.5, state)
    out = decode_step(*args, d ** -0.5, pool, slots=slots)
    assert torch.equal(out, dense) and torch.equal(pool[slots.long()], state)


def test_decode_graph_over_slots():
    """A graph of steps whose slots are refilled between replays."""
    N, H, d, P, steps = 3, 2, 64, 8, 4
    per = [decode_inputs(N, H, d, torch.bfloat16, {}, seed=s) for s in range(steps)]
    stacked = [torch.stack([p[i] for p in per]) for i in range(5)]
    pool = torch.randn(P, H, d, d, generator=torch.Generator().manual_seed(1)).cuda() * 0.1
    ref, slots = pool.clone(), i32([0, 1, 2])
    graph = DecodeGraph(*stacked, d ** -0.5, pool, slots=slots)
    assert torch.equal(pool, ref)
    for chosen in ([0, 1, 2], [5, 2, 7], [3, -1, 0]):
        slots.copy_(i32(chosen))
        graph.replay()
        outs = [decode_step(*p, d ** -0.5, ref, slots=i32(chosen)) for p in per]
        torch.cuda.synchronize()
        assert torch.equal(graph.out, torch.stack(outs)) and torch.equal(pool, ref)


def test_captured_maintenance():
    """Copies and compactions replayed on other entries; two graphs, replayed in turn, keep apart."""
    pool = pool_of(2, 16, 64).cuda()
    src, dst, live = i32([-1] * 6), i32([-1] * 6), torch.ones(16, dtype=torch.bool, device="cuda")
    state_copy(pool, src, dst, slot_dim=1)
    state_compact(pool, live, slot_dim=1)
    torch.cuda.synchronize()
    copy, compact, compact2 = (torch.cuda.CUDAGraph() for _ in range(3))
    with torch.cuda.graph(copy):
        state_copy(pool, src, dst, slot_dim=1)
    with torch.cuda.graph(compact):
        new_slot, count = state_compact(pool, live, slot_dim=1)
    with torch.cuda.graph(compact2):
        new_slot2, count2 = state_compact(pool, live, slot_dim=1)
    want = pool.cpu()
    rng = random.Random(2)
    for _ in range(3):
        s, d = ([rng.randrange(-1, 16) for _ in range(6)] for _ in range(2))
        src.copy_(i32(s))
        dst.copy_(i32(d))
        copy.replay()
        want = assigned(want, s, d)
        for graph, to, n in ((compact, new_slot, count), (compact2, new_slot2, count2)):
            alive = [rng.random() < 0.5 for _ in range(16)]
            live.copy_(torch.tensor(alive))
            graph.replay()
            want, map_, total = compacted(want, alive)
            torch.cuda.synchronize()
            assert torch.equal(pool.cpu(), want) and to.tolist() == map_ and n.item() == total


def test_offsets_past_32_bits():
    """Pools of more than 2^31 values: slots at both ends."""
    P, D = 600000, 4096
    pool = torch.zeros(P, D, device="cuda")
    pool[P - 1], pool[P - 2] = 3.0, 4.0
    state_copy(pool, i32([P - 1, P - 2, -1]), i32([0, P - 1, P - 2]))
    assert (pool[0] == 3).all() and (pool[P - 1] == 4).all() and (pool[P - 2] == 0).all()
    x = torch.ones(2, D, device="cuda")
    out = gated_scan_step(x, torch.zeros_like(x), pool, slots=i32([P - 1, 1]))
    assert (out[0] == 5).all() and (pool[P - 1] == 5).all() and (out[1] == 1).all() and (pool[1] == 1).all()
    live = torch.zeros(P, dtype=torch.bool, device="cuda")
    live[[0, P - 1]] = True
    new_slot, count = state_compact(pool, live)
    assert count.item() == 2 and new_slot[P - 1].item() == 1 and (pool[1] == 5).all() and (pool[0] == 3).all()
    del pool, x, out
    P, H, d = 33000, 16, 64
    pool = torch.zeros(P, H, d, d, device="cuda")
    pool[P - 1] = torch.randn(H, d, d, generator=torch.Generator().manual_seed(2)).cuda()
    state = pool[P - 1:].clone()
    args = decode_inputs(1, H, d, torch.bfloat16, {})
    out = decode_step(*args, 0.125, pool, slots=i32([P - 1]))
    dense = decode_step(*args, 0.125, state)
    assert torch.equal(out, dense) and torch.equal(pool[P - 1:], state) and not pool[:P - 1].any()


def test_on_another_stream():
    pool = pool_of(1, 64, 40000)
    dev, side = pool.cuda(), torch.cuda.Stream()
    perm = list(range(64))
    random.Random(1).shuffle(perm)
    torch.cuda.synchronize()
    src, dst, mask = i32(perm), i32(list(range(64))), torch.tensor([i % 3 > 0 for i in range(64)]).cuda()
    torch.cuda.synchronize()
    state_copy(dev, src, dst, slot_dim=1, stream=side)
    new_slot, count = state_compact(dev, mask, slot_dim=1, stream=side)
    side.synchronize()
    want, to, n = compacted(assigned(pool, perm, range(64)), mask.tolist())
    assert torch.equal(dev.cpu(), want) and new_slot.tolist() == to and count.item() == n


def test_a_serving_loop():
    """Two layers, one of matrix and one of vector states: prompts are prefilled and admitted, a
    request is forked, rows step by slot with padding, one ends, the pool is compacted, and the
    rest goes on densely. Every live request equals its own run without a pool, bit for bit."""
    H, d, D, P, T = 2, 64, 40, 8, 70
    gen = torch.Generator().manual_seed(8)

    def tokens(n, T):
        q, k = (torch.nn.functional.normalize(torch.randn(n, T, H, d, generator=gen), dim=-1).bfloat16().cuda() for _ in range(2))
        return dict(q=q, k=k, v=torch.randn(n, T, H, d, generator=gen).bfloat16().cuda(),
                    g=-torch.rand(n, T, H, d, generator=gen).cuda(), beta=torch.rand(n, T, H, generator=gen).cuda(),
                    x=torch.randn(n, T, D, generator=gen).bfloat16().cuda(),
                    z=torch.randn(n, T, D, generator=gen).bfloat16().cuda())

    how = dict(gate="logsigmoid", write="norm")
    t = tokens(3, T)
    _, matrix = chunk_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], d ** -0.5)
    _, vector, _ = gated_scan_fwd(t["x"], t["z"], **how)
    pool_m = torch.full((P, H, d, d), 9.0, device="cuda")
    pool_v = torch.full((P, D), 9.0, device="cuda")
    where = [6, 1, 4]                                       # the requests' slots
    for pool, states in ((pool_m, matrix), (pool_v, vector)):
        state_copy(pool, i32([0, 1, 2, -1]), i32(where + [0]), source=states)
        state_copy(pool, i32([6]), i32([3]))                # request 0 forked into slot 3
    where = where + [3, 0]                                  # the fork, and a request without a prompt
    own_m = [matrix[i:i + 1].clone() for i in (0, 1, 2, 0)] + [torch.zeros(1, H, d, d, device="cuda")]
    own_v = [vector[i:i + 1].clone() for i in (0, 1, 2, 0)] + [torch.zeros(1, D, device="cuda")]

    def step(rows, slots, dense=None):
        s = tokens(len(slots), 1)
        s = {k: v[:, 0].contiguous() for k, v in s.items()}
        if dense is None:
            o = decode_step(s["q"], s["k"], s["v"], s["g"], s["beta"], d ** -0.5, pool_m, slots=i32(slots))
            y = gated_scan_step(s["x"], s["z"], pool_v, slots=i32(slots), **how)
        else:
            o = decode_step(s["q"], s["k"], s["v"], s["g"], s["beta"], d ** -0.5, pool_m[:dense])
            y = gated_scan_step(s["x"], s["z"], pool_v[:dense], **how)
        for row, r in rows:
            one = {k: v[row:row + 1] for k, v in s.items()}
            assert torch.equal(o[row:row + 1], decode_step(one["q"], one["k"], one["v"], one["g"], one["beta"], d ** -0.5, own_m[r]))
            assert torch.equal(y[row:row + 1], gated_scan_step(one["x"], one["z"], own_v[r], **how))

    for _ in range(3):
        step([(0, 0), (1, 1), (2, 2), (4, 3), (5, 4)], [where[0], where[1], where[2], -1, where[3], where[4]])
    live = torch.zeros(P, dtype=torch.bool, device="cuda")
    live[[where[r] for r in (0, 2, 3, 4)]] = True           # request 1 ended
    maps = [state_compact(pool, live) for pool in (pool_m, pool_v)]
    assert torch.equal(maps[0][0], maps[1][0]) and maps[0][1].item() == 4
    to = maps[0][0].tolist()
    rows = [(to[where[r]], r) for r in (0, 2, 3, 4)]
    assert sorted(row for row, _ in rows) == [0, 1, 2, 3]
    for _ in range(2):
        step(rows, [0] * 4, dense=4)
    for row, r in rows:
        assert torch.equal(pool_m[row], own_m[r][0]) and torch.equal(pool_v[row], own_v[r][0])


def test_refusals():
    pool = torch.zeros(2, 6, 8, device="cuda")
    a, b = i32([0, 1]), i32([2, 3])
    for bad in (dict(src=a.long()), dict(dst=b[:1]), dict(src=a.cpu()), dict(slot_dim=2), dict(pool=pool.transpose(0, 1)),
                dict(pool=pool[0, 0]), dict(source=pool.bfloat16()), dict(source=pool[:1]), dict(source=pool[..., :4]),
                dict(source=torch.zeros(2, 3, 8)), dict(pool=pool[:, :0]), dict(src=None)):
        with pytest.raises((ValueError, TypeError)):
            state_copy(**{**dict(pool=pool, src=a, dst=b, slot_dim=1), **bad})
    with pytest.raises(RuntimeError, match="INVALID"):
        state_copy(pool[..., :3].contiguous(), a, b, slot_dim=1)      # slots of 12 bytes
    with pytest.raises(RuntimeError, match="INVALID"):
        state_copy(pool[0], a, b, source=pool[0][2:])                  # overlaps the pool
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        state_copy(pool[0], i32([0] * 4097), i32([0] * 4097))
    live = torch.ones(6, dtype=torch.bool, device="cuda")
    for bad in (dict(live=live[:5]), dict(live=live.int()), dict(live=live.cpu()), dict(new_slot=i32([0])),
                dict(count=torch.zeros(1, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            state_compact(**{**dict(pool=pool, live=live, slot_dim=1), **bad})
    args = decode_inputs(2, 3, 64, torch.bfloat16, {})
    state = torch.zeros(4, 3, 64, 64, device="cuda")
    for bad in (dict(slots=i32([0])), dict(slots=i32([0, 1]).long()), dict(state=state[:, :2].contiguous()),
                dict(state=state.bfloat16()), dict(out=args[0][:1])):
        with pytest.raises((ValueError, TypeError)):
            decode_step(*args, 0.1, **{**dict(state=state, slots=i32([0, 1])), **bad})


def test_padding_only():
    """A pool whose every entry is padding is left as it was, whatever it holds."""
    pool = torch.full((1, 4, 8), float("nan"))
    dev = pool.cuda()
    state_copy(dev, i32([0, 1]), i32([-1, -1]), slot_dim=1)
    assert np.array_equal(dev.cpu().numpy(), pool.numpy(), equal_nan=True)
