"""States in 8 bits: every code, scale and value bit for bit against the definition in fp32 on the CPU."""
import random

import pytest
import torch

from kimi_delta_attention_17_gb300 import build, state_copy, state_dequantize, state_quantize

pytestmark = pytest.mark.gpu

KINDS = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def coded(x, kind, block):
    """(codes as bytes, scales) of x [..., values], on the CPU."""
    top = torch.tensor(KINDS[kind])
    y = x.reshape(*x.shape[:-1], -1, block)
    most = y.abs().amax(-1, keepdim=True)
    some = most >= 2.0 ** -100
    codes = y * torch.where(some, top / most, torch.zeros(()))
    codes = (codes.round() if kind == torch.int8 else codes).to(kind).view(torch.uint8).reshape(x.shape)
    return codes, torch.where(some, most * torch.tensor(1.0 / KINDS[kind]), torch.zeros(())).squeeze(-1)


def values(codes, scales, kind, block):
    y = codes.view(kind).float().reshape(*codes.shape[:-1], -1, block)
    return (y * scales[..., None]).reshape(codes.shape)


def holders(src, dst, src_slots, dst_slots):
    """{destination: source} of the entries that hold."""
    return {d: s for s, d in zip(src, dst) if 0 <= d < dst_slots and s < src_slots}


def check(L, P, S, V, block, kind, src, dst, seed=0):
    gen = torch.Generator().manual_seed(seed)
    pool = torch.randn(L, P, V, generator=gen) * torch.exp(2 * torch.randn(L, P, 1, generator=gen))
    store = torch.randint(0, 120, (L, S, V), generator=gen).to(torch.uint8)
    scales = torch.rand(L, S, V // block, generator=gen)
    want, want_s = store.clone(), scales.clone()
    for d, s in holders(src, dst, P, S).items():
        want[:, d], want_s[:, d] = coded(pool[:, s] if s >= 0 else torch.zeros(L, V), kind, block)
    dev, devs, devp = store.cuda().view(kind), scales.cuda(), pool.cuda()
    got, gots = state_quantize(devp, i32(src), dev, devs, i32(dst), slot_dim=1)
    assert got is dev and gots is devs and torch.equal(devp.cpu(), pool)
    assert torch.equal(dev.view(torch.uint8).cpu(), want) and torch.equal(devs.cpu(), want_s)
    # And back, by the inverse lists: what the store holds in dst into the pool's src.
    after = pool.clone()
    for d, s in holders(dst, src, S, P).items():
        after[:, d] = values(want[:, s], want_s[:, s], kind, block) if s >= 0 else 0.0
    assert state_dequantize(dev, devs, i32(dst), devp, i32(src), slot_dim=1) is devp
    assert torch.equal(devp.cpu(), after)
    assert torch.equal(dev.view(torch.uint8).cpu(), want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("blocks", [1, 3, 31, 128, 321])
def test_codes_and_values(blocks, block, kind):
    check(2, 5, 7, blocks * block, block, kind, [4, 0, -1, 2], [6, 1, 2, 0])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("src,dst", [([], []), ([1], [3]), ([1, 1, 1], [0, 1, 2]), ([0, 1, 2], [4, 4, 4]),
                                     ([0, -1, 9], [4, 4, 4]), ([-1, 3], [4, 4]), ([3, -1], [4, 4]),
                                     ([0, 1, 2], [-1, 5, 1]), ([5, 2, 2 ** 31 - 1], [0, 0, 1]),
                                     ([0, 1], [2 ** 31 - 1, -2 ** 31]), ([-2, -2 ** 31], [0, 3])])
def test_lists(src, dst, kind):
    check(2, 5, 5, 384, 64, kind, src, dst)


@pytest.mark.parametrize("seed", range(4))
def test_random_lists(seed):
    rng = random.Random(seed)
    P, S, n = rng.randint(1, 300), rng.randint(1, 300), rng.choice([1, 300, 4096])
    src, dst = ([rng.randrange(-2, m + 2) for _ in range(n)] for m in (P, S))
    check(rng.randint(1, 3), P, S, 128 * rng.choice([1, 3, 40]), 128, rng.choice(list(KINDS)), src, dst, seed)


@pytest.mark.parametrize("kind", KINDS)
def test_ties_small_and_extreme_values(kind):
    top = KINDS[kind]
    x = torch.zeros(9, 64)
    x[0] = torch.arange(64) - 31.5
    x[0, 0] = top                                             # factor 1: halves between the codes, to even
    x[1, 3] = -2.0 ** -100                                    # the smallest block that is held
    x[2, 3] = 2.0 ** -100 * (1 - 2.0 ** -24)                  # and one below it
    x[3] = 3.4e38                                             # the largest magnitudes
    x[4] = torch.linspace(-1, 1, 64) * 1e-30
    x[5] = -0.0
    x[6, 0], x[6, 1:] = 1.0, 2.0 ** -20                       # far below the block's largest
    x[7] = torch.exp(-torch.arange(64) / 4.0)
    x[8] = torch.arange(64) / 63.0 * -5.0
    codes, scales = coded(x, kind, 64)
    store, dev = torch.zeros(9, 64, dtype=torch.uint8, device="cuda").view(kind), torch.zeros(9, 1, device="cuda")
    lists = i32(list(range(9)))
    state_quantize(x.cuda(), lists, store, dev, lists)
    assert torch.equal(dev.cpu(), scales)
    assert torch.equal(store.view(torch.uint8).cpu(), codes)
    back = state_dequantize(store, dev, lists, torch.ones(9, 64, device="cuda"), lists).cpu()
    assert torch.equal(back, values(codes, scales, kind, 64))
    most = x.abs().amax(-1, keepdim=True)
    # Half a code (and the rounding of the factor, the product and the value: 4 u of the value).
    bound = most / 254 if kind == torch.int8 else torch.maximum(x.abs() * 2.0 ** -4, most / 458752)
    held = most >= 2.0 ** -100
    assert ((back - x).abs() <= torch.where(held, bound * (1 + 2.0 ** -12) + 4 * 2.0 ** -24 * x.abs(), most)).all()


@pytest.mark.parametrize("kind", KINDS)
def test_blocks_that_are_not_finite_come_back_as_nan(kind):
    x = torch.randn(1, 256, generator=torch.Generator().manual_seed(1))
    x[0, 70], x[0, 200] = float("nan"), -float("inf")
    store, scales = torch.zeros(1, 256, dtype=torch.uint8, device="cuda").view(kind), torch.zeros(1, 4, device="cuda")
    one = i32([0])
    state_quantize(x.cuda(), one, store, scales, one)
    back = state_dequantize(store, scales, one, torch.zeros(1, 256, device="cuda"), one).cpu().reshape(4, 64)
    assert torch.isnan(back[1]).all() and torch.isnan(back[3]).all()
    assert torch.isfinite(back[0]).all() and torch.isfinite(back[2]).all()


def test_states_of_heads_and_vectors():
    """[P, H, dk, dv] with a scale per key channel, and vector states [P, D] with scales in blocks."""
    gen = torch.Generator().manual_seed(3)
    for shape, lead in (((6, 3, 64, 64), (3, 64)), ((6, 2, 128, 128), (2, 128)), ((6, 1280), (10,)), ((6, 1280), (40,))):
        pool = torch.randn(shape, generator=gen)
        store, scales = torch.zeros((4,) + shape[1:], dtype=torch.int8).cuda(), torch.zeros((4,) + lead).cuda()
        state_quantize(pool.cuda(), i32([5, 2]), store, scales, i32([0, 3]))
        block = pool[0].numel() // scales[0].numel()
        codes, s = coded(pool.reshape(6, -1), torch.int8, block)
        assert torch.equal(store[3].cpu().view(torch.uint8).reshape(-1), codes[2])
        assert torch.equal(scales[0].cpu().reshape(-1), s[5]) and not store[1:3].any()


@pytest.mark.slow
def test_offsets_past_32_bits():
    """A pool of 2^31 + values and a store as large."""
    V, P = 1 << 22, 513
    pool = torch.zeros(P, V, device="cuda")
    pool[-1] = torch.randn(V, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    store, scales = torch.zeros(P, V, dtype=torch.int8, device="cuda"), torch.zeros(P, V // 128, device="cuda")
    state_quantize(pool, i32([P - 1]), store, scales, i32([P - 1]))
    codes, s = coded(pool[-1].cpu(), torch.int8, 128)
    assert torch.equal(store[-1].cpu().view(torch.uint8), codes) and torch.equal(scales[-1].cpu(), s)
    state_dequantize(store, scales, i32([P - 1, P - 1]), pool, i32([P - 2, 0]))
    want = values(codes, s, torch.int8, 128)
    assert torch.equal(pool[0].cpu(), want) and torch.equal(pool[P - 2].cpu(), want) and not pool[1].any()


def test_streams_and_graphs():
    pool = torch.randn(8, 4, 64, 64, device="cuda")
    lists = i32([7, 0, 3]), i32([1, 2, 0])

    def step(stream=None):
        store = torch.zeros(3, 4, 64, 64, dtype=torch.float8_e4m3fn, device="cuda")
        scales, back = torch.zeros(3, 4, 64, device="cuda"), torch.zeros(8, 4, 64, 64, device="cuda")
        if stream is not None:
            torch.cuda.synchronize()
        state_quantize(pool, lists[0], store, scales, lists[1], stream=stream)
        state_dequantize(store, scales, lists[1], back, lists[0], stream=stream)
        return store.view(torch.uint8), scales, back
    want, got = step(), [step(torch.cuda.Stream())]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.append(step())
    lists[0].copy_(i32([0, 0, 0]))
    graph.replay()  # the lists are read at every replay
    torch.cuda.synchronize()
    assert not got[1][2][7].any()
    lists[0].copy_(i32([7, 0, 3]))
    graph.replay()
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals():
    pool, one = torch.zeros(4, 2, 64, device="cuda"), i32([0])
    store, scales = torch.zeros(3, 2, 64, dtype=torch.int8, device="cuda"), torch.zeros(3, 2, device="cuda")
    bad = [(pool.double(), one, store, scales, one), (pool, one, store.view(torch.uint8), scales, one),
           (pool, one, store[:, :1].contiguous(), scales, one), (pool, one, store, scales.view(6), one),
           (pool, one, store, torch.zeros(3, 8, device="cuda"), one), (pool, one, store, torch.zeros(3, 0, device="cuda"), one),
           (pool, one, store, torch.zeros(3, 3, device="cuda"), one), (pool, one.long(), store, scales, one),
           (pool, one, store, scales, i32([0, 1])), (pool, one, store, scales[:2], one), (pool[0, 0], one, store, scales, one)]
    for p, src, s, f, dst in bad:
        with pytest.raises(ValueError):
            state_quantize(p, src, s, f, dst)
        with pytest.raises(ValueError):
            state_dequantize(s, f, src, p, dst)
    many = i32([0] * 4097)
    with pytest.raises(RuntimeError):
        state_quantize(pool, many, store, scales, many)
    state_copy(pool, one, one)  # the context is as it was
