"""The decode over several tokens where most of a large call's rows have none: a CTA finds few blocks before the
end of the pairs that it looks at together, and long runs of pairs without tokens behind them."""
import pytest
import torch

from kimi_delta_attention_17_gb300 import build, decode_tokens

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
SMS, WINDOW, K = 152, 128, 24  # CTAs of 128 channels (twice as many of 64), pairs looked at together, tokens


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def run(d, dtype, held, write, pooled):
    """As many heads as CTAs, so that a CTA's pairs are the rows of its head. `held`: {row: tokens} of the rows that
    have any. Outputs and states are bit for bit those of these rows by themselves."""
    H, N = SMS if d == 128 else 2 * SMS, 2 * WINDOW + 6
    gen = torch.Generator(device="cuda").manual_seed(len(held) + d)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    tensors = dict(q=n(N, K, H, d).to(dtype), k=torch.nn.functional.normalize(n(N, K, H, d), dim=-1).to(dtype),
                   v=n(N, K, H, d).to(dtype), g=n(N, K, H, d) + 3.0, beta=torch.sigmoid(n(N, K, H)))
    rows = sorted(held)
    counts = [held.get(i, 0) for i in range(N)]
    slots = None
    if pooled:  # rows without tokens have no slot, or one that does not exist, and counts that say nothing
        slots = [rows.index(i) + 1 if i in held else (-1, 2 ** 31 - 1)[i % 2] for i in range(N)]
        counts = [c if i in held else i % (K + 1) for i, c in enumerate(counts)]
    state = 0.1 * n(len(rows) + 2 if pooled else N, H, d, d)
    before = state.clone()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    how = dict(gate="logsigmoid", write_state=write)
    out = decode_tokens(*tensors.values(), 0.1, state, counts=i32(counts), slots=None if slots is None else i32(slots), **how)
    places = torch.tensor(range(1, len(rows) + 1) if pooled else rows, dtype=torch.long, device="cuda")
    if rows:
        part, picked = before[places].clone(), torch.tensor(rows, device="cuda")
        want = decode_tokens(*(t[picked] for t in tensors.values()), 0.1, part, counts=i32([held[i] for i in rows]), **how)
        assert torch.equal(out[picked], want) and want[0, :held[rows[0]]].any()
        assert torch.equal(state[places], part) and torch.equal(part, before[places]) != write
    idle = torch.ones(N, dtype=torch.bool, device="cuda")
    idle[rows] = False
    assert not out[idle].any()
    rest = torch.ones(state.shape[0], dtype=torch.bool, device="cuda")
    rest[places] = False
    assert torch.equal(state[rest], before[rest])


@pytest.mark.parametrize("d,dtype", [(64, BF), (128, BF), (128, F)])
@pytest.mark.parametrize("blocks", range(6))
def test_few_blocks_before_a_windows_end(d, dtype, blocks):
    one = {5: 8 * blocks - 3} if 0 < blocks <= 3 else {5: 24, 9: 8 * (blocks - 3)} if blocks else {}
    each = {7 * i: 8 - i for i in range(blocks)}
    late = {WINDOW: 3, WINDOW + 1: 17, 2 * WINDOW: 8, 2 * WINDOW + 5: 1}
    run(d, dtype, one, write=True, pooled=True)
    run(d, dtype, {**each, **late}, write=True, pooled=True)
    run(d, dtype, {**one, 2 * WINDOW + 5: 9}, write=False, pooled=True)


@pytest.mark.parametrize("d,dtype", [(64, F), (128, BF)])
def test_at_a_windows_last_pairs(d, dtype):
    run(d, dtype, {WINDOW - 3: 8, WINDOW - 2: 8, WINDOW - 1: 8, 2 * WINDOW: 24}, write=True, pooled=False)
    run(d, dtype, {WINDOW - 1: 24, WINDOW: 24}, write=True, pooled=False)
    run(d, dtype, {0: 24, 2 * WINDOW - 1: 1}, write=False, pooled=False)
