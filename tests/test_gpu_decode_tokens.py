"""The delta rule over several tokens a row against the 64-bit recurrence and the single steps."""
import numpy as np
import pytest
import torch

from kimi_delta_attention_17_gb300 import build, decode_step, decode_tokens
from tests import layer_reference as ref
from tests.layer_reference import f64, half_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def inputs(N, K, H, d, dtype, P=None, decay="channel", gate="log", l2norm=False, seed=0, steep=0.0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k, v = n(N, K, H, d), n(N, K, H, d), n(N, K, H, d)
    if not l2norm:
        q, k = (torch.nn.functional.normalize(t, dim=-1) for t in (q, k))
    shape = (N, K, H, d) if decay == "channel" else (N, K, H)
    g = n(*shape)
    g = -torch.nn.functional.softplus(g - 3.0 + steep) if gate == "log" else g + 3.0 - steep
    a = dict(q=q.to(dtype), k=k.to(dtype), v=v.to(dtype), g=None if decay == "none" else g, beta=torch.sigmoid(n(N, K, H)),
             state=0.3 * n(N if P is None else P, H, d, d))
    return {x: None if t is None else t.cuda() for x, t in a.items()}


def check(a, scale, counts=None, slots=None, decay="channel", gate="log", lower=-5.0, l2norm=False, write=True, want=True):
    N, K, H, d = a["q"].shape
    before = a["state"].clone()
    out = decode_tokens(a["q"], a["k"], a["v"], a["g"], a["beta"], scale, a["state"], write_state=write, want_out=want,
                        counts=None if counts is None else i32(counts), slots=None if slots is None else i32(slots),
                        decay=decay, gate=gate, gate_lower=lower, l2norm_qk=l2norm)
    x = {n: None if t is None else f64(t) for n, t in a.items()}
    after, got = f64(before), None if out is None else f64(out)
    held = f64(a["state"])
    if not want:
        assert out is None
    for n in range(N):
        at = n if slots is None else slots[n]
        count = K if counts is None else min(max(counts[n], 0), K)
        if not 0 <= at < a["state"].shape[0]:
            count = 0
        for h in range(H):
            if count:
                al = np.ones((K, d)) if decay == "none" else ref.decay(x["g"][n, :, h], gate, lower)
                al = np.broadcast_to(al.reshape(K, -1), (K, d))
                r = ref.tokens(x["q"][n, :, h], x["k"][n, :, h], x["v"][n, :, h], al, x["beta"][n, :, h], scale,
                               after[at, h], count, l2norm)
                if write:
                    tol = r["tol_state"] + half_step(r["state"], False)
                    assert (np.abs(held[at, h] - r["state"]) <= tol).all(), "state of row %d" % n
                    after[at, h] = held[at, h]
                if want:
                    tol = r["tol_out"] + half_step(r["out"], a["q"].dtype == BF)
                    off = np.abs(got[n, :count, h] - r["out"][:count]) / tol[:count]
                    assert off.max() <= 1.0, "row %d: %.3g times its bound" % (n, off.max())
            if want:
                assert not got[n, count:, h].any()
    assert np.array_equal(held, after)  # every other state as it was
    return out


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 7, 8, 9, 16, 17, 33])
def test_tokens(K, d, dtype):
    check(inputs(2, K, 3, d, dtype, seed=K), d ** -0.5)
    check(inputs(2, K, 3, d, dtype, seed=K), d ** -0.5, write=False)


@pytest.mark.parametrize("decay", ["channel", "scalar", "none"])
@pytest.mark.parametrize("gate", ["log", "logsigmoid", "bounded"])
@pytest.mark.parametrize("l2norm", [False, True])
def test_options(decay, gate, l2norm):
    for d, dtype in ((64, F), (128, BF)):
        a = inputs(2, 6, 2, d, dtype, decay=decay, gate=gate, l2norm=l2norm)
        check(a, d ** -0.5, decay=decay, gate=gate, l2norm=l2norm, lower=-3.0)


@pytest.mark.parametrize("d,dtype", [(64, F), (128, BF), (128, F)])
def test_counts_and_slots(d, dtype):
    counts = [0, 1, 5, 9, 3, -4, 100, 8, 9, 2]
    slots = [4, -1, 0, 11, 7, 3, 10, 12, 1, 2 ** 31 - 1]
    a = inputs(10, 9, 2, d, dtype, P=12)
    check(a, d ** -0.5, counts, slots)
    a = inputs(10, 9, 2, d, dtype, P=12)
    check(a, d ** -0.5, counts, slots, write=False)
    check(a, d ** -0.5, counts, slots, want=False)
    check(inputs(10, 9, 2, d, dtype), d ** -0.5, counts)


@pytest.mark.parametrize("gate,steep", [("log", 60.0), ("logsigmoid", 60.0), ("log", -40.0)])
def test_extreme_decays(gate, steep):
    """Decays down to e^-100, and of 1: no quotient of decays is formed that could overflow."""
    a = inputs(2, 12, 2, 128, F, gate=gate, steep=steep)
    if steep > 0:
        a["g"][:, ::3] = 0.0 if gate == "log" else 30.0
    check(a, 0.1, gate=gate)


def test_zero_decay_clears_the_state():
    a = inputs(1, 4, 2, 64, F)
    a["g"][:, 2] = -float("inf")
    a["state"][0, 0, 3] = 1e30
    out = decode_tokens(a["q"], a["k"], a["v"], a["g"], a["beta"], 0.125, a["state"])
    rest = {n: t[:, 2:].contiguous() for n, t in a.items() if n != "state"}
    rest["g"][:, 0] = 0.0
    clean = torch.zeros_like(a["state"])
    want = decode_tokens(rest["q"], rest["k"], rest["v"], rest["g"], rest["beta"], 0.125, clean)
    assert torch.isfinite(out[:, 2:]).all() and torch.isfinite(a["state"]).all()
    assert torch.allclose(out[:, 2:], want, rtol=0, atol=1e-5) and torch.allclose(a["state"], clean, rtol=0, atol=1e-5)


def test_equals_single_steps():
    """The same tokens one at a time: outputs and states within the sum of both bounds (here: 2^-15 of order-one
    values covers 12 steps of 320 u each way)."""
    a = inputs(3, 12, 4, 128, F, gate="logsigmoid", l2norm=True)
    state = a["state"].clone()
    outs = [decode_step(*(a[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")), 0.1, state, gate="logsigmoid",
                        l2norm_qk=True) for t in range(12)]
    out = decode_tokens(a["q"], a["k"], a["v"], a["g"], a["beta"], 0.1, a["state"], gate="logsigmoid", l2norm_qk=True)
    assert (out - torch.stack(outs, 1)).abs().max() < 2.0 ** -12
    assert (a["state"] - state).abs().max() < 2.0 ** -12


def test_verify_then_commit():
    """Drafts verified without a write, then the accepted ones committed: the states are those of the accepted
    tokens alone, and the outputs of both calls agree."""
    a = inputs(5, 6, 3, 64, BF, P=9)
    slots, accepted = i32([8, 0, 3, 5, 2]), i32([6, 0, 2, 1, 4])
    before = a["state"].clone()
    args = (a["q"], a["k"], a["v"], a["g"], a["beta"], 0.125, a["state"])
    drafts = decode_tokens(*args, slots=slots, write_state=False)
    assert torch.equal(a["state"], before)
    again = decode_tokens(*args, slots=slots, counts=accepted, write_state=False)
    for n, c in enumerate(accepted.tolist()):
        assert torch.equal(again[n, :c], drafts[n, :c]) and not again[n, c:].any()
    assert decode_tokens(*args, slots=slots, counts=accepted, want_out=False) is None
    for n, c in enumerate(accepted.tolist()):
        one = before[slots[n]].clone()[None]
        rows = [t[n:n + 1, :c].contiguous() for t in args[:5]]
        decode_tokens(*rows, 0.125, one)
        assert torch.equal(a["state"][slots[n]], one[0])
    assert torch.equal(a["state"][1], before[1])


def test_a_row_that_is_not_finite_touches_no_other():
    a = inputs(4, 3, 2, 64, F)
    want = decode_tokens(a["q"], a["k"], a["v"], a["g"], a["beta"], 0.125, a["state"].clone())
    a["v"][1] = float("nan")
    a["state"][2, 1] = float("inf")
    out = decode_tokens(a["q"], a["k"], a["v"], a["g"], a["beta"], 0.125, a["state"])
    assert torch.equal(out[0], want[0]) and torch.equal(out[3], want[3]) and torch.equal(out[2, :, 0], want[2, :, 0])
    assert torch.isnan(out[1]).all() and torch.isfinite(a["state"][0]).all() and torch.isfinite(a["state"][3]).all()


@pytest.mark.parametrize("d,dtype", [(64, BF), (128, BF), (128, F)])
def test_what_lies_behind_the_counts_is_not_read(d, dtype):
    """NaN and infinities in the tokens behind a row's count, and in rows without a slot, touch nothing."""
    counts, slots = [3, 0, 9, 17, 8, 5, 1], [6, 5, 4, 3, 2, -1, 0]
    a = inputs(7, 17, 2, d, dtype, gate="logsigmoid", l2norm=True)
    how = dict(slots=i32(slots), counts=i32(counts), gate="logsigmoid", l2norm_qk=True)
    clean = a["state"].clone()
    want = decode_tokens(a["q"], a["k"], a["v"], a["g"], a["beta"], 0.1, clean, **how)
    for n, (c, s) in enumerate(zip(counts, slots)):
        for x, name in enumerate(("q", "k", "v", "g", "beta")):
            a[name][n, 0 if s < 0 else c:] = (float("nan"), float("inf"), -float("inf"))[(n + x) % 3]
    for _ in range(2):  # the second time over what the first left in shared memory
        state = a["state"].clone()
        out = decode_tokens(a["q"], a["k"], a["v"], a["g"], a["beta"], 0.1, state, **how)
        assert torch.equal(out, want) and torch.equal(state, clean)


def test_rows_may_share_a_state_that_is_not_written():
    a = inputs(4, 5, 3, 64, BF, P=3)
    before = a["state"].clone()
    out = decode_tokens(a["q"], a["k"], a["v"], a["g"], a["beta"], 0.1, a["state"], slots=i32([1, 1, 2, 1]), write_state=False)
    for n, at in enumerate((1, 1, 2, 1)):
        row = [a[x][n:n + 1] for x in ("q", "k", "v", "g", "beta")]
        assert torch.equal(out[n:n + 1], decode_tokens(*row, 0.1, before[at:at + 1].clone()))
    assert torch.equal(a["state"], before)


def test_no_rows_no_tokens_given_outputs():
    a = inputs(2, 3, 2, 64, BF)
    before = a["state"].clone()
    none = {n: t[:, :0].contiguous() for n, t in a.items() if n != "state"}
    assert decode_tokens(none["q"], none["k"], none["v"], none["g"], none["beta"], 1.0, a["state"]).shape == (2, 0, 2, 64)
    rows = {n: t[:0] for n, t in a.items() if n != "state"}
    assert decode_tokens(rows["q"], rows["k"], rows["v"], rows["g"], rows["beta"], 1.0, a["state"], slots=i32([])).numel() == 0
    assert torch.equal(a["state"], before)
    out = torch.full_like(a["v"], 9.0)
    got = decode_tokens(a["q"], a["k"], a["v"], a["g"], a["beta"], 1.0, a["state"], out=out, counts=i32([0, 0]))
    assert got is out and not out.any() and torch.equal(a["state"], before)


def test_streams_and_graphs():
    a = inputs(6, 5, 4, 128, BF, P=8, gate="logsigmoid", l2norm=True)
    slots, counts, first = i32([7, 0, 1, 2, 3, 4]), i32([5, 4, 3, 2, 1, 0]), a["state"].clone()
    args = (a["q"], a["k"], a["v"], a["g"], a["beta"], 0.1)
    how = dict(slots=slots, counts=counts, gate="logsigmoid", l2norm_qk=True)
    state = first.clone()
    want = decode_tokens(*args, state, **how)
    torch.cuda.synchronize()
    side, other = first.clone(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = decode_tokens(*args, side, stream=other, **how)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(side, state)
    held = first.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = decode_tokens(*args, held, **how)
    for change in (False, True):
        held.copy_(first)
        if change:
            counts.copy_(i32([0, 1, 2, 3, 4, 5]))  # read at every replay
        graph.replay()
        state = first.clone()
        want = decode_tokens(*args, state, **how)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(held, state)


@pytest.mark.parametrize("K", [3, 8])
def test_thousands_of_tokens_do_not_drift(K):
    """400 calls without decay, little written by each: a state that is rounded once a call is off by at most half a
    unit of its last place each time (400 x 2^-24 of its magnitudes), and what is written, 1e-3 of it, by far less."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    S = n(2, 2, 128, 128) * 0.1
    exact = S.double()
    beta = torch.full((2, K, 2), 1e-3, device="cuda")
    for _ in range(400):
        q, v, k = n(2, K, 2, 128), n(2, K, 2, 128), torch.nn.functional.normalize(n(2, K, 2, 128), dim=-1)
        decode_tokens(q, k, v, None, beta, 0.1, S, decay="none", want_out=False)
        for t in range(K):
            kt = k[:, t].double()
            e = 1e-3 * (v[:, t].double() - torch.einsum("nhij,nhi->nhj", exact, kt))
            exact += kt[..., None] * e[:, :, None]
    beta64 = float(torch.tensor(1e-3, dtype=F))  # the oracle's 1e-3 is off by 2^-25 of itself: nothing beside the bound
    assert abs(beta64 - 1e-3) < 1e-10
    assert ((S.double() - exact).norm() / exact.norm()).item() <= 430 * 2.0 ** -24


@pytest.mark.slow
def test_offsets_past_32_bits():
    """A pool of 2^31 + values: 2100 slots of 64 heads of 128 x 128 have 2.2e9."""
    H, d, P = 64, 128, 2100
    a = inputs(2, 3, H, d, BF)
    pool = torch.zeros(P, H, d, d, device="cuda")
    pool[P - 1], pool[5] = a["state"][0], a["state"][1]
    out = decode_tokens(a["q"], a["k"], a["v"], a["g"], a["beta"], 0.1, pool, slots=i32([P - 1, 5]))
    want = decode_tokens(a["q"], a["k"], a["v"], a["g"], a["beta"], 0.1, a["state"])
    assert torch.equal(out, want) and torch.equal(pool[P - 1], a["state"][0]) and torch.equal(pool[5], a["state"][1])


def test_many_rows_of_one_head():
    """More (row, head) pairs than a grid's second dimension holds."""
    N, d = 70001, 64
    a = inputs(3, 2, 1, d, F)
    big = {n: t[:1].expand(N, *t.shape[1:]).contiguous() for n, t in a.items()}
    out = decode_tokens(big["q"], big["k"], big["v"], big["g"], big["beta"], 0.1, big["state"])
    want = decode_tokens(a["q"], a["k"], a["v"], a["g"], a["beta"], 0.1, a["state"])
    assert torch.equal(out[N - 1], want[0]) and torch.equal(out[65536], want[0])
    assert (big["state"] == a["state"][0]).all()


@pytest.mark.parametrize("d,H,N,K,dtype", [(64, 1, 45001, 11, BF), (64, 3, 13001, 17, F), (128, 2, 10501, 9, BF),
                                           (128, 5, 4207, 10, F)])
def test_many_heads_a_cta(d, H, N, K, dtype):
    """Hundreds of heads for every CTA, most rows without tokens or with one block, some with several: outputs and
    states bit for bit those of the same rows in small calls."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, v = n(N, K, H, d).to(dtype), n(N, K, H, d).to(dtype)
    k = torch.nn.functional.normalize(n(N, K, H, d), dim=-1).to(dtype)
    g, beta = n(N, K, H, d) + 3.0, torch.sigmoid(n(N, K, H))
    state = n(N, H, d, d) * 0.1
    counts = torch.randint(-K, K + 1, (N,), generator=gen, device="cuda").to(torch.int32)
    counts[1000:1700] = 0  # runs of rows without tokens, longer than what a CTA looks at together takes
    slots = torch.randperm(N, generator=gen, device="cuda").to(torch.int32)
    slots[::50] = -1
    before = state.clone()
    out = decode_tokens(q, k, v, g, beta, 0.1, state, slots=slots, counts=counts, gate="logsigmoid")
    for lo in list(range(0, N - 40, N // 23)) + [N - 40]:
        rows = slice(lo, lo + 40)
        at = slots[rows].long().clamp(min=0)
        own = torch.arange(40, dtype=torch.int32, device="cuda")
        own[slots[rows] < 0] = -1
        part = before[at].clone()
        want = decode_tokens(q[rows], k[rows], v[rows], g[rows], beta[rows], 0.1, part, slots=own, counts=counts[rows],
                             gate="logsigmoid")
        assert torch.equal(out[rows], want)
        held = slots[rows] >= 0
        assert torch.equal(state[at][held], part[held])
    idle = torch.ones(N, dtype=torch.bool, device="cuda")
    idle[slots[(slots >= 0) & (counts > 0)].long()] = False
    assert torch.equal(state[idle], before[idle])


def test_refusals():
    a = inputs(2, 3, 2, 64, BF)
    def call(**kw):
        b = {**a, **{n: kw.pop(n) for n in list(kw) if n in a}}
        return decode_tokens(b["q"], b["k"], b["v"], b["g"], b["beta"], 1.0, b["state"], **kw)
    for kw in (dict(k=a["k"][:1]), dict(v=a["v"][:, :2].contiguous()), dict(beta=a["beta"][:1]), dict(g=a["g"][:1]),
               dict(state=a["state"][:1]), dict(state=a["state"][:, :1].contiguous()), dict(slots=i32([0])),
               dict(counts=i32([1, 2, 3])), dict(counts=torch.tensor([1, 2], device="cuda")),
               dict(write_state=False, want_out=False), dict(out=a["v"][:1]), dict(out=a["v"].clone(), want_out=False),
               dict(decay="row"), dict(gate="tanh"), dict(k=a["k"].float()), dict(q=a["q"].transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**kw)
