"""Gated linear recurrence on the GPU against the 64-bit reference, within the
bounds that fp32 arithmetic and the outputs' types allow (scan_reference)."""
import numpy as np
import pytest
import torch

from kimi_delta_attention_17_gb300 import (build, gated_scan_bwd, gated_scan_fwd, gated_scan_step)
from tests import scan_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": (torch.float32, torch.float32), "mixed": (torch.bfloat16, torch.float32),
         "bf16": (torch.bfloat16, torch.bfloat16)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def f64(t):
    return t.detach().double().cpu().numpy()


def make(B, T, D, types, gate="log", seed=0, N=None, init=True):
    gen = torch.Generator().manual_seed(1000 + seed)
    dt, gdt = TYPES[types]
    N = B if N is None else N
    n = torch.randn(B, T, D, generator=gen)
    z = {"log": -torch.nn.functional.softplus(n - 2), "logsigmoid": n + 2, "bounded": n - 2}[gate]
    return dict(x=torch.randn(B, T, D, generator=gen).to(dt), g=z.to(gdt),
                dout=torch.randn(B, T, D, generator=gen).to(dt),
                init=torch.randn(N, D, generator=gen) if init else None,
                dfinal=torch.randn(N, D, generator=gen) if init else None)


def cuda(v):
    return {k: None if t is None else t.cuda() for k, t in v.items()}


def close(got, want, tol, name):
    rounding = ref.BF16 if got.dtype == torch.bfloat16 else 0.0
    got = f64(got)
    assert got.shape == want.shape
    off = np.abs(got - want)
    bad = ~(off <= tol + rounding * (np.abs(want) + tol))
    assert not bad.any(), "%s: %d of %d out of bounds, first at %s: %r for %r, bound %.3g" % (
        name, bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], want[bad][0], tol[bad][0])


def check(v, gate, write, lower=-5.0, cu=None, backward=True, **kw):
    """Runs both directions and compares every output."""
    c = cuda(v)
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    how = dict(gate=gate, gate_lower=lower, write=write)
    out, final, carries = gated_scan_fwd(c["x"], c["g"], c["init"], cut, save_carries=True, **how, **kw)
    if backward:
        dx, dg, dinit = gated_scan_bwd(c["dout"], c["x"], c["g"], carries, cut, dfinal_state=c["dfinal"], **how)
    torch.cuda.synchronize()
    B, T, D = v["x"].shape
    x, g, do = (f64(v[n]).reshape(B * T, D) for n in ("x", "g", "dout"))
    for n, (lo, hi) in enumerate(ref.spans(B, T, cu)):
        r = ref.scan(x[lo:hi], g[lo:hi], None if v["init"] is None else f64(v["init"])[n], gate, lower, write,
                     do[lo:hi], None if v["dfinal"] is None else f64(v["dfinal"])[n])
        tag = "sequence %d " % n
        close(out.reshape(B * T, D)[lo:hi], r["out"], r["tol_out"], tag + "out")
        close(final[n], r["final"], r["tol_final"], tag + "final")
        if backward:
            close(dx.reshape(B * T, D)[lo:hi], r["dx"], r["tol_dx"], tag + "dx")
            close(dg.reshape(B * T, D)[lo:hi], r["dg"], r["tol_dg"], tag + "dg")
            close(dinit[n], r["dinit"], r["tol_dinit"], tag + "dinit")


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("write", ["plain", "complement", "norm"])
@pytest.mark.parametrize("gate", ["log", "logsigmoid", "bounded"])
def test_every_form(gate, write, types):
    check(make(2, 301, 72, types, gate), gate, write)


@pytest.mark.parametrize("write", ["plain", "complement", "norm"])
@pytest.mark.parametrize("gate", ["log", "logsigmoid", "bounded"])
def test_long_chains_of_bf16(gate, write):
    """One sequence of more than 1024 tokens: 8 tokens a thread in the forward pass."""
    check(make(1, 1333, 72, "bf16", gate, seed=7), gate, write)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 7, 8, 9, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 513, 1023, 2049, 5000])
@pytest.mark.parametrize("types", list(TYPES))
def test_lengths(T, types):
    check(make(1, T, 8, types, "logsigmoid", seed=T), "logsigmoid", "complement")


@pytest.mark.parametrize("T,D", [(200, 4), (77, 12), (300, 132)])
def test_fp32_shapes(T, D):
    check(make(2, T, D, "f32", "logsigmoid", seed=D), "logsigmoid", "norm")


@pytest.mark.parametrize("B,T,D", [(1, 300, 8), (3, 70, 24), (1, 130, 1032), (2, 40, 4096), (64, 3, 64), (400, 1, 264),
                                   (5, 200, 2048)])
def test_shapes(B, T, D):
    check(make(B, T, D, "bf16", "bounded", seed=B + T + D), "bounded", "norm")


@pytest.mark.parametrize("B,T", [(2, 1), (5, 4), (3, 16), (9, 15), (5, 17), (2, 32), (7, 31), (3, 33)])
@pytest.mark.parametrize("types", list(TYPES))
def test_many_short_sequences(B, T, types):
    """Around the lengths up to which each warp takes a sequence of its own (16, or 32)."""
    check(make(B, T, 72, types, "logsigmoid", seed=B * T), "logsigmoid", "complement")
    check(make(B, T, 264, types, "log", seed=T, init=False), "log", "norm")


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("cu", [[0, 1], [0, 0, 5, 5, 133, 134, 134], [0, 128, 256, 400], [0, 700, 701, 1400],
                                [0, 3, 6, 9, 12, 15, 18, 21], [0, 0, 0]])
def test_packed(cu, types):
    v = make(1, max(cu[-1], 0), 24, types, "log", seed=len(cu), N=len(cu) - 1)
    check(v, "log", "complement", cu=cu)


def test_no_states():
    check(make(2, 150, 16, "mixed", "log", init=False), "log", "plain")


@pytest.mark.parametrize("N,most", [(90, 40), (128, 300), (129, 9), (200, 100)])
def test_many_packed_sequences(N, most):
    """Up to 128 sequences are taken longest first, more in their order."""
    rng = np.random.default_rng(N)
    cu = np.concatenate([[0], np.cumsum(rng.integers(0, most, N))]).tolist()
    check(make(1, cu[-1], 8, "bf16", "logsigmoid", N=N), "logsigmoid", "norm", cu=cu)


def test_offsets_that_do_not_fit_stay_inside():
    """Offsets past the tokens, below zero or falling are clamped: values are unspecified, memory
    beside the outputs is not touched."""
    T, D = 70, 16
    v = cuda(make(1, T, D, "f32", N=4))
    cu = torch.tensor([-5, 30, 10, 2 ** 31 - 1, 60], dtype=torch.int32, device="cuda")

    def guarded(rows):
        whole = torch.full((rows + 2, D), 7.0, device="cuda")
        return whole, whole[1:-1]

    outw, out = guarded(T)
    finw, fin = guarded(4)
    carw, car = guarded(T // 64 + 4)
    gated_scan_fwd(v["x"], v["g"], v["init"], cu, out=out.view(1, T, D), final_state=fin, carries=car)
    dxw, dx = guarded(T)
    dgw, dg = guarded(T)
    dinw, din = guarded(4)
    gated_scan_bwd(v["dout"], v["x"], v["g"], car, cu, dfinal_state=v["dfinal"], dx=dx.view(1, T, D),
                   dg=dg.view(1, T, D), dinit_state=din)
    torch.cuda.synchronize()
    for whole in (outw, finw, carw, dxw, dgw, dinw):
        assert (whole[0] == 7.0).all() and (whole[-1] == 7.0).all()


def test_rows_outside_every_sequence_stay():
    v = make(1, 300, 16, "bf16", N=2)
    c = cuda(v)
    cu = torch.tensor([7, 150, 260], dtype=torch.int32, device="cuda")
    out = torch.full_like(c["x"], 3.0)
    carries = torch.full((300 // 64 + 2, 16), 5.0, device="cuda")
    gated_scan_fwd(c["x"], c["g"], c["init"], cu, out=out, carries=carries)
    dx, dg = torch.full_like(c["x"], 4.0), torch.full_like(c["g"], 6.0)
    gated_scan_bwd(c["dout"], c["x"], c["g"], carries, cu, dfinal_state=c["dfinal"], dx=dx, dg=dg)
    for t, value in ((out, 3.0), (dx, 4.0), (dg, 6.0)):
        assert (t[0, :7] == value).all() and (t[0, 260:] == value).all()
        assert not (t[0, 7:260] == value).all()
    x, g = f64(v["x"])[0], f64(v["g"])[0]
    for n, (lo, hi) in enumerate([(7, 150), (150, 260)]):
        r = ref.scan(x[lo:hi], g[lo:hi], f64(v["init"])[n])
        close(out[0, lo:hi], r["out"], r["tol_out"], "out")


def test_states_in_place():
    """init_state is final_state, dfinal_state is dinit_state; several CTAs read them."""
    v = make(1, 3000, 8, "f32", "logsigmoid")
    c = cuda(v)
    how = dict(gate="logsigmoid", write="complement")
    out, final, carries = gated_scan_fwd(c["x"], c["g"], c["init"], save_carries=True, **how)
    dx, dg, dinit = gated_scan_bwd(c["dout"], c["x"], c["g"], carries, dfinal_state=c["dfinal"], **how)
    state, grad = c["init"].clone(), c["dfinal"].clone()
    out2, _, _ = gated_scan_fwd(c["x"], c["g"], state, final_state=state, **how)
    gated_scan_bwd(c["dout"], c["x"], c["g"], carries, dfinal_state=grad, dinit_state=grad, **how)
    assert torch.equal(out, out2) and torch.equal(final, state) and torch.equal(dinit, grad)


def test_resumed_sequence_is_the_whole_one():
    v = make(1, 900, 16, "f32", "logsigmoid")
    c = cuda(v)
    whole, last, _ = gated_scan_fwd(c["x"], c["g"], c["init"], gate="logsigmoid", write="norm")
    a, mid, _ = gated_scan_fwd(c["x"][:, :333].contiguous(), c["g"][:, :333].contiguous(), c["init"],
                               gate="logsigmoid", write="norm")
    b, end, _ = gated_scan_fwd(c["x"][:, 333:].contiguous(), c["g"][:, 333:].contiguous(), mid,
                               gate="logsigmoid", write="norm")
    r = ref.scan(f64(v["x"])[0], f64(v["g"])[0], f64(v["init"])[0], "logsigmoid", -5.0, "norm")
    both = torch.cat([a, b], 1)[0]
    close(both, r["out"], 2 * r["tol_out"], "resumed")
    close(end[0], r["final"], 2 * r["tol_final"], "resumed final")
    close(whole[0], r["out"], r["tol_out"], "whole")


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("write", ["plain", "complement", "norm"])
def test_extreme_log_gates(types, write):
    """Restarts (-inf and the lowest finite value), a = 1, and decays next to 1."""
    v = make(1, 600, 8, types)
    lowest = torch.finfo(v["g"].dtype).min
    v["g"][0, ::7] = -float("inf")
    v["g"][0, 3::11] = lowest
    v["g"][0, 200:460] = 0.0
    v["g"][0, 500:, :4] = -1e-6
    v["g"][0, 420, :] = -100.0
    check(v, "log", write)


@pytest.mark.parametrize("gate", ["logsigmoid", "bounded"])
@pytest.mark.parametrize("write", ["plain", "complement", "norm"])
def test_extreme_logits(gate, write):
    v = make(1, 400, 8, "f32", gate)
    for i, z in enumerate((float("inf"), -float("inf"), 88.0, -88.0, 20.0, -20.0, 3e38, -3e38, 0.0)):
        v["g"][0, 10 + i::37] = z
    check(v, gate, write)


def test_slow_channels_keep_their_accuracy():
    """Decays of 0.9999 and up over thousands of tokens, where a rounding of a that leans to one
    side would add up."""
    v = make(1, 6000, 8, "f32")
    v["g"] = -torch.rand(1, 6000, 8, generator=torch.Generator().manual_seed(3)) * 2e-4
    c = cuda(v)
    for write in ("plain", "norm"):
        out, final, _ = gated_scan_fwd(c["x"], c["g"], c["init"], write=write)
        r = ref.scan(f64(v["x"])[0], f64(v["g"])[0], f64(v["init"])[0], "log", -5.0, write)
        # Unbiased roundings of u = 2^-24 per token over the 10^4 tokens remembered: a walk of
        # 100 u, i.e. 6e-6 of the state's size; a lean of u itself would give 6e-4.
        off = np.linalg.norm(f64(out)[0] - r["out"]) / np.linalg.norm(r["out"])
        assert off <= 1e-5


def test_nan_stays_in_its_channel_and_sequence():
    v = make(2, 300, 8, "f32")
    v["x"][0, 100, 2] = float("nan")
    c = cuda(v)
    out, final, carries = gated_scan_fwd(c["x"], c["g"], c["init"], save_carries=True)
    bad = torch.isnan(out)
    assert bad[0, 100:, 2].all() and bad.sum() == 200 and torch.isnan(final).sum() == 1
    dx, dg, dinit = gated_scan_bwd(c["dout"], c["x"], c["g"], carries, dfinal_state=c["dfinal"])
    assert not torch.isnan(dx).any() and not torch.isnan(dinit).any()
    assert torch.isnan(dg)[0, 101:, 2].all() and torch.isnan(dg).sum() == 199


def test_repeatable_and_on_another_stream():
    c = cuda(make(1, 4000, 40, "bf16", "logsigmoid"))
    how = dict(gate="logsigmoid", write="norm")

    def both(**kw):
        out, final, carries = gated_scan_fwd(c["x"], c["g"], c["init"], save_carries=True, **how, **kw)
        return (out, final) + gated_scan_bwd(c["dout"], c["x"], c["g"], carries, dfinal_state=c["dfinal"], **how, **kw)

    first = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for r in (both(), both(stream=side)):
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, r))


def test_calls_at_once_on_two_streams():
    """Clusters of several calls share the GPU; none waits for another's."""
    how = dict(gate="logsigmoid", write="norm")
    data = [cuda(make(1, 6000, 512, "bf16", "logsigmoid", seed=s)) for s in range(2)]

    def both(c, **kw):
        out, final, carries = gated_scan_fwd(c["x"], c["g"], c["init"], save_carries=True, **how, **kw)
        return (out, final) + gated_scan_bwd(c["dout"], c["x"], c["g"], carries, dfinal_state=c["dfinal"], **how, **kw)

    alone = [both(c) for c in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    for _ in range(5):
        got = [both(c, stream=s) for c, s in zip(data, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_channel_dimensions():
    c = cuda(make(2, 50, 24, "bf16"))
    flat, final, _ = gated_scan_fwd(c["x"], c["g"], c["init"])
    heads, hfinal, _ = gated_scan_fwd(c["x"].view(2, 50, 3, 8), c["g"].view(2, 50, 3, 8), c["init"].view(2, 3, 8))
    assert torch.equal(flat.view_as(heads), heads) and torch.equal(final.view_as(hfinal), hfinal)


def test_no_tokens():
    x = torch.empty(2, 0, 8, device="cuda")
    init = torch.randn(2, 8, device="cuda")
    out, final, carries = gated_scan_fwd(x, x, init, save_carries=True)
    assert out.shape == x.shape and torch.equal(final, init)
    dx, dg, dinit = gated_scan_bwd(x, x, x, carries, dfinal_state=init)
    assert dx.shape == x.shape and torch.equal(dinit, init)
    _, final, _ = gated_scan_fwd(x, x)
    assert (final == 0).all()


def test_offsets_past_32_bits():
    """2.2e9 elements: the last tokens, whose memory is short, against the reference."""
    T, D = 270000, 8192
    x = torch.zeros(1, T, D, dtype=torch.bfloat16, device="cuda")
    g = torch.full((1, T, D), -1.0, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(9)
    tail = torch.randn(200, D, generator=gen).bfloat16()
    x[0, -200:] = tail.cuda()
    out, final, carries = gated_scan_fwd(x, g, save_carries=True)
    r = ref.scan(f64(tail), np.full((200, D), -1.0), dout=f64(tail))
    close(out[0, -200:], r["out"], r["tol_out"], "out")
    close(final[0], r["final"], r["tol_final"], "final")
    assert (out[0, :-200:4999] == 0).all()
    del out
    dx, dg, dinit = gated_scan_bwd(x, x, g, carries)
    close(dx[0, -200:], r["dx"], r["tol_dx"], "dx")
    close(dg[0, -200:], r["dg"], r["tol_dg"], "dg")


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("write", ["plain", "complement", "norm"])
@pytest.mark.parametrize("gate", ["log", "logsigmoid", "bounded"])
def test_step(gate, write, types):
    """A pool: rows in any order, padding and slots out of range; the rest of the pool stays."""
    D, P = 40, 9
    v = make(1, 6, D, types, gate)
    pool0 = torch.randn(P, D, generator=torch.Generator().manual_seed(4))
    slots = [4, -1, 0, P, 8, 2]
    pool = pool0.cuda()
    x, g = v["x"][0].cuda(), v["g"][0].cuda()
    out = gated_scan_step(x, g, pool, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), gate=gate,
                          write=write)
    want = pool0.clone()
    for n, s in enumerate(slots):
        if not 0 <= s < P:
            assert (out[n] == 0).all()
            continue
        r = ref.scan(f64(v["x"])[0, n:n + 1], f64(v["g"])[0, n:n + 1], f64(pool0[s]), gate, -5.0, write)
        close(out[n:n + 1], r["out"], r["tol_out"], "out")
        close(pool[s], r["final"], r["tol_final"], "state")
        want[s] = pool[s].cpu()
    assert torch.equal(pool.cpu(), want)


@pytest.mark.parametrize("N,D", [(1, 8), (1, 2560), (3, 512), (300, 1032)])
def test_step_dense(N, D):
    v = make(1, N, D, "bf16", "logsigmoid")
    state0 = torch.randn(N, D, generator=torch.Generator().manual_seed(4))
    state, out = state0.cuda(), torch.empty(N, D, dtype=torch.bfloat16, device="cuda")
    got = gated_scan_step(v["x"][0].cuda(), v["g"][0].cuda(), state, out=out, gate="logsigmoid", write="norm")
    assert got is out
    for n in range(N):
        r = ref.scan(f64(v["x"])[0, n:n + 1], f64(v["g"])[0, n:n + 1], f64(state0[n]), "logsigmoid", -5.0, "norm")
        close(out[n:n + 1], r["out"], r["tol_out"], "out")
        close(state[n], r["final"], r["tol_final"], "state")


def test_steps_follow_the_scan():
    v = make(3, 40, 16, "f32", "bounded")
    c = cuda(v)
    out, final, _ = gated_scan_fwd(c["x"], c["g"], c["init"], gate="bounded", write="norm")
    state = c["init"].clone()
    steps = [gated_scan_step(c["x"][:, t].contiguous(), c["g"][:, t].contiguous(), state, gate="bounded",
                             write="norm") for t in range(40)]
    for n in range(3):
        r = ref.scan(f64(v["x"])[n], f64(v["g"])[n], f64(v["init"])[n], "bounded", -5.0, "norm")
        close(torch.stack(steps, 1)[n], r["out"], r["tol_out"], "steps")
        close(out[n], r["out"], r["tol_out"], "scan")
    assert torch.equal(torch.stack(steps, 1)[:, -1], state)


def test_captured_and_replayed():
    a, b = cuda(make(1, 700, 24, "bf16", "logsigmoid", seed=1)), cuda(make(1, 700, 24, "bf16", "logsigmoid", seed=2))
    buf = {k: t.clone() for k, t in a.items()}
    state = a["init"].clone()
    how = dict(gate="logsigmoid", write="complement")

    def calls(v, state):
        out, final, carries = gated_scan_fwd(v["x"], v["g"], v["init"], save_carries=True, **how)
        grads = gated_scan_bwd(v["dout"], v["x"], v["g"], carries, dfinal_state=v["dfinal"], **how)
        return (out, final) + grads + (gated_scan_step(v["x"][0, :1], v["g"][0, :1], state, **how),)

    calls(buf, state.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(buf, state)
    for v in (a, b, a):
        for k in buf:
            buf[k].copy_(v[k])
        state.copy_(v["init"])
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        eager = v["init"].clone()
        assert all(torch.equal(x, y) for x, y in zip(kept, calls(v, eager)))
        assert torch.equal(state, eager)


def test_refusals():
    x = torch.zeros(2, 8, 8, device="cuda")
    g = torch.zeros_like(x)
    i32 = dict(dtype=torch.int32, device="cuda")
    for bad in (dict(g=g[:, :4]), dict(g=g.double()), dict(g=g[..., :4]), dict(init_state=g[0]),
                dict(init_state=torch.zeros(2, 8, device="cuda").half()), dict(out=g.bfloat16()), dict(out=g[:1]),
                dict(final_state=torch.zeros(3, 8, device="cuda")), dict(carries=torch.zeros(1, 8, device="cuda")),
                dict(cu_seqlens=torch.zeros(3, **i32)), dict(cu_seqlens=torch.zeros(3, device="cuda")),
                dict(gate="tanh"), dict(write="sum"), dict(x=x.transpose(0, 1)), dict(x=x.half()), dict(x=x[0, 0]),
                dict(init_state=torch.zeros(2, 8)), dict(g=g.cpu())):
        with pytest.raises((ValueError, TypeError)):
            gated_scan_fwd(**{**dict(x=x, g=g), **bad})
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        gated_scan_fwd(x[..., :6].contiguous(), x[..., :6].contiguous())
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        gated_scan_fwd(x, g.bfloat16())
    with pytest.raises(RuntimeError, match="INVALID"):
        gated_scan_fwd(x, g, gate="bounded", gate_lower=1.0)
    carries = torch.zeros(2, 8, device="cuda")  # 2 x 8 tokens: 16 // 64 + 2 rows
    for bad in (dict(dout=x.bfloat16()), dict(dout=None), dict(carries=carries[:1]), dict(carries=None),
                dict(dx=x[:1]), dict(dg=g.bfloat16()), dict(dfinal_state=carries[0]), dict(dinit_state=x)):
        with pytest.raises((ValueError, TypeError)):
            gated_scan_bwd(**{**dict(dout=x, x=x, g=g, carries=carries), **bad})
    s = torch.zeros(2, 8, device="cuda")
    for bad in (dict(state=s[:1]), dict(state=s.bfloat16()), dict(slots=torch.zeros(3, **i32)),
                dict(slots=torch.zeros(2, device="cuda")), dict(g=s[:, :4]), dict(out=s.bfloat16()),
                dict(state=torch.zeros(2, 4, 2, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            gated_scan_step(**{**dict(x=s, g=s, state=s.clone()), **bad})
