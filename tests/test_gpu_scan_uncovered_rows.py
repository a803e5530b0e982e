"""Tokens that no packed sequence covers: zeros in what the call allocates, untouched in what the
caller gives. Fresh memory is made NaN here, so that a row left as it was shows."""
import pytest
import torch

from kimi_delta_attention_17_gb300 import build, gated_scan_bwd, gated_scan_fwd
from tests.test_gpu_gated_scan import TYPES, cuda, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


@pytest.fixture
def nan_memory(monkeypatch):
    """torch.empty and torch.empty_like give memory full of NaN."""
    for name in ("empty", "empty_like"):
        plain = getattr(torch, name)

        def filled(*a, plain=plain, **kw):
            t = plain(*a, **kw)
            return t.fill_(float("nan")) if t.is_floating_point() else t
        monkeypatch.setattr(torch, name, filled)


def offsets(cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


CUTS = [(300, [7, 150, 260]), (300, [0, 150, 260]), (300, [7, 150, 300]), (300, [0, 0, 0]), (300, [300, 300, 300]),
        (300, [40, 40, 40]), (1, [0, 0, 0]), (1, [0, 1, 1]), (4000, [1, 3, 3998]), (4000, [1500, 1500, 1501]),
        (2500, [0] + list(range(100, 2301, 11)))]


@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("T,cu", CUTS)
def test_zeros_where_the_call_allocates(T, cu, types, nan_memory):
    D, N = 136, len(cu) - 1
    c = cuda(make(1, T, D, types, "logsigmoid", seed=T + len(cu), N=N))
    cut, how = offsets(cu), dict(gate="logsigmoid", write="norm")
    out, final, carries = gated_scan_fwd(c["x"], c["g"], c["init"], cut, save_carries=True, **how)
    dx, dg, dinit = gated_scan_bwd(c["dout"], c["x"], c["g"], carries, cut, dfinal_state=c["dfinal"], **how)
    for t in (out, dx, dg):
        assert not t[0, :cu[0]].any() and not t[0, cu[-1]:].any()
    # Every sequence as if the others and the padding were not there, given buffers included.
    given = [torch.full_like(t, 3.0) for t in (c["x"], c["x"], c["g"])]
    fwd2 = gated_scan_fwd(c["x"], c["g"], c["init"], cut, out=given[0], carries=carries.clone(), **how)
    bwd2 = gated_scan_bwd(c["dout"], c["x"], c["g"], carries, cut, dfinal_state=c["dfinal"], dx=given[1],
                          dg=given[2], **how)
    for t, kept in zip((out, dx, dg), given):
        assert torch.equal(t[0, cu[0]:cu[-1]], kept[0, cu[0]:cu[-1]]) and not torch.isnan(t).any()
        assert (kept[0, :cu[0]] == 3).all() and (kept[0, cu[-1]:] == 3).all()
    assert torch.equal(final, fwd2[1]) and torch.equal(dinit, bwd2[2])
    assert not torch.isnan(final).any() and not torch.isnan(dinit).any()


@pytest.mark.parametrize("given", ["dx", "dg"])
def test_one_gradient_given(given, nan_memory):
    c = cuda(make(1, 300, 16, "mixed", N=2))
    cut = offsets([7, 150, 260])
    _, _, carries = gated_scan_fwd(c["x"], c["g"], c["init"], cut, save_carries=True)
    buffer = torch.full_like(c["x" if given == "dx" else "g"], 3.0)
    dx, dg, _ = gated_scan_bwd(c["dout"], c["x"], c["g"], carries, cut, **{given: buffer})
    fresh = dg if given == "dx" else dx
    assert (dx if given == "dx" else dg) is buffer
    assert not fresh[0, :7].any() and not fresh[0, 260:].any() and not torch.isnan(fresh).any()
    assert (buffer[0, :7] == 3).all() and (buffer[0, 260:] == 3).all()


def test_offsets_that_do_not_fit_with_fresh_outputs():
    """Offsets past the tokens, below zero or falling: values are unspecified, the calls end, and
    memory beside the outputs is not touched (the outputs are views within larger buffers)."""
    T, D = 70, 16
    c = cuda(make(1, T, D, "f32", N=4))
    for cu in ([-5, 30, 10, 2 ** 31 - 1, 60], [60, 10, 90, -3, 5], [-9, -8, -7, -6, -5], [71, 80, 90, 99, 2 ** 31 - 1]):
        cut = offsets(cu)
        out, final, carries = gated_scan_fwd(c["x"], c["g"], c["init"], cut, save_carries=True)
        dx, dg, dinit = gated_scan_bwd(c["dout"], c["x"], c["g"], carries, cut, dfinal_state=c["dfinal"])
        torch.cuda.synchronize()
        assert out.shape == dx.shape == dg.shape == c["x"].shape and final.shape == dinit.shape


def test_captured_with_other_offsets(nan_memory):
    """A replay on offsets that cover less zeroes what it does not cover."""
    c = cuda(make(1, 500, 24, "bf16", N=2))
    cut = offsets([0, 200, 500])

    def calls():
        out, _, carries = gated_scan_fwd(c["x"], c["g"], c["init"], cut, save_carries=True)
        return (out,) + gated_scan_bwd(c["dout"], c["x"], c["g"], carries, cut)[:2]

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for cu in ([0, 200, 500], [30, 100, 450], [0, 1, 2]):
        cut.copy_(offsets(cu))
        graph.replay()
        torch.cuda.synchronize()
        for t, want in zip(got, calls()):
            assert torch.equal(t, want)
            assert not t[0, :cu[0]].any() and not t[0, cu[2]:].any()
