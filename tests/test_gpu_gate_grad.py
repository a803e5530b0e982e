"""The gradient of the output gate + RMS norm against the 64-bit definition, and of the forward call."""
import numpy as np
import pytest
import torch

from kimi_delta_attention_17_gb300 import build, output_gate_rmsnorm, output_gate_rmsnorm_bwd
from tests import layer_reference as ref
from tests.layer_reference import f64, half_step

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def inputs(shape, dtype, seed=0, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    o, z, dout = (torch.randn(shape, generator=gen).mul(s).to(dtype).cuda() for s in (1.0, spread, 1.0))
    return dout, o, z, (1 + 0.3 * torch.randn(shape[-1], generator=gen)).cuda()


def check(dout, o, z, w, got):
    dv = o.shape[-1]
    rows = [f64(t).reshape(-1, dv) for t in (dout, o, z)]
    r = ref.gate_grad(*rows, None if w is None else f64(w), EPS)
    bf16 = o.dtype == torch.bfloat16
    for name, t, b in (("do", got[0], bf16), ("dz", got[1], bf16), ("dw", got[2], False)):
        if t is None:
            assert name == "dw" and w is None
            continue
        want = r[name]
        off = np.abs(f64(t).reshape(want.shape) - want) / (r["tol_" + name] + half_step(want, b))
        assert off.max() <= 1.0, "%s: %.3g times its bound" % (name, off.max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("lead", [(1, 1), (7, 3), (2, 5, 4), (5, 51), (1, 257), (77, 32), (20011, 1)])
def test_gradient(lead, dv, dtype):
    for weighted in (True, False):
        dout, o, z, w = inputs(lead + (dv,), dtype, seed=dv)
        w = w if weighted else None
        check(dout, o, z, w, output_gate_rmsnorm_bwd(dout, o, z, w, EPS))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wide_logits_and_rows_of_zeros(dtype):
    dout, o, z, w = inputs((64, 4, 128), dtype, spread=30.0)
    z[0, 0, :4] = torch.tensor([-1000.0, 1000.0, -85.0, 85.0])
    o[3] = 0.0
    dout[5] = 0.0
    got = output_gate_rmsnorm_bwd(dout, o, z, w, EPS)
    check(dout, o, z, w, got)
    assert not got[0][5].any() and not got[1][3].any() and got[1][0, 0, 1] == 0


def test_what_is_not_finite_stays_in_its_row():
    dout, o, z, w = inputs((8, 2, 64), torch.float32)
    clean = output_gate_rmsnorm_bwd(dout, o, z, None, EPS)
    o[2, 1, 3] = float("nan")
    z[4, 0, 5] = float("nan")
    do, dz, _ = output_gate_rmsnorm_bwd(dout, o, z, None, EPS)
    assert torch.isnan(do[2, 1]).all() and torch.isnan(dz[2, 1]).all() and torch.isnan(do[4, 0]).all()
    assert torch.isnan(dz[4, 0, 5]) and torch.isfinite(dz[4, 0, 6:]).all()
    keep = torch.ones(8, 2, dtype=torch.bool)
    keep[2, 1] = keep[4, 0] = False
    assert torch.equal(do[keep], clean[0][keep]) and torch.equal(dz[keep], clean[1][keep])


def test_differences_of_the_forward_call():
    """Along a direction, the forward call's own outputs in fp32: central differences at h = 2^-6, off by the
    third derivative (measured against the 64-bit difference at the same h, whose own error is 2^-52 / h) and
    by the outputs' rounding: 24 u of sum |y dout| over h."""
    dout, o, z, w = inputs((9, 3, 64), torch.float32)
    do, dz, dw = output_gate_rmsnorm_bwd(dout, o, z, w, EPS)
    h = 2.0 ** -6
    gen = torch.Generator().manual_seed(8)
    for i, (t, g) in enumerate(((o, do), (z, dz), (w, dw))):
        d = torch.randn(t.shape, generator=gen).cuda()

        def along(step, call, cast):
            args = [cast(a) for a in (o, z, w)]
            args[i] = cast(t + step * d)
            return call(*args, EPS)
        y = [along(s, output_gate_rmsnorm, lambda a: a) for s in (h, -h)]
        got = ((y[0].double() - y[1].double()) * dout.double()).sum().item() / (2 * h)
        y64 = [along(s, ref.gate, f64) for s in (h, -h)]
        curved = ((y64[0] - y64[1]) * f64(dout)).sum() / (2 * h)
        exact = (f64(g) * f64(d)).sum()
        bound = 24 * ref.U * (np.abs(y64[0]) * np.abs(f64(dout))).sum() / h
        assert abs(got - curved) <= bound
        assert abs(curved - exact) <= 0.02 * abs(exact) + 0.02 * np.linalg.norm(f64(g)) * np.linalg.norm(f64(d))


@pytest.mark.parametrize("which", ["dout", "o", "z"])
def test_in_place(which):
    dout, o, z, w = inputs((50, 3, 128), torch.bfloat16)
    want = output_gate_rmsnorm_bwd(dout, o, z, w, EPS)
    for name in ("do", "dz"):
        t = {"dout": dout.clone(), "o": o.clone(), "z": z.clone()}
        got = output_gate_rmsnorm_bwd(t["dout"], t["o"], t["z"], w, EPS, **{name: t[which]})
        assert got[name == "dz"] is t[which] and all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_tokens_streams_and_graphs():
    dout, o, z, w = inputs((0, 3, 64), torch.bfloat16)
    do, dz, dw = output_gate_rmsnorm_bwd(dout, o, z, w, EPS, dweight=torch.full_like(w, 3.0))
    assert do.shape == (0, 3, 64) and dz.shape == (0, 3, 64) and not dw.any()
    dout, o, z, w = inputs((999, 8, 128), torch.bfloat16)
    want = output_gate_rmsnorm_bwd(dout, o, z, w, EPS)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(output_gate_rmsnorm_bwd(dout, o, z, w, EPS))
    got.append(output_gate_rmsnorm_bwd(dout, o, z, w, EPS, stream=streams[1]))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got.append(output_gate_rmsnorm_bwd(dout, o, z, w, EPS))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals():
    dout, o, z, w = inputs((4, 2, 64), torch.bfloat16)
    with pytest.raises(RuntimeError):
        output_gate_rmsnorm_bwd(dout, o, z, w, do=o, dz=o)
    for call in (lambda: output_gate_rmsnorm_bwd(dout, o, z.float(), w), lambda: output_gate_rmsnorm_bwd(dout[:2], o, z, w),
                 lambda: output_gate_rmsnorm_bwd(dout, o, z, w[:32]), lambda: output_gate_rmsnorm_bwd(dout, o, z, dweight=w),
                 lambda: output_gate_rmsnorm_bwd(dout, o, z, w, dz=z[:1]), lambda: output_gate_rmsnorm_bwd(w, w, w, w),
                 lambda: output_gate_rmsnorm_bwd(dout.half(), o.half(), z.half())):
        with pytest.raises(ValueError):
            call()
