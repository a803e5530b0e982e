"""The row norm, its 8-bit form and its gradient against the 64-bit definitions."""
import numpy as np
import pytest
import torch

from kimi_delta_attention_17_gb300 import _lib, build, rmsnorm_bwd, rmsnorm_fwd, rmsnorm_quant
from tests import layer_reference as ref
from tests.layer_reference import f64, half_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
TYPES = [(BF, None), (BF, BF), (BF, F), (F, None), (F, F)]
# Widths around every change of the threads and groups that a row takes, up to the most.
WIDTHS = [8, 64, 72, 128, 136, 248, 264, 512, 520, 1024, 1032, 1288, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392,
          32760, 32768]
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def inputs(rows, D, dtype, rdtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, D, generator=gen).to(dtype).cuda()
    res = None if rdtype is None else (3 * torch.randn(rows, D, generator=gen)).to(rdtype).cuda()
    w = (1 + 0.3 * torch.randn(D, generator=gen)).cuda()
    return x, res, w


def stored_sum(x, res):
    """h as it is stored: the fp32 sum, rounded to the residual's type."""
    return x if res is None else (x.float() + res.float()).to(res.dtype)


def close(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    worst = (np.abs(got - want) / np.maximum(tol, 1e-300)).max() if got.size else 0.0
    assert worst <= 1.0, "%s: %.3g times its bound" % (what, worst)


def check_fwd(x, res, w, **kw):
    y, h, rstd = rmsnorm_fwd(x, w, EPS, residual=res, save_rstd=True, **kw)
    want_h = stored_sum(x, res)
    assert h.dtype == want_h.dtype and torch.equal(h, want_h)
    r = ref.norm(f64(want_h), None if w is None else f64(w), EPS)
    close(y, r["y"], r["tol_y"] + half_step(r["y"], y.dtype == BF), "y")
    close(rstd, r["rstd"], r["tol_rstd"] + half_step(r["rstd"], False), "rstd")
    return y, h, rstd


@pytest.mark.parametrize("dtype,rdtype", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_forward(D, dtype, rdtype):
    for rows in (1, 5, 77) if D <= 4104 else (3,):
        x, res, w = inputs(rows, D, dtype, rdtype, seed=rows)
        check_fwd(x, res, w if rows != 5 else None)


@pytest.mark.parametrize("per", ["row", "block"])
@pytest.mark.parametrize("dtype,rdtype", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_eight_bits(D, dtype, rdtype, per):
    rows = 33 if D <= 4104 else 3
    x, res, w = inputs(rows, D, dtype, rdtype)
    q, scales, h = rmsnorm_quant(x, w, EPS, residual=res, scale_per=per)
    assert q.dtype == torch.float8_e4m3fn and torch.equal(h, stored_sum(x, res))
    y = ref.norm(f64(h), f64(w), EPS)["y"]
    size = D if per == "row" else 128
    top = ref.blocks_top(y, size)
    # 30 u of y, the rounded constant and the product.
    close(scales, top / 448, 34 * ref.U * top / 448, "scales")
    s = np.repeat(f64(scales), size, 1)[:, :D]
    codes = f64(q.float())
    # Half a step of e4m3 (2^-4 of the value, 2^-10 below 2^-6) and the 40 u of y, the factor and the product.
    close(torch.from_numpy(codes * s), y, np.maximum(ref.E4M3 * np.abs(y), 2.0 ** -10 * s) * (1 + 2.0 ** -10)
          + 40 * ref.U * np.abs(y), "q * scale")
    blocks = torch.from_numpy(ref.blocks_top(codes, size))
    assert (blocks == 448).all()


@pytest.mark.parametrize("dtype,rdtype", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_gradient(D, dtype, rdtype):
    for rows in (1, 77) if D <= 4104 else (5,):
        x, res, w = inputs(rows, D, dtype, rdtype, seed=rows)
        if rows == 1:
            w = None
        gen = torch.Generator().manual_seed(9)
        dy = torch.randn(rows, D, generator=gen).to(dtype).cuda()
        _, h, rstd = rmsnorm_fwd(x, w, EPS, residual=res, save_rstd=True)
        dh = torch.randn(rows, D, generator=gen).to(h.dtype).cuda() if res is not None or rows == 1 else None
        dx, dres, dw = rmsnorm_bwd(dy, h, rstd, w, dh=dh)
        r = ref.norm_grad(f64(dy), f64(h), None if w is None else f64(w), EPS, None if dh is None else f64(dh))
        close(dx, r["dx"], r["tol_dx"] + half_step(r["dx"], dtype == BF), "dx")
        if h.dtype == dtype:
            assert dres is dx
        else:
            assert dres.dtype == F
            close(dres, r["dx"], r["tol_dx"] + half_step(r["dx"], False), "dresidual")
        if w is None:
            assert dw is None
        else:
            close(dw, r["dw"], r["tol_dw"] + half_step(r["dw"], False), "dweight")


@pytest.mark.parametrize("D", [64, 1024, 4096])
def test_gradient_of_many_rows(D):
    """More rows than the CTAs take at once, an odd number of them."""
    rows = 20011 if D < 4096 else 2011
    x, res, w = inputs(rows, D, BF, F)
    dy = torch.randn(rows, D, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
    _, h, rstd = rmsnorm_fwd(x, w, EPS, residual=res, save_rstd=True)
    dx, dres, dw = rmsnorm_bwd(dy, h, rstd, w)
    r = ref.norm_grad(f64(dy), f64(h), f64(w), EPS)
    close(dx, r["dx"], r["tol_dx"] + half_step(r["dx"], True), "dx")
    close(dres, r["dx"], r["tol_dx"] + half_step(r["dx"], False), "dresidual")
    close(dw, r["dw"], r["tol_dw"] + half_step(r["dw"], False), "dweight")
    again = rmsnorm_bwd(dy, h, rstd, w)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dres, dw)))


@pytest.mark.parametrize("dtype,rdtype", [(BF, None), (BF, BF), (BF, F), (F, F)])
@pytest.mark.parametrize("D", [8200, 10240, 12280, 12288, 12296])
def test_gradient_of_wide_rows(D, dtype, rdtype):
    """Several rows a CTA at the widths where a thread takes three groups and where it no longer does, also in place."""
    rows = 317
    x, res, w = inputs(rows, D, dtype, rdtype)
    gen = torch.Generator().manual_seed(6)
    dy = torch.randn(rows, D, generator=gen).to(dtype).cuda()
    _, h, rstd = rmsnorm_fwd(x, w, EPS, residual=res, save_rstd=True)
    dh = None if res is None else torch.randn(rows, D, generator=gen).to(h.dtype).cuda()
    dx, dres, dw = rmsnorm_bwd(dy, h, rstd, w, dh=dh)
    r = ref.norm_grad(f64(dy), f64(h), f64(w), EPS, None if dh is None else f64(dh))
    close(dx, r["dx"], r["tol_dx"] + half_step(r["dx"], dtype == BF), "dx")
    close(dres, r["dx"], r["tol_dx"] + half_step(r["dx"], h.dtype == BF), "dresidual")
    close(dw, r["dw"], r["tol_dw"] + half_step(r["dw"], False), "dweight")
    kw = {} if dh is None or h.dtype == dtype else {"dresidual": dh}
    got = rmsnorm_bwd(dy, h, rstd, w, dh=dh, dx=dy, **kw)
    assert got[0] is dy and all(torch.equal(a, b) for a, b in zip(got, (dx, dres, dw)))


@pytest.mark.parametrize("D", [128, 1288, 16384])
@pytest.mark.parametrize("dtype,rdtype", [(BF, BF), (BF, F), (F, F)])
def test_in_place(dtype, rdtype, D):
    x, res, w = inputs(50, D, dtype, rdtype)
    y, h, rstd = rmsnorm_fwd(x, w, EPS, residual=res, save_rstd=True)
    at = res.clone()
    y2, h2, _ = rmsnorm_fwd(x, w, EPS, residual=at, residual_out=at)
    assert h2 is at and torch.equal(at, h) and torch.equal(y2, y)
    at = res.clone()
    q, s, _ = rmsnorm_quant(x, w, EPS, residual=res)
    q2, s2, h2 = rmsnorm_quant(x, w, EPS, residual=at, residual_out=at)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s) and torch.equal(h2, h)
    dy, dh = torch.randn_like(x), torch.randn_like(res)
    want = rmsnorm_bwd(dy, h, rstd, w, dh=dh)
    if rdtype == dtype:
        kept = dh.clone()
        assert all(torch.equal(a, b) for a, b in zip(rmsnorm_bwd(dy, h, rstd, w, dh=kept, dx=kept), want))
        got = rmsnorm_bwd(dy, h, rstd, w, dh=dh, dx=dy)
    else:
        got = rmsnorm_bwd(dy, h, rstd, w, dh=dh, dx=dy, dresidual=dh)
        assert got[1] is dh
    assert got[0] is dy and all(torch.equal(a, b) for a, b in zip(got, want))


def test_leading_dimensions_and_no_rows():
    x, res, w = inputs(30, 128, BF, BF)
    y, h, rstd = rmsnorm_fwd(x, w, EPS, residual=res, save_rstd=True)
    y3, h3, rstd3 = rmsnorm_fwd(x.view(2, 3, 5, 128), w, EPS, residual=res.view(2, 3, 5, 128), save_rstd=True)
    assert rstd3.shape == (2, 3, 5) and torch.equal(y3.view(30, 128), y) and torch.equal(h3.view(30, 128), h)
    y1, _, r1 = rmsnorm_fwd(x[4], w, EPS, residual=res[4], save_rstd=True)
    assert r1.shape == () and torch.equal(y1, y[4]) and torch.equal(r1, rstd[4])
    q, s, _ = rmsnorm_quant(x.view(2, 15, 128), w, EPS, scale_per="row")
    assert s.shape == (2, 15, 1)
    none = x[:0]
    y0, _, r0 = rmsnorm_fwd(none, w, EPS, save_rstd=True)
    assert y0.shape == (0, 128) and r0.shape == (0,)
    dx, _, dw = rmsnorm_bwd(none, none, r0, w, dweight=torch.full_like(w, 7.0))
    assert dx.shape == (0, 128) and not dw.any()
    assert rmsnorm_quant(none, w)[1].shape == (0, 1)


@pytest.mark.parametrize("per", ["row", "block"])
def test_rows_of_zeros_and_of_what_is_not_finite(per):
    x, _, w = inputs(6, 512, F, None)
    x[1] = 0.0
    x[2, 300] = float("nan")
    x[3, 10] = float("inf")
    x[4] = 0.0
    x[4, 200] = 1e-3
    y, _, rstd = rmsnorm_fwd(x, w, EPS, save_rstd=True)
    q, s, _ = rmsnorm_quant(x, w, EPS, scale_per=per)
    codes = q.float()
    clean, _, _ = rmsnorm_fwd(x[:1], w, EPS)
    assert torch.equal(y[0], clean[0]) and torch.isfinite(y[5]).all()          # rows do not touch one another
    assert not y[1].any() and not codes[1].any() and not s[1].any()            # zeros: scale 0
    assert torch.isnan(y[2]).all() and torch.isnan(s[2]).all() and torch.isnan(codes[2]).all()
    assert torch.isnan(y[3, 10]) and not y[3, 11:].any() and rstd[3] == 0      # x / inf = 0, inf / inf = NaN
    at = torch.isnan(s[3])
    assert at[0] and at.sum() == 1
    assert codes[4, 200] == 448 and (codes[4] != 0).sum() == 1
    if per == "block":
        assert (s[4] > 0).tolist() == [False, True, False, False]


def test_offsets_past_32_bits():
    """70000 rows of 32768 bf16 values: rows past 2^31 values."""
    rows, D = 70000, 32768
    x = torch.zeros(rows, D, dtype=BF, device="cuda")
    tail, res, w = inputs(3, D, BF, BF, seed=4)
    x[-3:] = tail
    y, h, rstd = rmsnorm_fwd(x, w, EPS, residual=x, save_rstd=True)
    one = rmsnorm_fwd(tail, w, EPS, residual=tail, save_rstd=True)
    assert torch.equal(y[-3:], one[0]) and torch.equal(h[-3:], one[1]) and torch.equal(rstd[-3:], one[2])
    del y
    q, s, _ = rmsnorm_quant(x, w, EPS, residual=x, residual_out=x)  # x + x in place, as h is
    assert torch.equal(x[-3:], one[1])
    q1, s1, _ = rmsnorm_quant(tail, w, EPS, residual=tail)
    assert torch.equal(q[-3:].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[-3:], s1)
    del q
    h[:-3] = 0
    dx, _, dw = rmsnorm_bwd(x, h, rstd, w)
    dx1, _, _ = rmsnorm_bwd(x[-3:], h[-3:], rstd[-3:], w)
    assert torch.equal(dx[-3:], dx1) and torch.isfinite(dw).all()


def test_streams_and_graphs():
    x, res, w = inputs(300, 2048, BF, BF)
    dy = torch.randn_like(x)

    def step(stream=None):
        y, h, rstd = rmsnorm_fwd(x, w, EPS, residual=res, save_rstd=True, stream=stream)
        q, s, _ = rmsnorm_quant(x, w, EPS, residual=res, stream=stream)
        return (y, h, q.view(torch.uint8), s) + rmsnorm_bwd(dy, h, rstd, w, stream=stream)
    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in streams:  # two at once, each with its own workspace
        with torch.cuda.stream(s):
            got.append(step())
    got.append(step(stream=streams[0]))
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    x.mul_(-1)
    res.mul_(-1)
    for g, _ in graphs:
        g.replay()
    x.mul_(-1)
    res.mul_(-1)
    for g, out in graphs:
        g.replay()
        got.append(out)
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals():
    x, res, w = inputs(4, 64, BF, F)
    _, h, rstd = rmsnorm_fwd(x, w, EPS, residual=res, save_rstd=True)
    bad = [lambda: rmsnorm_fwd(x.half(), w), lambda: rmsnorm_fwd(x, w[:32]), lambda: rmsnorm_fwd(x, w.bfloat16()),
           lambda: rmsnorm_fwd(x.float(), w, residual=x), lambda: rmsnorm_fwd(x, w, residual=res[:3]),
           lambda: rmsnorm_fwd(x, w, residual_out=res), lambda: rmsnorm_fwd(x, w, residual=res, residual_out=x),
           lambda: rmsnorm_fwd(x.t(), w), lambda: rmsnorm_fwd(x, w, out=h), lambda: rmsnorm_quant(x, w, scale_per="tensor"),
           lambda: rmsnorm_quant(x, w, out=x), lambda: rmsnorm_quant(x, w, scales=rstd),
           lambda: rmsnorm_bwd(x, h[:2], rstd, w), lambda: rmsnorm_bwd(x, h, rstd[:2], w),
           lambda: rmsnorm_bwd(x.float(), x, rstd, w), lambda: rmsnorm_bwd(x, h, rstd, w, dh=x),
           lambda: rmsnorm_bwd(x, h, rstd, dweight=w), lambda: rmsnorm_bwd(x, x, rstd, w, dresidual=x),
           lambda: rmsnorm_bwd(x, h, rstd, w, dweight=w[:8]), lambda: rmsnorm_fwd(x[:, :0])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for kw in (dict(out=x), dict(residual=x, out=x), dict(residual=x, residual_out=h.to(BF), out=x)):
        with pytest.raises(_lib.KdaError):
            rmsnorm_fwd(x, w, **kw)
    for D, eps in ((60, EPS), (32776, EPS), (64, 0.0)):
        with pytest.raises(_lib.KdaError):
            rmsnorm_fwd(torch.zeros(2, D, device="cuda"), None, eps)
