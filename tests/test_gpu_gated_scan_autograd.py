"""The README's autograd function of the gated scan, as it stands there: it runs, and its gradients
are the 64-bit reference's."""
import os
import re

import numpy as np
import pytest
import torch

import kimi_delta_attention_17_gb300 as kda
from kimi_delta_attention_17_gb300 import build
from tests import scan_reference as ref
from tests.test_gpu_gated_scan import close, cuda, f64, make

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.fixture(scope="module")
def function():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    blocks = re.findall(r"```python\n(class GatedScan.*?)```", open(README, encoding="utf-8").read(), flags=re.S)
    assert len(blocks) == 1
    names = dict(torch=torch, gated_scan_fwd=kda.gated_scan_fwd, gated_scan_bwd=kda.gated_scan_bwd)
    exec(blocks[0], names)
    return names["GatedScan"]


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 30, 30, 200], [5, 90, 180]])
def test_gradients(function, cu, init):
    T, D, N = 200, 24, 1 if cu is None else len(cu) - 1
    v = make(1, T, D, "f32", "logsigmoid", N=N, init=init)
    c = cuda(v)
    leaves = {k: c[k].requires_grad_() for k in ("x", "g", "init") if c[k] is not None}
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    h, last = function.apply(c["x"], c["g"], c["init"], cut)
    loss = (h * c["dout"]).sum() + ((last * c["dfinal"]).sum() if init else 0.0)
    got = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    x, g, do = (f64(v[n])[0] for n in ("x", "g", "dout"))
    spans = ref.spans(1, T, cu)
    for n, (lo, hi) in enumerate(spans):
        r = ref.scan(x[lo:hi], g[lo:hi], f64(v["init"])[n] if init else None, "logsigmoid", -5.0, "norm", do[lo:hi],
                     f64(v["dfinal"])[n] if init else None)
        close(h[0, lo:hi], r["out"], r["tol_out"], "out")
        close(got["x"][0, lo:hi], r["dx"], r["tol_dx"], "dx")
        close(got["g"][0, lo:hi], r["dg"], r["tol_dg"], "dg")
        if init:
            close(got["init"][n], r["dinit"], r["tol_dinit"], "dinit")
    inside = np.zeros(T, bool)
    for lo, hi in spans:
        inside[lo:hi] = True
    for t in (h, got["x"], got["g"]):
        assert not t[0].detach().cpu().numpy()[~inside].any()


def test_calls_without_it_build_no_graph(function):
    c = cuda(make(1, 8, 8, "f32"))
    c["x"].requires_grad_()
    out, final, carries = kda.gated_scan_fwd(c["x"], c["g"], save_carries=True)
    assert not out.requires_grad and not final.requires_grad and not carries.requires_grad
