"""Channels that remember thousands of tokens: every gate, both directions, and thousands of
single steps. A rounding of the decay that leans to one side adds up here; one that does not
walks away from the value no faster than the square root of the tokens.

The bounds. With u = 2^-24 and decays of a ~ 0.9999 a token is remembered over at most 10^4 others.
Roundings of at most u each way per token, which do not lean, come to a walk of 100 u of the size
of what is computed; the factors formed per element (w, and a itself) add 24 u, and the 21 maps
that are composed on the way to a token, two roundings each, 42 u once: 166 u, below 1e-5. dg
is the product of e and h, with 64 u of its own: 396 u, below 2.4e-5. Steps compose nothing and are
held to the same 1e-5. (In fp32 on the host, logits of 9 to 9.5 and 6000 tokens: the product of
rounded decays over four tokens is off by 317 u in the outputs and 458 u in the last state, 1 - A
carried beside it by 10 u and 15 u.)
"""
import numpy as np
import pytest
import torch

from kimi_delta_attention_17_gb300 import build, gated_scan_bwd, gated_scan_fwd, gated_scan_step
from tests import scan_reference as ref
from tests.test_gpu_gated_scan import cuda, f64, make

pytestmark = pytest.mark.gpu

T, VALUES, GRADIENT = 6000, 1e-5, 2.4e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def slow_gates(shape, gate, seed):
    """1 - a between 0 and 2e-4 ("log"), of 0.75e-4 to 1.23e-4 ("logsigmoid") and of 0.6e-4 to 1.7e-4
    ("bounded", log a = -5 sigmoid)."""
    r = torch.rand(shape, generator=torch.Generator().manual_seed(seed))
    return {"log": -2e-4 * r, "logsigmoid": 9 + 0.5 * r, "bounded": -11.3 + r}[gate]


def off(got, want):
    return np.linalg.norm(f64(got) - want) / np.linalg.norm(want)


@pytest.mark.parametrize("write", ["plain", "complement", "norm"])
@pytest.mark.parametrize("gate", ["log", "logsigmoid", "bounded"])
def test_scan_and_gradient(gate, write):
    v = make(1, T, 32, "f32", seed=2)
    v["g"] = slow_gates((1, T, 32), gate, 3)
    c = cuda(v)
    how = dict(gate=gate, write=write)
    out, final, carries = gated_scan_fwd(c["x"], c["g"], c["init"], save_carries=True, **how)
    dx, dg, dinit = gated_scan_bwd(c["dout"], c["x"], c["g"], carries, dfinal_state=c["dfinal"], **how)
    r = ref.scan(f64(v["x"])[0], f64(v["g"])[0], f64(v["init"])[0], gate, -5.0, write, f64(v["dout"])[0],
                 f64(v["dfinal"])[0])
    for got, name, bound in ((out[0], "out", VALUES), (final[0], "final", VALUES), (dx[0], "dx", VALUES),
                             (dinit[0], "dinit", VALUES), (dg[0], "dg", GRADIENT)):
        assert off(got, r[name]) <= bound, name


@pytest.mark.parametrize("slots", [False, True])
@pytest.mark.parametrize("write", ["plain", "complement", "norm"])
@pytest.mark.parametrize("gate", ["log", "logsigmoid", "bounded"])
def test_thousands_of_steps(gate, write, slots):
    N, D = 4, 32
    v = make(1, T * N, D, "f32", seed=4, N=N)
    x, g = v["x"].view(T, N, D), slow_gates((T, N, D), gate, 5)
    state, rows = v["init"].cuda(), None
    if slots:
        rows = torch.tensor([5, 0, 3, 2], dtype=torch.int32, device="cuda")
        pool = torch.zeros(7, D, device="cuda")
        pool[rows.long()] = state
        state = pool
    xc, gc, out = x.cuda(), g.cuda(), torch.empty(T, N, D, device="cuda")
    for t in range(T):
        gated_scan_step(xc[t], gc[t], state, slots=rows, out=out[t], gate=gate, write=write)
    if slots:
        state = state[rows.long()]
    r = ref.scan(f64(x).reshape(T, N * D), f64(g).reshape(T, N * D), f64(v["init"]).reshape(N * D), gate, -5.0, write)
    assert off(out.view(T, N * D), r["out"]) <= VALUES
    assert off(state.reshape(N * D), r["final"]) <= VALUES
