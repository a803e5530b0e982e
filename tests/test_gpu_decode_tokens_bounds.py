"""The decode over several tokens within the bounds of its computation in blocks, and beside the single steps."""
import numpy as np
import pytest
import torch

from kimi_delta_attention_17_gb300 import build, decode_step, decode_tokens
from tests import layer_reference, token_blocks_reference as ref
from tests.layer_reference import f64, half_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def inputs(N, K, H, d, dtype, decay, gate, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k, v, z = n(N, K, H, d), n(N, K, H, d), n(N, K, H, d), n(*((N, K, H, d) if decay == "channel" else (N, K, H)))
    q, k = (torch.nn.functional.normalize(t, dim=-1) for t in (q, k))
    g = -torch.nn.functional.softplus(z - 3.0) if gate == "log" else z + 3.0 if gate == "logsigmoid" else z - 2.0
    return [t.cuda() for t in (q.to(dtype), k.to(dtype), v.to(dtype), g, torch.sigmoid(n(N, K, H)), 0.3 * n(N, H, d, d))]


def heads(args, decay, gate):
    """Every row and head in 64 bits: (n, h, q, k, v, a, its error, beta, state)."""
    q, k, v, g, beta, S = (f64(t) for t in args)
    N, K, H, d = q.shape
    for n in range(N):
        for h in range(H):
            z = np.broadcast_to(g[n, :, h].reshape(K, -1), (K, d))
            kind = "none" if decay == "none" else gate
            a = np.ones((K, d)) if decay == "none" else layer_reference.decay(z, gate, -3.0)
            yield n, h, q[n, :, h], k[n, :, h], v[n, :, h], a, ref.decay_error(z, kind, -3.0), beta[n, :, h], S[n, h]


def within(got, want, tol, what):
    off = np.abs(got - want) / tol
    assert off.max() <= 1.0, "%s: %.3g times its bound" % (what, off.max())


def options(decay, gate, l2norm):
    return dict(decay=decay, gate=gate, gate_lower=-3.0, l2norm_qk=l2norm)


@pytest.mark.parametrize("d,dtype", [(64, BF), (64, F), (128, BF), (128, F)])
@pytest.mark.parametrize("K", [1, 4, 5, 8, 9, 27])
@pytest.mark.parametrize("decay,gate,l2norm", [("channel", "log", False), ("channel", "logsigmoid", True),
                                               ("channel", "bounded", False), ("scalar", "logsigmoid", True),
                                               ("none", "log", False)])
def test_bounds_of_blocks(d, dtype, K, decay, gate, l2norm):
    args = inputs(2, K, 2, d, dtype, decay, gate, seed=K)
    before = list(heads(args, decay, gate))
    out = f64(decode_tokens(*args[:5], 0.125, args[5], **options(decay, gate, l2norm)))
    state = f64(args[5])
    for n, h, q, k, v, a, ea, beta, S in before:
        r = ref.tokens(q, k, v, a, ea, beta, 0.125, S, K, l2norm)
        within(out[n, :, h], r["out"], r["tol_out"] + half_step(r["out"], dtype == BF), "out")
        within(state[n, h], r["state"], r["tol_state"] + half_step(r["state"], False), "state")


@pytest.mark.parametrize("d", [64, 128])
def test_beside_single_steps(d):
    """Within the sum of the bounds of both ways, in every output and every value of the state."""
    K, how = 12, options("channel", "logsigmoid", True)
    args = inputs(3, K, 4, d, F, "channel", "logsigmoid", seed=4)
    before, one = list(heads(args, "channel", "logsigmoid")), args[5].clone()
    steps = torch.stack([decode_step(*(x[:, t].contiguous() for x in args[:5]), 0.1, one, **how) for t in range(K)], 1)
    out = decode_tokens(*args[:5], 0.1, args[5], **how)
    out, steps, many, one = f64(out), f64(steps), f64(args[5]), f64(one)
    for n, h, q, k, v, a, ea, beta, S in before:
        r = ref.tokens(q, k, v, a, ea, beta, 0.1, S, K, True)
        s = layer_reference.tokens(q, k, v, a, beta, 0.1, S, K, True)
        assert np.allclose(r["out"], s["out"], rtol=1e-12, atol=1e-12)
        within(out[n, :, h], steps[n, :, h], r["tol_out"] + s["tol_out"] + 2 * half_step(r["out"], False), "out")
        within(many[n, h], one[n, h], r["tol_state"] + s["tol_state"] + 2 * half_step(r["state"], False), "state")
