"""The 64-bit references' gradients against differences of the formulas they belong to."""
import numpy as np
import pytest

from tests import layer_reference as ref

EPS = 1e-6


def slope(f, x, d):
    """Central difference of f along d; off by O(h^2) and 2^-52 / h: about 1e-10 at h = 1e-5."""
    h = 1e-5
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("weighted", [False, True])
def test_norm_gradient(weighted):
    rng = np.random.default_rng(1)
    h, dy, dh = (rng.standard_normal((3, 24)) for _ in range(3))
    w = 1 + 0.3 * rng.standard_normal(24) if weighted else None
    g = ref.norm_grad(dy, h, w, EPS, dh)
    d = rng.standard_normal(h.shape)
    want = slope(lambda x: (ref.norm(x, w, EPS)["y"] * dy).sum() + (x * dh).sum(), h, d)
    assert abs((g["dx"] * d).sum() - want) < 1e-8
    if weighted:
        dw = rng.standard_normal(24)
        want = slope(lambda x: (ref.norm(h, x, EPS)["y"] * dy).sum(), w, dw)
        assert abs((g["dw"] * dw).sum() - want) < 1e-8


@pytest.mark.parametrize("weighted", [False, True])
def test_gate_gradient(weighted):
    rng = np.random.default_rng(2)
    o, z, dout = (rng.standard_normal((5, 16)) for _ in range(3))
    w = 1 + 0.3 * rng.standard_normal(16) if weighted else None
    g = ref.gate_grad(dout, o, z, w, EPS)
    for name, x, f in (("do", o, lambda x: ref.gate(x, z, w, EPS)), ("dz", z, lambda x: ref.gate(o, x, w, EPS)),
                       ("dw", w, lambda x: ref.gate(o, z, x, EPS))):
        if x is None:
            continue
        d = rng.standard_normal(x.shape)
        assert abs((g[name] * d).sum() - slope(lambda x: (f(x) * dout).sum(), x, d)) < 1e-8


def test_tokens_are_the_oracles_steps():
    import oracle
    rng = np.random.default_rng(3)
    K, d = 5, 64
    q, k, v = (rng.standard_normal((K, d)) / 8 for _ in range(3))
    g, beta, S = -rng.random((K, d)), rng.random(K), rng.standard_normal((d, d))
    got = ref.tokens(q, k, v, np.exp(g), beta, 0.3, S, K, False)
    out, fin = oracle.scan(q[None, :, None], k[None, :, None], v[None, :, None], g[None, :, None], beta[None, :, None],
                           0.3, S[None, None])
    assert np.abs(got["out"] - out[0, :, 0]).max() < 1e-12 and np.abs(got["state"] - fin[0, 0]).max() < 1e-12
    assert not ref.tokens(q, k, v, np.exp(g), beta, 0.3, S, 2, False)["out"][2:].any()
