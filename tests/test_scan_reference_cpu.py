"""The 64-bit reference of the gated linear recurrence against differences: its
gradients are those of its values."""
import numpy as np
import pytest

from tests import scan_reference as ref


@pytest.mark.parametrize("write", ["plain", "complement", "norm"])
@pytest.mark.parametrize("kind", ["log", "logsigmoid", "bounded"])
def test_gradients_match_differences(kind, write):
    rng = np.random.default_rng(5)
    T, D, step = 7, 3, 1e-5
    g = rng.standard_normal((T, D)) + (2.0 if kind == "logsigmoid" else -1.0)
    if kind == "log":
        g = -np.abs(g) - 0.05
    v = dict(x=rng.standard_normal((T, D)), g=g, init=rng.standard_normal(D))
    dout, dfinal = rng.standard_normal((T, D)), rng.standard_normal(D)

    def loss(v):
        r = ref.scan(v["x"], v["g"], v["init"], kind, -5.0, write)
        return (r["out"] * dout).sum() + (r["final"] * dfinal).sum()

    r = ref.scan(v["x"], v["g"], v["init"], kind, -5.0, write, dout, dfinal)
    for name, grad in (("x", r["dx"]), ("g", r["dg"]), ("init", r["dinit"])):
        for at in np.ndindex(v[name].shape):
            up, down = ({k: a.copy() for k, a in v.items()} for _ in range(2))
            up[name][at] += step
            down[name][at] -= step
            # The difference's own error: step^2 times a third derivative of
            # some tens (1e-9) and the rounding of a loss of some tens over
            # 2 step (1e-10): far below 1e-6.
            assert abs((loss(up) - loss(down)) / (2 * step) - grad[at]) <= 1e-6


def test_slope_of_the_norm_weight_at_one_is_zero():
    r = ref.scan(np.ones((1, 2)), np.array([[0.0, -1.0]]), None, "log", -5.0, "norm", np.ones((1, 2)))
    assert r["out"][0, 0] == 0.0 and r["dg"][0, 0] == 0.0 and r["dg"][0, 1] != 0.0
