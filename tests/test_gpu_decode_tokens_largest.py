"""Values next to the largest that the call takes, 2^128 (1 - 2^-12): what the single step keeps finite stays finite
over several tokens."""
import pytest
import torch

from kimi_delta_attention_17_gb300 import build, decode_step, decode_tokens

pytestmark = pytest.mark.gpu

MOST = 3.40199e38  # the next 11-bit value is the largest, not infinity, for what is below 3.401994e38
# Such a value's first part is off by up to 2^-11 of it, so what is left has 12 bits, cut off to 11 (2^-23); the other
# factor's parts leave as much; the product of the two second parts is left out (2^-22); three sums in an MMA are
# cut off (2^-22 each): less than 2^-19.
REL = 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def zeros(K, d, H=2, N=2):
    q, k, v = (torch.zeros(N, K, H, d, device="cuda") for _ in range(3))
    return q, k, v, torch.ones(N, K, H, device="cuda"), torch.zeros(N, H, d, d, device="cuda")


def both(q, k, v, beta, state):
    """The outputs of the call and of the single steps, and their states."""
    one, many = state.clone(), state.clone()
    first = torch.stack([decode_step(*(t[:, i].contiguous() for t in (q, k, v)), None, beta[:, i].contiguous(), 1.0, one,
                                     decay="none") for i in range(q.shape[1])], 1)
    return decode_tokens(q, k, v, None, beta, 1.0, many, decay="none"), many, first, one


def near(got, want):
    assert torch.isfinite(want).all() and want.any()
    assert ((got.double() - want.double()).abs() <= REL * want.double().abs()).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("K", [1, 3, 8, 11])
def test_a_channel_that_no_token_touches(K, d):
    gen = torch.Generator(device="cuda").manual_seed(K)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v = n(2, K, 2, d), torch.nn.functional.normalize(n(2, K, 2, d), dim=-1), n(2, K, 2, d)
    beta, state, at = torch.sigmoid(n(2, K, 2)), n(2, 2, d, d), d // 2 + 3
    q[..., at] = k[..., at] = 0.0
    state[:, :, at] = 0.0
    out, held, _, _ = both(q, k, v, beta, state)
    state[:, :, at] = torch.where(n(2, 2, d) > 0, MOST, -MOST)
    got, after, single, _ = both(q, k, v, beta, state)
    assert torch.isfinite(single).all() and torch.equal(got, out)
    assert torch.equal(after[:, :, at], state[:, :, at])
    after[:, :, at] = 0.0
    assert torch.equal(after, held)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("K", [1, 3, 8])
def test_products_with_the_largest_values(K, d):
    q, k, v, beta, state = zeros(K, d)
    state[:, :, 5] = MOST  # read by a small q
    q[..., 5], k[..., 7] = 0.25, 1.0
    out, after, single, one = both(q, k, v, beta, state)
    near(out, single)
    assert torch.equal(after, one)
    q, k, v, beta, state = zeros(K, d)
    state[:, :, 5] = -(2.0 ** -100)  # read by a large q
    q[..., 5], k[..., 7] = MOST, 1.0
    near(*both(q, k, v, beta, state)[::2])


@pytest.mark.parametrize("d", [64, 128])
def test_products_that_the_state_takes(d):
    for key, value in ((2.0 ** -20, MOST), (-MOST, 2.0 ** -60)):
        q, k, v, beta, state = zeros(1, d)
        k[..., 9] = key
        v[:] = value
        q[..., 9] = 2.0 ** -70
        out, after, single, one = both(q, k, v, beta, state)
        near(out, single)
        assert ((after.double() - one.double()).abs() <= REL * one.double().abs()).all() and one[:, :, 9].all()
