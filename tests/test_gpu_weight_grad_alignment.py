"""A weight's gradient inside a flat buffer of gradients, where it may begin at any float."""
import pytest
import torch

from kimi_delta_attention_17_gb300 import build, output_gate_rmsnorm_bwd, rmsnorm_bwd, rmsnorm_fwd

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def check(call, D):
    want = call(None)
    assert want.any()
    for offset in (1, 2, 3, 4):
        flat = torch.full((D + 8,), 7.0, device="cuda")
        got = call(flat[offset:offset + D])
        assert got.data_ptr() == flat.data_ptr() + 4 * offset and torch.equal(got, want)
        assert (flat[:offset] == 7.0).all() and (flat[offset + D:] == 7.0).all()


@pytest.mark.parametrize("dtype,hdtype", [(BF, BF), (BF, F), (F, F)])
@pytest.mark.parametrize("D", [8, 128, 264, 512, 520, 1288, 2048, 4104, 8200, 12296, 16392, 32768])
def test_rmsnorm(D, dtype, hdtype):
    """Few rows, which one CTA takes and writes the gradient itself, and more."""
    for rows in (1, 6, 7, 41):
        gen = torch.Generator(device="cuda").manual_seed(rows)
        n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        x, dy, w = n(rows, D).to(dtype), n(rows, D).to(dtype), n(D)
        _, h, rstd = rmsnorm_fwd(x, w, residual=None if hdtype == dtype else n(rows, D), save_rstd=True)
        check(lambda to: rmsnorm_bwd(dy, h, rstd, w, dweight=to)[2], D)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("d", [64, 128])
def test_output_gate(d, dtype):
    for tokens in (1, 50, 3000):
        gen = torch.Generator(device="cuda").manual_seed(tokens)
        dout, o, z = (torch.randn(tokens, 3, d, generator=gen, device="cuda").to(dtype) for _ in range(3))
        w = torch.rand(d, generator=gen, device="cuda") + 0.5
        check(lambda to: output_gate_rmsnorm_bwd(dout, o, z, w, dweight=to)[2], d)
