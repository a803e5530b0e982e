"""A serving loop's step on a batch that has no rows, for both kinds of state."""
import pytest
import torch

from kimi_delta_attention_17_gb300 import build, decode_step, gated_scan_step, state_copy

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def test_steps_of_no_rows():
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    vectors, matrices = torch.ones(5, 16, device="cuda"), torch.ones(5, 2, 64, 64, device="cuda")
    x = torch.empty(0, 16, device="cuda")
    assert gated_scan_step(x, x, vectors, slots=none).shape == (0, 16)
    assert gated_scan_step(x.bfloat16(), x, vectors, slots=none).shape == (0, 16)
    assert gated_scan_step(x, x, vectors[:0]).shape == (0, 16)
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert decode_step(q, q, q, q.float(), torch.empty(0, 2, device="cuda"), 0.1, matrices, slots=none).shape == q.shape
    state_copy(vectors, none, none)
    torch.cuda.synchronize()
    assert (vectors == 1).all() and (matrices == 1).all()
