"""The binding's options, and sizes at which the C entries of the gated scan and the state pool have
nothing to do or refuse, without a GPU."""
import pytest
import torch

from kimi_delta_attention_17_gb300 import _lib, build, scan

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 1 << 20  # 16-byte aligned, never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def test_lower_bound_is_read_at_every_call():
    """A tensor changed in place counts as it is now."""
    lower = torch.tensor(-5.0)
    assert scan._scan_options("bounded", lower, "plain")._obj.gate_lower == -5.0
    lower.fill_(-2.0)
    assert scan._scan_options("bounded", lower, "plain")._obj.gate_lower == -2.0
    assert scan._scan_options("bounded", -2, "plain")._obj.gate_lower == -2.0


def test_a_step_of_no_rows_over_a_pool(L):
    """An empty slots tensor has a NULL pointer; the pool has its slots all the same."""
    for slots in (None, FAKE):
        for dtype in (0, 1):
            assert L.kda_gated_scan_step(None, None, FAKE, slots, None, 0, 4, 8, dtype, dtype, None, None) == OK
    assert L.kda_gated_scan_step(None, None, None, None, None, 0, 0, 8, 1, 1, None, None) == OK
    assert L.kda_gated_scan_step(None, None, FAKE, None, None, 0, -1, 8, 1, 1, None, None) == INVALID
    # Rows without slots still need a state each.
    assert L.kda_gated_scan_step(FAKE, FAKE, FAKE, None, FAKE, 1, 4, 8, 1, 1, None, None) == INVALID
