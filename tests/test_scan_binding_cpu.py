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


def test_carries_size_of_sizes_that_are_refused(L):
    f = L.kda_gated_scan_carries_size
    most = 2 ** 31 - 1
    for bad in ((most, most, most, most), (1, most, 8, 1), (2 ** 20, 2 ** 12, 8, 2 ** 20), (1, 2 ** 22, 2 ** 18, 1),
                (1, 0, most, most), (1, 0, 8, most), (1, 0, most - 7, 1)):
        assert f(*bad) == 0, bad
        B, T, D, N = bad
        cu = FAKE if N != B else None
        assert L.kda_gated_scan_fwd(FAKE, FAKE, None, cu, FAKE, None, None, B, T, D, N, 1, 1, None, None) == INVALID
    assert f(1, 2 ** 20, 2 ** 19, 1) == (2 ** 14 + 1) * 2 ** 21


def test_compaction_of_more_slots_than_its_indices_hold(L):
    P = 2 ** 30 + 1
    assert L.kda_state_compact_workspace_size(P) == 0
    assert L.kda_state_compact_workspace_size(2 ** 31 - 1) == 0
    assert L.kda_state_compact_workspace_size(2 ** 30) > 2 ** 33
    for slots in (P, 2 ** 31 - 1):
        assert L.kda_state_compact(FAKE, slots, FAKE, FAKE, FAKE, 1, 16, FAKE, 2 ** 40, None) == UNSUPPORTED
