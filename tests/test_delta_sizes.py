"""CPU: sizes of the gated delta rule at the ends of what the C ABI takes; nothing is launched."""
import ctypes

import pytest

import ssd_chunked_scan_fwd_amd as ssd
from test_delta_abi import INVALID, MB, delta, ptr


@pytest.mark.parametrize("slots", [2 ** 31 - 1, 2 ** 30, 2 ** 29 + 7])
def test_step_overlap_of_the_largest_pools(slots):
    """A pool whose bytes pass 64 bits still holds what lies behind its start."""
    sh = delta(batch=1, nheads=65535, nqk_heads=1, dk=256, dv=256)
    far = [ptr(256 * MB * (i + 1)) for i in range(10)]
    args = [ptr(16 * MB), *far[1:7], slots, 1.0, far[9], ctypes.byref(sh), None]
    for i in (1, 2, 3, 4, 5, 6, 9):
        assert ssd.lib().ssd_gated_delta_step(*args) == INVALID, i
