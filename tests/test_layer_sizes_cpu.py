"""Sizes at the ends of what the operators around a layer's recurrence take, without a GPU: a size
that no launch can hold is refused as unsupported before any CUDA call."""
import ctypes

import pytest

from gated_delta_rule_45_gb300 import kda

G = 1 << 42     # fake buffers far apart; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_45_gb300 import build
    build.build()
    return kda.load()


@pytest.mark.parametrize("B,H,d", [(2 ** 15 - 1, 2 ** 20, 1), (2 ** 16 - 1, 2 ** 19, 1),
                                   (2 ** 15, 2 ** 20, 1), (2 ** 25, 2 ** 10, 1)])
def test_scan_step_has_a_launch(lib, B, H, d):
    r = kda._ScanRows(*(G * i for i in range(1, 5)), None, H * d, H * d, H, H, 0)
    st = lib.selscan_decode_step(ctypes.byref(r), 6 * G, None, None, 7 * G, B, None, B, H, d, 1, 0,
                                 1, 8 * G, 9 * G, None)
    assert st == kda.ERR_UNSUPPORTED
