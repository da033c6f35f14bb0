"""Empty calls of the state operators are no-ops, whatever pointers come with them: a tensor
without elements has a null one."""
import ctypes

import pytest

from gated_delta_rule_45_gb300 import kda

M = 0x1000000   # fake buffers 16 MB apart; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_45_gb300 import build
    build.build()
    return kda.load()


@pytest.mark.parametrize("S", [None, 1 * M])
@pytest.mark.parametrize("parents", [None, 2 * M])
@pytest.mark.parametrize("rows", [0, 5])
def test_linrec_decode_step_of_no_sequences(lib, rows, parents, S):
    """B == 0 with `parents` an empty tensor (null) over a table of states."""
    assert lib.linrec_decode_step(None, None, 0, S, rows, parents, 0, 2, 64, 0, 0, None, None,
                                  None) == kda.OK


@pytest.mark.parametrize("rows", [0, 5])
@pytest.mark.parametrize("parents", [None, 2 * M])
def test_decode_step_parents_of_no_sequences(lib, rows, parents):
    assert lib.kda_decode_step_parents(None, None, None, None, 0, None, 1 * M, rows, parents,
                                       None, 0, 2, 64, 64, 0, None, None) == kda.OK


def test_beams_of_no_requests(lib):
    assert lib.beam_select(None, 100, None, None, 0, 4, 100, 8, 0, 0, None, None, None, None, 0,
                           None) == kda.OK
    d = (kda._BeamState * 1)()
    d[0].row_bytes = 64
    assert lib.beam_reorder(ctypes.byref(d), 1, None, 0, 4, None) == kda.OK


def test_sizes_are_checked_all_the_same(lib):
    f = lib.linrec_decode_step
    assert f(None, None, 0, None, -1, None, 0, 2, 64, 0, 0, None, None, None) == kda.ERR_INVALID_ARG
    assert f(None, None, 0, None, 0, None, 0, 0, 64, 0, 0, None, None, None) == kda.ERR_INVALID_ARG
    assert f(None, None, 7, None, 0, None, 0, 2, 64, 0, 0, None, None, None) == kda.ERR_INVALID_ARG


def test_scan_timeout_check_rejects_on_host(lib):
    f = lib.kda_check_scan_timeout
    n = kda.SCAN_CHECK_BYTES
    for args in ((None, n, 10 ** 6), (M + 8, n, 10 ** 6), (M, n - 1, 10 ** 6), (M, n, 999),
                 (M, n, 10 ** 9 + 1)):
        assert f(*args, None) == kda.ERR_INVALID_ARG
