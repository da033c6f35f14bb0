"""The wait limit of the gated linear recurrence's tiles, run on purpose.

kda_check_scan_timeout runs the forward kernel on three tiles of which nobody takes the
first, with a limit of 1 ms.  Nothing faults or hangs: the tiles behind it give up, the
kernel returns, the workspace's status word reads KDA_ERR_DEVICE_TIMEOUT, and the same
workspace serves a correct call right after."""
import time

import numpy as np
import pytest
import torch

from gated_delta_rule_45_gb300 import kda
from oracle import linrec as ref

pytestmark = pytest.mark.gpu


def _timeout_once(ws, ns):
    kda.check_scan_timeout(ws, ns)
    with pytest.raises(kda.KdaError) as e:
        kda.device_status(ws)
    assert e.value.status == kda.ERR_DEVICE_TIMEOUT


def test_waits_run_out_and_the_workspace_serves_the_next_call():
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for ns in (1_000_000, 100_000, 1_000_000):
        t0 = time.perf_counter()
        _timeout_once(ws, ns)
        assert time.perf_counter() - t0 < 1.5      # well before the calls' own 2 s
        g = torch.Generator().manual_seed(ns)
        T, d = 3000, 40
        x, a = torch.randn(T, 1, d, generator=g), torch.rand(T, 1, d, generator=g)
        cu = [0, 1700, T]
        y, S_T = torch.empty(T, 1, d, device="cuda"), torch.empty(2, 1, d, device="cuda")
        kda.linrec_prefill_into(x.cuda(), a.cuda(), None,
                                torch.tensor(cu, dtype=torch.int32, device="cuda"), y, S_T, ws)
        kda.device_status(ws)
        args = (x.double().numpy(), a.double().numpy(), None, cu)
        h, S_ref = ref.forward(*args)
        _, e, e_S = ref.forward_bound(*args, False, 2)
        assert (np.abs(y.double().cpu().numpy() - h) <= e + 2.0 ** -126).all()
        assert (np.abs(S_T.double().cpu().numpy() - S_ref) <= e_S + 2.0 ** -126).all()


def test_bad_arguments():
    ws = torch.empty(kda.SCAN_CHECK_BYTES, dtype=torch.uint8, device="cuda")
    for bad in (10, 2_000_000_000):
        with pytest.raises(kda.KdaError) as e:
            kda.check_scan_timeout(ws, bad)
        assert e.value.status == kda.ERR_INVALID_ARG
    with pytest.raises(kda.KdaError) as e:
        kda.check_scan_timeout(ws[:-16], 1_000_000)
    assert e.value.status == kda.ERR_INVALID_ARG
