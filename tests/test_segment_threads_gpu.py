"""Segment combinations of different widths from two host threads at once, each on its own
stream, through the library itself (which runs without Python's lock)."""
import ctypes
import threading

import pytest
import torch

from gated_delta_rule_45_gb300 import kda

pytestmark = pytest.mark.gpu


def test_two_threads_with_different_widths():
    ready, errors = threading.Barrier(2), []

    def work(dk):
        try:
            s = torch.cuda.Stream()
            N, H, dv = 2, 2, 64
            t = [torch.randn(*sh, device="cuda") for sh in ((N, H, dv, dk), (N, H, dv),
                                                           (N, H, dk, dk), (N, H, dv, dk))]
            want, out = kda.segment_combine(*t), torch.empty_like(t[0])
            torch.cuda.synchronize()
            p, i32 = ctypes.c_void_p, ctypes.c_int32
            args = (*(p(u.data_ptr()) for u in t), i32(N), i32(H), i32(dk), i32(dv),
                    p(out.data_ptr()), p(s.cuda_stream))
            call = kda.load().kda_segment_combine
            ready.wait(60)
            for i in range(3000):
                st = call(*args)
                assert st == kda.OK, f"call {i}: {st}"
                if i % 200 == 199:
                    s.synchronize()
            s.synchronize()
            assert torch.equal(out, want)
        except BaseException as e:
            errors.append((dk, e))

    threads = [threading.Thread(target=work, args=(dk,)) for dk in (64, 128)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
