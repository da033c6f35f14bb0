"""Selections of different sizes from several host threads at once, each on its own stream
and workspace.  The threads call the library itself, which runs without Python's lock: the
binding's own work before each call would keep them from ever being in it together."""
import ctypes
import threading

import pytest
import torch

from gated_delta_rule_45_gb300 import kda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape,sizes", [
    ((64, 4, 128000, torch.bfloat16), (32, 64)),      # the pieces' lists of one kernel
    ((1, 32, 1 << 20, torch.float32), (48, 64)),      # and the joining kernel's
])
def test_two_threads_with_different_sizes(shape, sizes):
    B, K, V, dtype = shape
    z = torch.randn(B * K, V, generator=torch.Generator(device="cuda").manual_seed(0),
                    device="cuda").mul_(3).to(dtype)
    sc = -torch.rand(B, K, device="cuda")
    want = {n: [t.cpu() for t in kda.beam_select(z, sc, n)] for n in sizes}
    ready, errors = threading.Barrier(len(sizes)), []

    def work(n):
        try:
            s = torch.cuda.Stream()
            ws = torch.empty(kda.beam_select_workspace_size(B, K, V, n), dtype=torch.uint8,
                             device="cuda")
            out = tuple(torch.empty(B, n, dtype=t, device="cuda")
                        for t in (torch.float32, torch.int32, torch.int32))
            torch.cuda.synchronize()
            p, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
            args = (p(z.data_ptr()), i64(V), p(sc.data_ptr()), p(None), i32(B), i32(K), i32(V),
                    i32(n), i32(0), ctypes.c_int(kda._DTYPE_CODES[dtype]),
                    *(p(t.data_ptr()) for t in out), p(ws.data_ptr()),
                    ctypes.c_size_t(ws.numel()), p(s.cuda_stream))
            call = kda.load().beam_select
            ready.wait(60)
            for i in range(3000):
                st = call(*args)
                assert st == kda.OK, f"call {i}: {st}"
                if i % 200 == 199:
                    s.synchronize()
            s.synchronize()
            for u, v in zip(out, want[n]):
                assert torch.equal(u.cpu(), v)
        except BaseException as e:
            errors.append((n, e))

    threads = [threading.Thread(target=work, args=(n,)) for n in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
