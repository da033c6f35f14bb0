"""The operators around a layer's recurrence where offsets pass 32 bits: the last rows against the
same rows in a call of their own."""
import pytest
import torch

from gated_delta_rule_45_gb300 import kda

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _room():
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB")
    yield
    torch.cuda.empty_cache()


def _cu(*c):
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def test_convolution_beyond_2_to_31_elements():
    D, T, tail = 4096, 600_000, 200
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, D, device="cuda", generator=g, dtype=BF)
    dy = torch.randn(T, D, device="cuda", generator=g, dtype=BF)
    w = torch.randn(D, 4, device="cuda", generator=g)
    cu = _cu(0, T - tail, T)
    y, S_T = kda.causalconv_prefill(x, w, None, None, cu)
    ys, Ss = kda.causalconv_prefill(x[-tail:], w, None, None, _cu(0, tail))
    assert torch.equal(y[-tail:], ys) and torch.equal(S_T[1:], Ss)
    del y
    gr = kda.causalconv_backward(x, w, None, None, cu, dy)
    gs = kda.causalconv_backward(x[-tail:], w, None, None, _cu(0, tail), dy[-tail:])
    assert torch.equal(gr["dx"][-tail:], gs["dx"])


def test_norm_beyond_2_to_31_elements():
    H, d, T, tail = 32, 128, 600_000, 100
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, H, d, device="cuda", generator=g, dtype=BF)
    z = torch.randn(T, H, d, device="cuda", generator=g, dtype=BF)
    w = torch.randn(d, device="cuda", generator=g)
    y = kda.groupnorm_forward(x, w, z=z)
    assert torch.equal(y[-tail:], kda.groupnorm_forward(x[-tail:], w, z=z[-tail:]))
    gr = kda.groupnorm_backward(x, w, None, y, z=z)
    gs = kda.groupnorm_backward(x[-tail:], w, None, y[-tail:].contiguous(), z=z[-tail:])
    assert torch.equal(gr["dx"][-tail:], gs["dx"]) and torch.equal(gr["dz"][-tail:], gs["dz"])


@pytest.mark.parametrize("lens", [[600_000 - 64, 64], [1000] * 599 + [936, 64]])
def test_scan_beyond_2_to_31_elements(lens):
    """Cut along the tokens, and whole sequences."""
    D, n, tail, T = 4096, 4, 64, sum(lens)
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g, dtype=BF)
    x, dt, B, C = rn(T, 1, D), rn(T, 1, D), rn(T, 1, n), rn(T, 1, n)
    A = -torch.rand(1, D, n, device="cuda", generator=g)
    cu = [0]
    for L in lens:
        cu.append(cu[-1] + L)
    y, S_T, st = kda.selscan_prefill(x, dt, A, B, C, None, _cu(*cu), save_states=True)
    small = [t[-tail:] for t in (x, dt)] + [A] + [t[-tail:] for t in (B, C)]
    ys, Ss, sts = kda.selscan_prefill(*small, None, _cu(0, tail), save_states=True)
    assert torch.equal(y[-tail:], ys) and torch.equal(S_T[-1:], Ss)
    gr = kda.selscan_backward(x, dt, A, B, C, None, _cu(*cu), y, states=st)
    gs = kda.selscan_backward(*small, None, _cu(0, tail), ys, states=sts)
    for k in ("dx", "ddt", "dB", "dC"):
        assert torch.equal(gr[k][-tail:], gs[k]), k


def test_steps_beyond_2_to_31_state_values():
    D, n, R = 4096, 16, 33_000
    g = torch.Generator(device="cuda").manual_seed(4)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)
    x, dt, B, C = (rn(R, 1, k).to(BF) for k in (D, D, n, n))
    A, S = -torch.rand(1, D, n, device="cuda", generator=g), rn(R, 1, D, n)
    last = [t[-3:] for t in (x, dt)] + [A] + [t[-3:] for t in (B, C)]
    S_last = S[-3:].clone()
    y = kda.selscan_decode_step(x, dt, A, B, C, S)
    assert torch.equal(y[-3:], kda.selscan_decode_step(*last, S_last))
    assert torch.equal(S[-3:], S_last)
