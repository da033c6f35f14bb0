"""Gates of the linear recurrence at the ends of their range on the GPU: log gates of zero
and next to it, constant over long sequences, and gates above one.  Bounds as in
``test_linrec_gpu``: the largest error that 32-bit arithmetic can leave."""
import numpy as np
import pytest
import torch

from gated_delta_rule_45_gb300 import kda
from oracle import linrec as ref

pytestmark = pytest.mark.gpu

ULPS = {"channel": 2, "log_bf16": 6}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _within(got, want, bound):
    got = _np(got)
    assert np.isfinite(got).all()
    off = np.abs(got - want) - (np.asarray(bound) + 2.0 ** -126)
    assert (off <= 0).all(), f"{(off > 0).sum()} of {off.size} beyond, worst by {off.max():.3g}"


def _every_log_gate():
    """Every bf16 value from -0 down to -inf, and +0."""
    bits = torch.cat([torch.arange(0x8000, 0xff81), torch.tensor([0])]).to(torch.int32)
    return (bits << 16).view(torch.float32).to(torch.bfloat16)


def test_log_gates_one_by_one():
    """a = e^(log a) of every bf16 value: within an instruction's error of it and that of its
    argument, never above 1, and at 0 exactly 1."""
    la = _every_log_gate()
    n = la.numel()
    x, S = torch.zeros(n, 1, 1, device="cuda"), torch.ones(n, 1, 1, device="cuda")
    kda.linrec_decode_step(x, la.reshape(n, 1, 1).cuda(), S, gate="log_bf16")
    a, want = _np(S).reshape(-1), np.exp(_np(la))
    v = np.abs(_np(la))
    assert (a[v < 2.0 ** -26] == 1.0).all(), a[v < 2.0 ** -26]
    assert (a <= 1.0).all()
    # a rounding of log a times log2 e (2^-24 of it), that of log2 e (1.4e-8 of it)
    tol = 1.6e-7 + np.where(v < 200, v, 0) * (2.0 ** -24 + 1.4e-8)
    assert (np.abs(a - want) <= tol * want + 2.0 ** -126).all()
    # the same gates in a prefill, each over one token
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    _, S_T = kda.linrec_prefill(x, la.reshape(n, 1, 1).cuda(), torch.ones_like(S), cu,
                                gate="log_bf16", check_device_status=True)
    assert torch.equal(S_T, S)


@pytest.mark.parametrize("d", [64, 33])
def test_log_gates_of_zero_keep_the_state(d):
    """log a = 0 (padding, a saturated gate) hands the state on unchanged however long."""
    T = 20000
    S0 = torch.randn(1, 1, d, generator=torch.Generator().manual_seed(d)).cuda()
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    x = torch.zeros(T, 1, d, device="cuda")
    for zero in (0.0, -0.0):
        la = torch.full((T, 1, d), zero, dtype=torch.bfloat16, device="cuda")
        y, S_T, st = kda.linrec_prefill(x, la, S0, cu, gate="log_bf16", save_states=True,
                                        check_device_status=True)
        assert torch.equal(S_T, S0) and torch.equal(y, S0.expand_as(y))
        dS = torch.randn(1, 1, d, generator=torch.Generator().manual_seed(1)).cuda()
        g = kda.linrec_backward(x, la, S0, cu, x, dS, states=st, gate="log_bf16")
        assert torch.equal(g["dS0"], dS) and torch.equal(g["dx"], dS.expand_as(x))
        # the complement takes nothing in
        big = torch.full_like(x, 1e3)
        y, S_T = kda.linrec_prefill(big, la, S0, cu, gate="log_bf16", complement=True)
        assert torch.equal(S_T, S0) and torch.equal(y, S0.expand_as(y))


@pytest.mark.parametrize("complement", [False, True])
def test_constant_log_gates_over_long_sequences(complement):
    """One log gate a channel, from the smallest bf16 values to 1/8, over 100000 tokens: the
    error of one input is raised to the number of tokens."""
    T, d = 100000, 64
    la = -torch.cat([torch.tensor([0.0, 2.0 ** -133, 2.0 ** -126, 1e-30, 1e-12]),
                     torch.logspace(-9, np.log10(0.125), 59)]).to(torch.bfloat16)
    g = torch.Generator().manual_seed(3)
    x, S0 = torch.rand(T, 1, d, generator=g), torch.randn(1, 1, d, generator=g)
    gate = la.expand(T, 1, d).contiguous()
    cu = torch.tensor([0, T], dtype=torch.int32)
    y, S_T = kda.linrec_prefill(x.cuda(), gate.cuda(), S0.cuda(), cu.cuda(), gate="log_bf16",
                                complement=complement, check_device_status=True)
    # 1 - a in 64 bits without the loss next to 1: u = -expm1(log a) x
    lg = _np(la)
    u = _np(x) * (-np.expm1(lg) if complement else 1.0)
    a = np.broadcast_to(np.exp(lg), (T, 1, d))
    h, S_ref = ref.forward(u, a, _np(S0), [0, T])
    _, e, e_S = ref.forward_bound(u, a, _np(S0), [0, T], False, ULPS["log_bf16"])
    _within(y, h, e)
    _within(S_T, S_ref, e_S)


def _run(x, a, S0, dy, dS_T, lens, complement=False):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    dev = [t.cuda() if t is not None else None for t in (x, a, S0)]
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = kda.linrec_prefill(*dev, cud, complement=complement, save_states=True,
                             check_device_status=True)
    args = (_np(x), _np(a), _np(S0), cu)
    h, S_ref = ref.forward(*args, complement)
    _, e, e_S = ref.forward_bound(*args, complement, 2)
    _within(out[0], h, e)
    _within(out[1], S_ref, e_S)
    _within(out[2], ref.chunk_states(h, cu, kda.LINREC_CHUNK),
            ref.chunk_states(e, cu, kda.LINREC_CHUNK))
    if dy is not None:
        got = kda.linrec_backward(*dev, cud, dy.cuda(), dS_T.cuda(), states=out[2],
                                  complement=complement, check_device_status=True)
        full = (*args, _np(dy), _np(dS_T), complement, "channel")
        want, bound = ref.backward(*full), ref.backward_bound(*full, 2)
        for k in want:
            _within(got[k], want[k], bound[k])


@pytest.mark.parametrize("lens", [[300], [5000], [40, 2000, 3, 900]])
def test_gates_above_one_of_a_zero_state(lens):
    """Gates of 1.5, whose product over 256 tokens is infinite, multiply a state of zero: it
    stays zero until the first input."""
    T, d = sum(lens), 66
    x = torch.zeros(T, 1, d)
    a = torch.full((T, 1, d), 1.5)
    a[:, :, 1::2] = 0.9                  # a lane's other channel decays
    at = 0
    for n in lens:                       # an input near each sequence's end
        x[at + n - 2] = 1.0
        at += n
    zeros = torch.zeros(len(lens), 1, d)
    _run(x, a, None, torch.zeros(T, 1, d), zeros, lens)
    _run(x, a, zeros, torch.zeros(T, 1, d), zeros, lens)


def test_gates_above_one_of_a_small_state():
    """A state of 1e-30 behind gates of 1.4 over 280 tokens, at the edge of what the header
    allows: over 256 their product is 3e37, over 280 it is infinite, and the state comes to
    8e10; then it decays again."""
    T, d = 3000, 64
    for begin in (0, 256, 300, 1000):
        a = torch.full((T, 1, d), 0.99)
        a[:begin] = 1.0
        a[begin:begin + 280] = 1.4
        a[:, :, ::3] = 0.97
        S0 = torch.full((1, 1, d), 1e-30)
        g = torch.Generator().manual_seed(begin)
        dy = torch.randn(T, 1, d, generator=g) * 1e-30
        _run(torch.zeros(T, 1, d), a, S0, dy, torch.full((1, 1, d), 1e-30), [T])
