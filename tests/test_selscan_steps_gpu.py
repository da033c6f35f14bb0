"""Step sizes and decays of the selective scan by themselves: calls whose states and gradients are
a step, or a product of decays, and nothing else."""
import numpy as np
import pytest
import torch

from gated_delta_rule_45_gb300 import kda
from layer_checks import np64, offsets

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
EX2 = 2.0 ** -22     # published error of the fast exponential


def _zeros(*shape):
    return torch.zeros(*shape, device="cuda")


def _ones(*shape):
    return torch.ones(*shape, device="cuda")


def test_steps_keep_their_relative_precision():
    """softplus from e^-86 to 30: the exponential's error, and five roundings or errors of 2^-24
    each (the polynomial's fit, its last two sums, the exponential's correction, the sum with v).  A
    state of D x B with x = B = 1 from zero is the step, and so is dx with g = 1."""
    R, d = 64, 128
    v = torch.linspace(-86.0, 30.0, R * d)
    want = np.logaddexp(np64(v), 0.0).reshape(R, 1, d)
    tol = EX2 + 5 * U32
    dt, one, par = v.view(R, 1, d).cuda(), _ones(R, 1, 1), _zeros(1, d, 1)

    def held(what, got):
        off = np.abs(np64(got).reshape(want.shape) - want) / want
        assert off.max() <= tol, (what, off.max() / U32, float(v[off.argmax()]))

    S = _zeros(R, 1, d, 1)
    kda.selscan_decode_step(_ones(R, 1, d), dt, par, one, one, S)
    held("decode step", S)
    cu = torch.arange(R + 1, dtype=torch.int32, device="cuda")
    for x in (_ones(R, 1, d), _ones(R, 1, d + 1)[:, :, 1:]):      # wide loads and single values
        ins = (x, dt, par, one, one, None, cu)
        _, S_T = kda.selscan_prefill(*ins)
        held("prefill", S_T)
        g = kda.selscan_backward(*ins[:4], _zeros(R, 1, 1), None, cu, _zeros(R, 1, d),
                                 _ones(R, 1, d, 1))
        held("backward", g["dx"])


def test_steps_of_masked_and_broken_tokens():
    """A dt of -inf, or of the type's lowest value, is a step of 0; a NaN stays one, and so is exp of
    an infinite step times a rate of 0."""
    low = torch.finfo(torch.float32).min
    dt = torch.tensor([float("-inf"), low, -200.0, float("inf"), float("nan"), 1e30]).view(6, 1, 1)
    one = _ones(6, 1, 1)
    S = _zeros(6, 1, 1, 1)
    kda.selscan_decode_step(one, dt.cuda(), _zeros(1, 1, 1), one, one, S)
    cu = torch.arange(7, dtype=torch.int32, device="cuda")
    _, S_T = kda.selscan_prefill(one, dt.cuda(), _zeros(1, 1, 1), one, one, None, cu)
    for got in (S.flatten().tolist(), S_T.flatten().tolist()):
        assert got[:3] == [0.0] * 3 and got[5] == float(torch.tensor(1e30))
        assert np.isnan(got[3]) and np.isnan(got[4])


def _decay_bound(arg):
    """Of one decay: the rate's rounding and the constant's, the argument's; the exponential."""
    return 3 * U32 * np.abs(arg) + EX2 + 2 * U32


def test_single_decays():
    R, d = 32, 256
    g = torch.Generator().manual_seed(1)
    step = torch.exp(torch.rand(R, 1, d, generator=g) * 12 - 10)       # 4.5e-5 to 7.4
    A = -torch.exp(torch.rand(1, d, 8, generator=g) * 4 - 2)
    S = _ones(R, 1, d, 8)
    kda.selscan_decode_step(_zeros(R, 1, d), step.cuda(), A.cuda(), _zeros(R, 1, 8),
                            _zeros(R, 1, 8), S, softplus=False)
    arg = np64(step)[..., None] * np64(A)
    assert (np.abs(np64(S) / np.exp(arg) - 1.0) <= _decay_bound(arg)).all()


def test_decays_of_a_whole_sequence():
    """200 tokens in one walk: the decays' own errors add up, and a rounding a product."""
    T, d, n = 200, 64, 16
    g = torch.Generator().manual_seed(2)
    step = torch.rand(T, 1, d, generator=g) * 0.1
    A = -torch.exp(torch.rand(1, d, n, generator=g) * 4 - 2)
    cu = offsets([T])[1].cuda()
    assert kda.selscan_workspace_size(1, T, 1, d, n) <= 256       # not cut along the tokens
    ins = (_zeros(T, 1, d), step.cuda(), A.cuda(), _zeros(T, 1, n), _zeros(T, 1, n), None, cu)
    S0 = _ones(1, 1, d, n)
    _, S_T = kda.selscan_prefill(*ins[:5], S0, cu, softplus=False)
    gr = kda.selscan_backward(*ins[:5], S0, cu, _zeros(T, 1, d), S0, softplus=False)
    arg = np64(step)[..., None] * np64(A)
    want, tol = np.exp(arg.sum(0)), (_decay_bound(arg) + U32).sum(0)
    for got in (S_T, gr["dS0"]):
        assert (np.abs(np64(got)[0] / want - 1.0) <= tol).all()


@pytest.mark.parametrize("lens", [[200], [900], [70, 0, 3, 500]])
def test_a_rate_of_zero_keeps_the_state(lens):
    """Whole sequences, and cut along the tokens."""
    d, n = 24, 16
    cu = offsets(lens)[1].cuda()
    T, N = sum(lens), len(lens)
    g = torch.Generator().manual_seed(3)
    dt = torch.randn(T, 1, d, generator=g).cuda()
    S0, dS = (torch.randn(N, 1, d, n, generator=g).cuda() for _ in range(2))
    ins = (_zeros(T, 1, d), dt, _zeros(1, d, n), _zeros(T, 1, n), _zeros(T, 1, n), S0, cu)
    assert torch.equal(kda.selscan_prefill(*ins)[1], S0)
    assert torch.equal(kda.selscan_backward(*ins, _zeros(T, 1, d), dS)["dS0"], dS)
