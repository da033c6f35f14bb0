"""Rates of the selective scan at the ends of their range."""
import pytest
import torch

from gated_delta_rule_45_gb300 import kda
from layer_checks import offsets

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rate", [torch.finfo(torch.float32).min, -2.9e38, -1e38])
@pytest.mark.parametrize("lens", [[5, 33, 0, 40], [450]])
def test_rates_at_the_end_of_the_range(lens, rate):
    """A rate of the type's lowest value leaves nothing of a state at any step, as one of -1e6 does
    at these steps (above 1e-3): the same bits.  Forward some steps are 0, where both keep all
    of it; backward none is: there the derivative by the step is the rate times a state and its
    gradient, beyond 3.4e38."""
    d, n = 24, 5
    cu = offsets(lens)[1].cuda()
    T, N = sum(lens), len(lens)
    g = torch.Generator().manual_seed(4)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()
    x, B, C, S0, dy, dS = (rn(T, 1, d), rn(T, 1, n), rn(T, 1, n), rn(N, 1, d, n), rn(T, 1, d),
                           rn(N, 1, d, n))
    dt = rn(T, 1, d).clamp(min=-5.0)
    some = dt.clone()
    some[::3] = -200.0
    A = -torch.exp(rn(1, d, n))

    def run(r):
        rates = A.clone()
        rates[:, ::2, 1], rates[:, :, 3] = r, r
        y, S_T, _ = kda.selscan_prefill(x, some, rates, B, C, S0, cu, save_states=True)
        S = S0.clone()
        y1 = kda.selscan_decode_step(x[:N], some[:N], rates, B[:N], C[:N], S)
        grads = kda.selscan_backward(x, dt, rates, B, C, S0, cu, dy, dS)
        return dict(grads, y=y, S_T=S_T, y1=y1, S=S)

    got, want = run(rate), run(-1e6)
    for k in want:
        assert torch.isfinite(got[k]).all() and torch.equal(got[k], want[k]), k
