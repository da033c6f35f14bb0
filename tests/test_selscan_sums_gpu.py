"""Sums over many tokens in the backward pass of the selective scan."""
import numpy as np
import pytest
import torch

from gated_delta_rule_45_gb300 import kda
from layer_checks import np64, offsets

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


@pytest.mark.parametrize("n", [4, 16])
def test_sums_over_a_long_sequence(n):
    """One sequence of 30000 tokens among 151 of one token, which is not cut.  With rates of 0, no
    input to the state and a gradient of c that comes from behind, every token adds D h g = c to
    dA, c to dD and, by dD_t = A (..) + B . g x = 0, nothing to ddt_bias; c is such that a sum
    beyond 2^14 drops almost half a step of it each time.  Sums of 512 tokens, and of those 59
    and one a sequence: no more than 800 additions deep."""
    T, N, d = 30000, 152, 8
    c = 1.0 + 0.98 * 2.0 ** -10
    lens = [1] * 60 + [T] + [1] * (N - 61)
    cu, cut = offsets(lens)
    long = slice(cu[60], cu[61])
    z = lambda *s: torch.zeros(*s, device="cuda")
    x, dy = z(cu[-1], 1, d), z(cu[-1], 1, d)
    dt = z(cu[-1], 1, d)
    dt[long] = 1.0
    x[long], dy[long] = 1.0, c
    S0, dS = z(N, 1, d, n), z(N, 1, d, n)
    S0[60], dS[60] = 1.0, c
    g = kda.selscan_backward(x, dt, z(1, d, n), z(cu[-1], 1, n), z(cu[-1], 1, n), S0, cut.cuda(), dy,
                             dS, D=z(1, d), dt_bias=z(1, d), softplus=False)
    want = T * float(torch.tensor(c, dtype=torch.float32))
    for k in ("dA", "dD"):
        off = np.abs(np64(g[k]) / want - 1.0).max()
        assert off <= 800 * U32, (k, off / U32)
    assert (g["ddt_bias"] == 0).all()
