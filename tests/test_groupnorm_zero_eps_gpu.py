"""The gated group norm with an eps of 0, which only a head without deviations turns into NaN:
every gradient, where warps hold several tokens and the last ones lack some."""
import pytest
import torch

from test_groupnorm_gpu import _case, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,d", [(33, 1, 64), (5, 1, 128), (7, 3, 8), (1, 2, 16), (131, 1, 24),
                                   (3, 5, 67), (9, 1, 256), (3, 1, 2048)])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_without_an_eps(T, H, d, center, dtype):
    for z in (False, True):
        for act in ("none", "silu", "sigmoid"):
            _check(_case(T, H, d, dtype, z, "shared" if z else "head", seed=d), act, center, 0.0)
