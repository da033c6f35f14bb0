"""The selective scan cut along the tokens with several blocks of channels and wide states, and
batches of very different lengths, against its fp64 oracle."""
import pytest
import torch

from test_selscan_gpu import _case, _check, _cut

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,H,d,n", [([700], 1, 200, 48), ([300, 0, 500, 4], 2, 136, 16),
                                        ([600], 1, 150, 64), ([1, 800], 3, 70, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_cut_along_the_tokens_with_blocks_of_channels(lens, H, d, n, dtype):
    c = _case(lens, H, d, n, dtype, tail=3, seed=n)
    assert _cut(c)
    _check(c)


@pytest.mark.parametrize("n", [4, 16, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_long_sequence_among_short_ones(n, dtype):
    """Taken whole, as the number of sequences says."""
    _check(_case([3] * 40 + [1700] + [0, 2] * 60, 1, 40, n, dtype, seed=n))
