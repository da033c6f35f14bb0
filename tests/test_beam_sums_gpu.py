"""The selection's log-sum-exp on the GPU, held to what ``include/beam.h`` states of it, and
the order of candidates of different beams, which depends on it.

A piece's sum is of terms 2^(x log2 e - c).  A term is off, relatively, by 2^-22 for the
special-function unit, by half a unit in the last place of its argument (times ln 2), and by
1.34e-8 of |x - M| for log2 e in fp32; in the sum each counts by its share.  (A fixed 2e-7
is not enough: bf16 logits around -100 lie half a unit apart, so thousands of terms have one
argument and err together, by up to 1.4e-7 + 1.65e-7 at 2.8 to 5.5 below the maximum.)  The
additions' roundings are independent over a thousand accumulators of up to 64 terms: sqrt(64 /
1024) 2^-24, six times that at most, and 14 more join those, sqrt(14) 2^-24: together below
6 x 2^-24.  ``_lse_err`` adds these up for a row.  The reference is the maximum of the part of
the row seen first, at most REF below the row's own here, so that arguments of terms above it
are as large as REF.  A value is rounded to fp32 once more (2^-24 of it)."""
import numpy as np
import pytest
import torch

from gated_delta_rule_45_gb300 import kda
from oracle import beam as ref

pytestmark = pytest.mark.gpu

F32_HALF = 2.0 ** -24
REF = 4.0


def _lse_err(x, rising=False):
    """Largest error of the log-sum-exp of each row [rows, V], as above: [rows, 1].  Where
    later parts lie far above the first (`rising`), arguments are as large as 32, 22 below
    or above the reference, or the sums are scaled to new references, each time by one more
    exponential.  Those rows have equal terms, whose additions round alike in all threads:
    the sums are in pairs (exact then), but for 8 vectors of a part, of which the 3rd, 5th
    .. 8th addition round, by 2^-24 of 3/8, 5/8 .. 8/8 of the result (3.6), up to 8 parts
    (as much) and two last factors: 10 x 2^-24 in all, 4 more."""
    ref = 22.0 if rising else REF
    big = np.finfo(np.float32).max
    x = np.minimum(np.where(np.isnan(x), -np.inf, x), big)
    top = x.max(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        below = np.where(x == top, 0.0, np.where(x == -np.inf, np.inf, top - x))
    share = np.exp(-below)
    share /= share.sum(-1, keepdims=True)
    near = np.minimum(below, 200.0)
    far = np.maximum(near, ref)
    arg = (far / np.log(2)).astype(np.float32)
    term = 2.0 ** -22 + np.log(2) * np.spacing(arg).astype(np.float64) / 2 + 1.34e-8 * far
    if rising:
        term += (np.floor(near / 4) + 1) * 2.0 ** -22
        term += 4 * F32_HALF
    return (share * term).sum(-1, keepdims=True) + 6 * F32_HALF


def _np(t):
    return t.detach().double().cpu().numpy()


def _check(logits, scores, n, rising=False):
    err = _lse_err(_np(logits), rising).reshape(scores.shape).max(-1, keepdims=True)
    assert err.max() < (3e-6 if rising else 1e-6)   # as the header states
    vals, par, tok = ref.select(_np(logits), _np(scores), n)
    s, p, t = kda.beam_select(logits.cuda(), scores.cuda(), n)
    torch.cuda.synchronize()
    s = _np(s)
    np.testing.assert_array_equal(p.cpu().numpy(), par)
    np.testing.assert_array_equal(t.cpu().numpy(), tok)
    assert np.array_equal(np.isneginf(s), np.isneginf(vals))
    ok = np.isfinite(vals)
    vals[~ok] = s[~ok] = 0.0
    off = np.abs(s - vals)[ok] - (err + F32_HALF * np.abs(vals))[ok]
    assert (off <= 0).all(), f"worst by {off.max():.3g} beyond {err.max():.3g}"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [-1e4, -1000.0, -100.0, 0.0, 30.0, 100.0, 1000.0, 1e4, 1e6])
def test_rows_around(offset, dtype):
    """Logits far from zero: requests of one beam, so that the order is that of the logits."""
    g = torch.Generator().manual_seed(int(abs(offset)) + 1)
    for rows, V in ((12, 32000), (300, 5000), (3, 130001)):
        z = (torch.randn(rows, V, generator=g) * 3 + offset).to(dtype)
        _check(z, -0.5 * torch.rand(rows, 1, generator=g), 8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [30.0, 300.0, 3e4])
def test_wide_rows(scale, dtype):
    """Logits far apart: the largest stands nearly alone."""
    g = torch.Generator().manual_seed(int(scale))
    z = (torch.randn(16, 32000, generator=g) * scale).to(dtype)
    _check(z, -0.5 * torch.rand(16, 1, generator=g), 8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_token(dtype):
    """A row of one logit has the value of its score, whatever the logit is."""
    z = torch.tensor([0.0, -0.0, 1e-6, 0.3, 7.7, -20.1, 33.3, -100.7, 1000.3, 12345.6, -1e6,
                      3e7, -1e30, 3e38]).to(dtype)[:, None]
    _check(z, torch.linspace(-1, 0, z.shape[0])[:, None].contiguous(), 1)


@pytest.mark.parametrize("shift", [5.0, 37.0, 100.5, 1000.0, -333.25])
def test_order_of_beams_that_differ_by_a_constant(shift):
    """The second beam has the first one's logits and a constant, which its normaliser takes
    out again, and a score 2^-20 better: its candidate of each logit comes first."""
    for seed, V in ((0, 32000), (1, 129000), (2, 700)):
        g = torch.Generator().manual_seed(seed)
        z = (torch.randn(1, V, generator=g) * 3 * 64).round() / 64
        sc = torch.tensor([[-0.25 - 2.0 ** -20, -0.25]])
        _check(torch.cat([z, z + shift]), sc, 32)
        _check(torch.cat([z + shift, z]), sc, 32)


# Tokens far above the rest of their row, behind the part of it that is seen first.  The sums
# stay relative to what is near the largest logit.
FAR = [10.0, 20.0, 21.5, 27.0, 40.0, 80.0, 88.5, 120.0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("above", FAR)
def test_tokens_far_above_the_first_ones(above, dtype):
    """A row's fill of -100 and two allowed tokens, each in another piece of the row."""
    rows, V = 256, 128000
    z = torch.full((rows, V), -100.0)
    z[:, 40000], z[:, 100000] = -100.0 + above, -100.0 + above
    z[7, 100000] += 0.25
    z[9, 3] = -100.0 + above           # one more, seen first
    z[11, 40000:40400] = -100.0 + above
    z[13, 5000:125000:97] += above / 2     # some in every part, on the way up
    _check(z.to(dtype), torch.zeros(rows, 1), 4, rising=True)
    if above < 100:
        # logits that differ, so that few of them are listed; two sums of e^88.5 overflow
        g = torch.Generator().manual_seed(int(above))
        z = torch.minimum(z, z - torch.rand(rows, V, generator=g).round(decimals=2))
        z[:, 40000], z[:, 100000] = -100.0 + above, -100.0 + above
        _check(z.to(dtype), torch.zeros(rows, 1), 4, rising=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rising_rows(dtype):
    """Logits that rise along the row, so that each part lies above the ones before, and a
    few steps of it, from a fill as low as the type has."""
    V = 100003
    ramp = torch.linspace(-60, 60, V)
    steps = torch.full((V,), torch.finfo(torch.float32).min)
    steps[30000:] = -1e4
    steps[70000:] = 5.0
    steps[99000:] = 25.5
    _check(torch.stack([ramp, -ramp, 3 * ramp, steps, steps.flip(0)]).to(dtype),
           torch.zeros(5, 1), 16, rising=True)
