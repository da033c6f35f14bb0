"""Gradients of the parameters of the operators around a layer's recurrence, held closely enough to
64 bits that a token left out, or taken twice, shows: sums are allowed as many roundings as the
kernels make additions in a row, not as many as there are terms."""
import numpy as np
import pytest
import torch

from gated_delta_rule_45_gb300 import kda
from layer_checks import cuda, np64
from oracle import causalconv as conv_ref
from oracle import groupnorm as norm_ref
from test_causalconv_gpu import _case as conv_case
from test_causalconv_gpu import _flat
from test_groupnorm_gpu import _case as norm_case

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


# Additions in a row: a lane's tokens (at most 1024 rows of sums a head), every eighth row of a column
# (of all heads where they share the weights), the eight, and up to 8 pairs and vectors.
@pytest.mark.parametrize("T,H,d,par,deep", [(3000, 2, 16, "head", 3 + 128 + 16),
                                            (5000, 1, 64, "shared", 5 + 128 + 16),
                                            (4000, 4, 128, "shared", 4 + 512 + 16),
                                            (3000, 1, 2048, "shared", 3 + 128 + 16),
                                            (2500, 3, 67, "head", 3 + 128 + 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_parameters(T, H, d, par, deep, dtype):
    c = norm_case(T, H, d, dtype, par=par, seed=d)
    dev = cuda(c)
    got = kda.groupnorm_backward(dev["x"], dev["w"], dev["b"], dev["dy"], z=dev["z"])
    x, w, b, z, dy = (np64(c[k]) for k in ("x", "w", "b", "z", "dy"))
    want, err = norm_ref.backward(x, w, b, z, "silu", False, 1e-5, dy)
    dv = dy * conv_ref.silu(z)
    xh = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
    over = (0, 1) if par == "shared" else (0,)
    for k, term in (("dw", dv * xh), ("db", dv)):
        tol = err[k] - (T * H - deep) * U32 * np.abs(term).sum(over)
        assert (tol > 0).all() and (np.abs(np64(got[k]) - want[k]) <= tol).all(), k


@pytest.mark.parametrize("lens", [[3000], [700, 0, 1, 1500, 900]])
@pytest.mark.parametrize("W", [2, 4])
def test_convolution_parameters(lens, W):
    """A run of 32 tokens, every eighth of some 100 runs, the eight."""
    c = conv_case(lens, (12,), W, torch.float32, seed=W)
    dev, f, cu, deep = cuda(c), _flat(c), c["cu_list"], 32 + 13 + 8
    got = kda.causalconv_backward(dev["x"], dev["w"], dev["b"], dev["S0"], dev["cu"], dev["dy"],
                                  dev["dS_T"])
    want, err = conv_ref.backward(f["x"], f["w"], f["b"], f["S0"], cu, f["dy"], f["dS_T"])
    win, _ = conv_ref._history(f["x"], f["S0"], cu, W)
    dv = np.abs(f["dy"] * conv_ref.silu_grad(np.einsum("twd,dw->td", win, f["w"]) + f["b"]))
    for k, mag in (("dw", np.einsum("td,twd->dw", dv, np.abs(win))), ("db", dv.sum(0))):
        tol = err[k] - (cu[-1] + 16 - deep) * U32 * mag
        assert (tol > 0).all() and (np.abs(np64(got[k]) - want[k]) <= tol).all(), k


# ---- where offsets pass 32 bits: terms of one sign, summed in 64 bits a piece at a time

BIG = 600_000
PIECE = 20_000


@pytest.fixture
def room():
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB")
    yield
    torch.cuda.empty_cache()


def _positive(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(*shape, device="cuda", generator=g, dtype=torch.bfloat16)


def _sum64(f):
    return sum(f(slice(t, t + PIECE)) for t in range(0, BIG, PIECE))


def _relative(got, want, tol):
    off = float((got.double() / want - 1.0).abs().max())
    assert off <= tol * U32, off / U32


def test_large_convolution(room):
    """Runs of 512 tokens, 1172 of them."""
    D = 4096
    x, dy = _positive(1, BIG, D), _positive(2, BIG, D)
    cu = torch.tensor([0, BIG], dtype=torch.int32, device="cuda")
    w, b = torch.ones(D, 4, device="cuda"), torch.zeros(D, device="cuda")
    g = kda.causalconv_backward(x, w, b, None, cu, dy, silu=False)
    for k in range(4):
        def term(s):
            to = slice(max(s.start, k), s.stop)
            return (dy[to].double() * x[to.start - k:to.stop - k].double()).sum(0)
        _relative(g["dw"][:, 3 - k], _sum64(term), 512 + 147 + 16)
    _relative(g["db"], _sum64(lambda s: dy[s].double().sum(0)), 512 + 147 + 16)


@pytest.mark.parametrize("shared", [False, True])
def test_large_norm(room, shared):
    """A lane's 1974 tokens, every eighth of 304 rows (of 32 heads); each value's norm has 16
    roundings."""
    H, d = 32, 128
    x, dy = _positive(3, BIG, H, d), _positive(4, BIG, H, d)
    w = torch.ones(d, device="cuda") if shared else torch.ones(H, d, device="cuda")
    g = kda.groupnorm_backward(x, w, None, dy, act="none", eps=1e-5)

    def term(s):
        v = x[s].double()
        v = dy[s].double() * v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5)
        return v.sum((0, 1) if shared else 0)
    _relative(g["dw"], _sum64(term), 1974 + (1216 if shared else 38) + 32)


@pytest.mark.parametrize("lens", [[BIG], [1000] * (BIG // 1000)])
def test_large_scan(room, lens):
    """Rates of 0 and no way to or from the states: h and its gradient are 1 at every token, which
    adds its step to dA and dy x to dD.  Sums of 512 tokens, some 60 of them, and of every eighth of
    up to 600 segments."""
    D, n, N = 4096, 4, len(lens)
    x, dt, dy = (_positive(s, BIG, 1, D) for s in (5, 6, 7))
    zero = torch.zeros(BIG, 1, n, device="cuda", dtype=torch.bfloat16)
    cu = torch.arange(0, BIG + 1, lens[0], dtype=torch.int32, device="cuda")
    one = torch.ones(N, 1, D, n, device="cuda")
    g = kda.selscan_backward(x, dt, torch.zeros(1, D, n, device="cuda"), zero, zero, one, cu, dy, one,
                             D=torch.zeros(1, D, device="cuda"), softplus=False)
    steps = _sum64(lambda s: dt[s].double().sum(0))
    _relative(g["dA"], steps[..., None].expand(1, D, n), 512 + 62 + 75 + 32)
    _relative(g["dD"], _sum64(lambda s: (dy[s].double() * x[s].double()).sum(0)), 512 + 62 + 75 + 32)
