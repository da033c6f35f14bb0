"""The gated group norm on the GPU against its fp64 oracle: forward and backward over widths,
types, activations, gates and parameters.  Every output is held to the largest error that 32-bit
arithmetic can leave (``oracle.groupnorm``)."""
import pytest
import torch

from gated_delta_rule_45_gb300 import kda
from layer_checks import cuda, np64, wide_rows, within
from oracle import groupnorm as ref

pytestmark = pytest.mark.gpu


def _case(T, H, d, dtype, z=True, par="shared", bias=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    shape = (d,) if par == "shared" else (H, d)
    return dict(x=(rn(T, H, d) * torch.exp(rn(T, H, 1)) + 0.4).to(dtype),
                z=rn(T, H, d).to(dtype) if z else None, dy=rn(T, H, d).to(dtype),
                w=1 + 0.3 * rn(*shape) if par != "none" else None,
                b=0.3 * rn(*shape) if bias and par != "none" else None)


def _check(c, act="silu", center=False, eps=1e-5, x=None, z=None):
    dev = cuda(c)
    x, z = dev["x"] if x is None else x, dev["z"] if z is None else z
    kw = dict(z=z, act=act, eps=eps, center=center)
    y = kda.groupnorm_forward(x, dev["w"], dev["b"], **kw)
    got = kda.groupnorm_backward(x, dev["w"], dev["b"], dev["dy"], **kw)
    torch.cuda.synchronize()
    ins = [np64(c[k]) for k in ("x", "w", "b", "z")]
    wy, ey = ref.forward(*ins, act, center, eps)
    within("y", y, wy, ey, c["x"].dtype == torch.bfloat16)
    want, err = ref.backward(*ins, act, center, eps, np64(c["dy"]))
    assert set(got) == set(want)
    for k in got:
        within(k, got[k], want[k], err[k])
    return y, got


@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forms(dtype, center, z, act):
    for par in ("shared", "head", "none"):
        _check(_case(19, 3, 64, dtype, z, par, bias=par == "head"), act, center)


@pytest.mark.parametrize("T,H,d", [(1, 1, 1), (5, 1, 2), (3, 4, 3), (40, 40, 8), (7, 2, 67),
                                   (9, 5, 100), (6, 3, 128), (300, 1, 256), (4, 2, 320),
                                   (3, 2, 512), (3, 1, 1000), (2, 3, 1024), (3, 1, 1025),
                                   (2, 2, 2048), (2, 1, 8192), (2, 1, 16384), (1, 1, 16383)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_widths(T, H, d, dtype):
    _check(_case(T, H, d, dtype, seed=d), "silu", center=d % 2 == 1 and d > 1)
    _check(_case(T, H, d, dtype, z=False, par="head", seed=d), "sigmoid", center=d > 2)


@pytest.mark.parametrize("left,right", [(32, 32), (8, 0), (1, 2)])
@pytest.mark.parametrize("d", [64, 2048])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_rows(left, right, d, dtype):
    c = _case(21, 2, d, dtype, seed=3)
    y, g = _check(c, x=wide_rows(c["x"].cuda(), left, right))
    y2, g2 = _check(c, z=wide_rows(c["z"].cuda(), right, left))
    _check(c)
    assert torch.isfinite(y.float()).all() and torch.isfinite(y2.float()).all()


def test_many_tokens_of_few_heads():
    """More tokens than the parameters' gradients have partial sums."""
    _check(_case(3000, 2, 16, torch.float32, par="head", seed=1), center=True)
    _check(_case(1500, 1, 4, torch.bfloat16, seed=2))


def test_no_tokens():
    c = cuda(_case(0, 2, 16, torch.bfloat16))
    assert kda.groupnorm_forward(c["x"], c["w"], c["b"], z=c["z"]).shape == (0, 2, 16)
    g = kda.groupnorm_backward(c["x"], c["w"], c["b"], c["dy"], z=c["z"])
    assert (g["dw"] == 0).all() and (g["db"] == 0).all() and g["dx"].shape == (0, 2, 16)


def test_constant_rows_and_large_means():
    c = _case(6, 2, 64, torch.float32, z=False, seed=4)
    c["x"][0] = 3.0                    # no deviation at all
    c["x"][1] = 0.0
    c["x"][2] += 1000.0                # deviations far below the mean
    _check(c, "none", center=True, eps=1e-3)
    _check(c, "none", center=False, eps=1e-3)


@pytest.mark.parametrize("d", [64, 2048])
def test_in_place_and_values_stay_in_their_row(d):
    c = cuda(_case(40, 2, d, torch.bfloat16, seed=5))
    y = kda.groupnorm_forward(c["x"], c["w"], c["b"], z=c["z"])
    bad = c["x"].clone()
    bad[7, 1] = float("nan")
    y2 = kda.groupnorm_forward(bad, c["w"], c["b"], z=c["z"])
    keep = torch.ones(40, 2, dtype=torch.bool)
    keep[7, 1] = False
    assert torch.equal(y[keep], y2[keep]) and torch.isnan(y2[7, 1].float()).all()
    for name in ("x", "z"):
        t = dict(c, x=c["x"].clone(), z=c["z"].clone())
        out = kda.groupnorm_forward(t["x"], c["w"], c["b"], t[name], z=t["z"])
        assert out is t[name] and torch.equal(out, y)


def test_gradients_of_the_parameters_alone_or_not_at_all():
    c = cuda(_case(50, 3, 32, torch.float32, par="head", seed=6))
    g = kda.groupnorm_backward(c["x"], c["w"], c["b"], c["dy"], z=c["z"])
    out = dict(dx=torch.empty_like(g["dx"]))
    kda.groupnorm_backward_into(c["x"], c["w"], c["b"], c["dy"], out, None, z=c["z"])
    assert torch.equal(out["dx"], g["dx"])
    ws = torch.empty(kda.groupnorm_backward_workspace_size(50, 3, 32), dtype=torch.uint8,
                     device="cuda")
    out["db"] = torch.empty(3, 32, device="cuda")
    kda.groupnorm_backward_into(c["x"], c["w"], c["b"], c["dy"], out, ws, z=c["z"])
    assert torch.equal(out["db"], g["db"])


def test_captured_on_another_stream_with_the_same_bits():
    c = cuda(_case(500, 4, 128, torch.bfloat16, seed=7))
    y = kda.groupnorm_forward(c["x"], c["w"], c["b"], z=c["z"], center=True)
    g = kda.groupnorm_backward(c["x"], c["w"], c["b"], c["dy"], z=c["z"], center=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y2 = kda.groupnorm_forward(c["x"], c["w"], c["b"], z=c["z"], center=True)
        g2 = kda.groupnorm_backward(c["x"], c["w"], c["b"], c["dy"], z=c["z"], center=True)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in g)
