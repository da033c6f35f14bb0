"""The short causal convolution on the GPU against its fp64 oracle: prefill, backward and decode
step over widths, types, ragged and empty sequences, strided rows and odd channels.  Every output
is held to the largest error that 32-bit arithmetic can leave (``oracle.causalconv``)."""
import numpy as np
import pytest
import torch

from gated_delta_rule_45_gb300 import kda
from layer_checks import LENS, cuda, np64, offsets, wide_rows, within
from oracle import causalconv as ref

pytestmark = pytest.mark.gpu


def _case(lens, ch, W, dtype, bias=True, S0=True, tail=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    cu, cut = offsets(lens)
    T, N = cu[-1] + tail, len(lens)
    return dict(x=rn(T, *ch).to(dtype), w=rn(*ch, W) * 0.5, b=rn(*ch) if bias else None,
                S0=rn(N, W - 1, *ch).to(dtype) if S0 else None, dy=rn(T, *ch).to(dtype),
                dS_T=rn(N, W - 1, *ch), cu=cut, cu_list=cu)


def _flat(c):
    D = int(np.prod(c["w"].shape[:-1]))
    W = c["w"].shape[-1]
    f = lambda t, *s: None if t is None else np64(t).reshape(*s)
    return dict(x=f(c["x"], -1, D) if c["x"].numel() else np.zeros((0, D)), w=f(c["w"], D, W),
                b=f(c["b"], D), S0=f(c["S0"], -1, W - 1, D),
                dy=f(c["dy"], -1, D) if c["dy"].numel() else np.zeros((0, D)),
                dS_T=f(c["dS_T"], -1, W - 1, D))


def _check(c, silu=True, x=None):
    dev, f, cu = cuda(c), _flat(c), c["cu_list"]
    x = dev["x"] if x is None else x
    end, D = cu[-1], f["w"].shape[0]
    bf = c["x"].dtype == torch.bfloat16
    y, S_T = kda.causalconv_prefill(x, dev["w"], dev["b"], dev["S0"], dev["cu"], silu=silu,
                                    check_device_status=True)
    wy, wS, ey = ref.forward(f["x"], f["w"], f["b"], f["S0"], cu, silu)
    torch.cuda.synchronize()
    within("y", y.reshape(-1, D)[:end], wy[:end], ey[:end], bf)
    assert (np64(S_T).reshape(wS.shape) == wS).all()
    got = kda.causalconv_backward(x, dev["w"], dev["b"], dev["S0"], dev["cu"], dev["dy"],
                                  dev["dS_T"], silu=silu, check_device_status=True)
    want, err = ref.backward(f["x"], f["w"], f["b"], f["S0"], cu, f["dy"], f["dS_T"], silu)
    torch.cuda.synchronize()
    within("dx", got["dx"].reshape(-1, D)[:end], want["dx"][:end], err["dx"][:end])
    for k in ("dw", "dS0") + (("db",) if c["b"] is not None else ()):
        within(k, got[k].reshape(want[k].shape), want[k], err[k])
    return dev, y, S_T, got


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill_and_backward(lens, dtype, W):
    _check(_case(LENS[lens], (2, 36), W, dtype, bias=W != 3, S0=lens != "ragged", seed=W),
           silu=lens != "tile")


@pytest.mark.parametrize("ch", [(1,), (2,), (3,), (5, 7), (4, 33), (1030,), (8, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_widths(ch, dtype):
    _check(_case([40, 0, 3, 61], ch, 4, dtype, tail=5, seed=len(ch)))


@pytest.mark.parametrize("left,right", [(64, 0), (8, 24), (1, 0), (3, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_rows(left, right, dtype):
    c = _case([33, 2, 90], (64,), 4, dtype, seed=left)
    _, y, S_T, g = _check(c, x=wide_rows(c["x"].cuda(), left, right))
    dev, y2, S2, g2 = _check(c)
    assert torch.equal(y, y2) and torch.equal(S_T, S2)
    assert all(torch.equal(g[k], g2[k]) for k in g)


@pytest.mark.parametrize("lens", [[], [0 if i % 3 else 2 for i in range(1500)]])
def test_many_and_no_sequences(lens):
    """More sequences than a CTA checks by itself, and tokens that belong to none."""
    _check(_case(lens, (12,), 4, torch.float32, tail=9, seed=2))


def test_no_rows():
    c = cuda(_case([], (12,), 4, torch.bfloat16))
    y = kda.causalconv_decode_step(c["x"], c["w"], c["b"], c["S0"])
    assert y.shape == (0, 12)


def test_extreme_values():
    c = _case([50], (8,), 4, torch.float32, seed=3)
    c["x"] *= 60.0      # arguments of silu from -300 to 300
    _check(c)


def test_long_batch_in_runs():
    """More runs than the gradients' partial sums may have rows, so that runs get longer."""
    c = _case([70000, 1, 30000], (2,), 4, torch.float32, seed=5)
    dev, f = cuda(c), _flat(c)
    got = kda.causalconv_backward(dev["x"], dev["w"], dev["b"], dev["S0"], dev["cu"], dev["dy"],
                                  dev["dS_T"], check_device_status=True)
    x = f["x"]
    win = np.zeros((x.shape[0], 4, 2))
    for n, (a, e) in enumerate(zip(c["cu_list"], c["cu_list"][1:])):
        full = np.concatenate([f["S0"][n], x[a:e]])
        for j in range(4):
            win[a:e, j] = full[j:j + e - a]
    v = np.einsum("twd,dw->td", win, f["w"]) + f["b"]
    dv = f["dy"] * ref.silu_grad(v)
    mag = np.abs(dv)[:, None] * np.abs(win)
    # each sum: 50 tokens in a run, 2048 / 8 runs a thread, 8 threads; its terms 40 roundings
    tol = 500 * ref.U32
    assert (np.abs(np64(got["dw"]) - np.einsum("td,twd->dw", dv, win)) <=
            tol * mag.sum(0).T).all()
    assert (np.abs(np64(got["db"]) - dv.sum(0)) <= tol * np.abs(dv).sum(0) +
            40 * ref.U32 * np.abs(f["dy"]).sum(0)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_state_carries_over_and_in_place(dtype):
    """Two halves give what the whole does; S_T in the place of S0."""
    c = cuda(_case([37, 0, 64, 2], (12,), 4, dtype, seed=8))
    y, S_T = kda.causalconv_prefill(c["x"], c["w"], c["b"], c["S0"], c["cu"])
    cut = [20, 0, 1, 2]
    S = c["S0"].clone()
    parts = [[], []]
    at = c["cu_list"]
    for half in (0, 1):
        rows = [slice(a, a + k) if half == 0 else slice(a + k, e)
                for a, e, k in zip(at, at[1:], cut)]
        x = torch.cat([c["x"][r] for r in rows])
        _, cu = offsets([r.stop - r.start for r in rows])
        yh = torch.empty_like(x)
        ws = torch.empty(kda.causalconv_workspace_size(4, x.shape[0], 12, 4, dtype),
                         dtype=torch.uint8, device="cuda")
        kda.causalconv_prefill_into(x, c["w"], c["b"], S, cu.cuda(), yh, S, ws)
        parts[half] = torch.split(yh, [r.stop - r.start for r in rows])
    joined = torch.cat([torch.cat([a, b]) for a, b in zip(*parts)])
    assert torch.equal(joined, y) and torch.equal(S, S_T)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("ch", [(3,), (64,), (4, 33)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_steps_are_the_prefill(dtype, ch, W):
    B, steps = 5, 6
    c = cuda(_case([steps] * B, ch, W, dtype, seed=W))
    y, S_T = kda.causalconv_prefill(c["x"], c["w"], c["b"], c["S0"], c["cu"])
    x = c["x"].reshape(B, steps, *ch)
    S = c["S0"].clone()
    for t in range(steps):
        yt = kda.causalconv_decode_step(wide_rows(x[:, t].contiguous(), 8, 8), c["w"], c["b"], S)
        assert torch.equal(yt, y.reshape(B, steps, *ch)[:, t])
    assert torch.equal(S, S_T)


def test_decode_parents():
    c = cuda(_case([1] * 6, (24,), 4, torch.bfloat16, seed=1))
    par = torch.tensor([0, 0, 5, -1, 6, 2], dtype=torch.int32, device="cuda")
    S_out = torch.empty_like(c["S0"])
    y = kda.causalconv_decode_step(c["x"], c["w"], c["b"], c["S0"], parents=par, S_out=S_out)
    S = torch.stack([c["S0"][p] if 0 <= p < 6 else torch.zeros_like(c["S0"][0])
                     for p in par.tolist()])
    want = kda.causalconv_decode_step(c["x"], c["w"], c["b"], S)
    assert torch.equal(y, want) and torch.equal(S_out, S)


def test_rows_behind_the_last_sequence_are_left():
    c = cuda(_case([5, 9], (16,), 4, torch.bfloat16, tail=20, seed=2))
    c["x"][14:], c["dy"][14:] = float("nan"), float("nan")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    y = torch.full_like(c["x"], 7.0)
    S_T = torch.empty_like(c["S0"])
    kda.causalconv_prefill_into(c["x"], c["w"], c["b"], c["S0"], c["cu"], y, S_T, ws)
    assert (y[14:] == 7.0).all() and torch.isfinite(y.float()).all()
    grads = dict(dx=torch.full((34, 16), 7.0, device="cuda"), dw=torch.empty(16, 4, device="cuda"),
                 db=torch.empty(16, device="cuda"), dS0=torch.empty(2, 3, 16, device="cuda"))
    kda.causalconv_backward_into(c["x"], c["w"], c["b"], c["S0"], c["cu"], c["dy"], c["dS_T"],
                                 grads, ws)
    assert (grads["dx"][14:] == 7.0).all()
    assert all(torch.isfinite(g).all() for g in grads.values())


def test_values_stay_in_their_sequence():
    c = cuda(_case([20, 20, 20], (16,), 4, torch.float32, seed=4))
    y, _ = kda.causalconv_prefill(c["x"], c["w"], c["b"], c["S0"], c["cu"])
    g = kda.causalconv_backward(c["x"], c["w"], c["b"], c["S0"], c["cu"], c["dy"], c["dS_T"])
    c["x"][20:40], c["S0"][1], c["dy"][20:40], c["dS_T"][1] = (float("nan"),) * 4
    y2, _ = kda.causalconv_prefill(c["x"], c["w"], c["b"], c["S0"], c["cu"])
    g2 = kda.causalconv_backward(c["x"], c["w"], c["b"], c["S0"], c["cu"], c["dy"], c["dS_T"])
    for a, b in ((y, y2), (g["dx"], g2["dx"])):
        assert torch.equal(a[:20], b[:20]) and torch.equal(a[40:], b[40:])


@pytest.mark.parametrize("lens", [[4, 4], [2] * 1500])
def test_malformed_offsets_write_nothing(lens):
    c = cuda(_case(lens, (16,), 4, torch.float32, seed=6))
    cu = c["cu"].clone()
    cu[1] = cu[2] + 1
    N, ws = len(lens), torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    y, S_T = torch.full_like(c["x"], 7.0), torch.full_like(c["S0"], 7.0)
    kda.causalconv_prefill_into(c["x"], c["w"], c["b"], c["S0"], cu, y, S_T, ws)
    with pytest.raises(kda.KdaError):
        kda.device_status(ws)
    grads = dict(dx=torch.full_like(c["dy"], 7.0), dw=torch.full_like(c["w"], 7.0),
                 db=torch.full_like(c["b"], 7.0), dS0=torch.full_like(c["dS_T"], 7.0))
    kda.causalconv_backward_into(c["x"], c["w"], c["b"], c["S0"], cu, c["dy"], c["dS_T"], grads, ws)
    with pytest.raises(kda.KdaError):
        kda.device_status(ws)
    torch.cuda.synchronize()
    for t in (y, S_T, *grads.values()):
        assert (t == 7.0).all()
    kda.causalconv_prefill_into(c["x"], c["w"], c["b"], c["S0"], c["cu"], y, S_T, ws)
    kda.device_status(ws)


def test_captured_on_another_stream_with_the_same_bits():
    c = cuda(_case([300, 5, 77], (64,), 4, torch.bfloat16, seed=9))
    args = (c["x"], c["w"], c["b"], c["S0"], c["cu"])
    y, S_T = kda.causalconv_prefill(*args)
    g = kda.causalconv_backward(*args, c["dy"], c["dS_T"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y2, S2 = kda.causalconv_prefill(*args)
        g2 = kda.causalconv_backward(*args, c["dy"], c["dS_T"])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(S_T, S2)
    assert all(torch.equal(g[k], g2[k]) for k in g)
    y3, _ = kda.causalconv_prefill(*args, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, y3)
