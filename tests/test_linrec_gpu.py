"""The gated linear recurrence on the GPU against its fp64 oracle: prefill, backward and
decode step over layouts, types, ragged and empty sequences and odd widths.

Every output is held element by element to the largest error that 32-bit arithmetic of
the recurrence can leave (``oracle.linrec.forward_bound`` / ``backward_bound``: one
rounding at most 2^-24 of the running magnitude, decaying with the state), plus, for bf16
outputs, half a bf16 step (2^-8 of the value)."""
import numpy as np
import pytest
import torch

from gated_delta_rule_45_gb300 import kda
from oracle import linrec as ref

pytestmark = pytest.mark.gpu

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2
# roundings inside the gate and the input: fp32 gates 1 - a and (1 - a) x (2); log gates
# also expf / expm1f, at most 2 units in the last place (4 half units)
ULPS = {"channel": 2, "head": 2, "log_bf16": 6}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _case(lens, H, d, dtype, gate, S0, tail=0, mu=2.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens) + tail, len(lens)
    rn = lambda *s: torch.randn(*s, generator=g)
    c = dict(x=rn(T, H, d).to(dtype), dy=rn(T, H, d).to(dtype),
             S0=rn(N, H, d) if S0 else None, dS_T=rn(N, H, d))
    if gate == "head":
        c["a"] = torch.sigmoid(rn(T, H) + mu)
    elif gate == "channel":
        c["a"] = torch.sigmoid(rn(T, H, d) + mu)
    else:
        c["a"] = torch.nn.functional.logsigmoid(rn(T, H, d) + mu).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64) if N else np.zeros(1, np.int64)
    c["cu"] = torch.tensor(cu, dtype=torch.int32)
    c["cu_list"] = [int(v) for v in cu]
    return c


def _cuda(c):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def _within(got, want, bound, rounded=False):
    got, want = _np(got), np.asarray(want)
    # the smallest normal number: below it a rounding is absolute
    tol = np.asarray(bound) + 2.0 ** -126
    if rounded:
        tol = tol * (1 + BF16_HALF) + BF16_HALF * np.abs(want)
    off = np.abs(got - want) - tol
    assert np.isfinite(got).all()
    assert (off <= 0).all(), f"{(off > 0).sum()} of {off.size} beyond, worst by {off.max():.3g}"


def _check_prefill(c, dtype, gate, complement, saved=True, **kw):
    dev, cu = _cuda(c), c["cu_list"]
    a = ref.expand_gate(_np(c["a"]), gate, c["x"].shape)
    h, S_T = ref.forward(_np(c["x"]), a, _np(c["S0"]), cu, complement)
    _, e, e_S = ref.forward_bound(_np(c["x"]), a, _np(c["S0"]), cu, complement, ULPS[gate])
    out = kda.linrec_prefill(dev["x"], dev["a"], dev["S0"], dev["cu"], gate=gate,
                             complement=complement, save_states=saved, check_device_status=True,
                             **kw)
    torch.cuda.synchronize()
    end = cu[-1]
    _within(out[0][:end], h[:end], e[:end], rounded=dtype == torch.bfloat16)
    _within(out[1], S_T, e_S)
    if saved:
        want = ref.chunk_states(h, cu, kda.LINREC_CHUNK)
        bound = ref.chunk_states(e, cu, kda.LINREC_CHUNK)
        _within(out[2], want, bound)
    return dev, out


def _check_backward(c, dev, states, gate, complement):
    cu = c["cu_list"]
    a = ref.expand_gate(_np(c["a"]), gate, c["x"].shape)
    args = (_np(c["x"]), a, _np(c["S0"]), cu, _np(c["dy"]), _np(c["dS_T"]), complement, gate)
    want, bound = ref.backward(*args), ref.backward_bound(*args, ULPS[gate])
    got = kda.linrec_backward(dev["x"], dev["a"], dev["S0"], dev["cu"], dev["dy"], dev["dS_T"],
                              states=states, gate=gate, complement=complement,
                              check_device_status=True)
    torch.cuda.synchronize()
    end = cu[-1]
    for name in ("dx", "dgate"):
        _within(got[name][:end], want[name][:end], bound[name][:end])
    _within(got["dS0"], want["dS0"], bound["dS0"])
    return got


LENS = {
    "one_token": [1],
    "one_short": [5],
    "chunk": [128],
    "chunk_and_one": [129],
    "several_chunks": [700],
    "ragged": [3, 0, 130, 1, 0, 0, 257, 128, 64, 2],
    "all_empty": [0, 0, 0],
    "many_short": [1, 2, 0, 3, 1] * 40,
}


@pytest.mark.parametrize("gate", ["channel", "head", "log_bf16"])
@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill_and_backward(lens, dtype, gate):
    complement, S0 = lens in ("ragged", "chunk"), lens != "several_chunks"
    c = _case(LENS[lens], 2, 48, dtype, gate, S0, seed=len(lens))
    dev, out = _check_prefill(c, dtype, gate, complement)
    got = _check_backward(c, dev, out[2], gate, complement)
    again = _check_backward(c, dev, None, gate, complement)
    for name in got:   # the recomputed states are the saved ones
        assert torch.equal(got[name][:c["cu_list"][-1]] if name != "dS0" else got[name],
                           again[name][:c["cu_list"][-1]] if name != "dS0" else again[name])


@pytest.mark.parametrize("H,d", [(1, 1), (1, 2), (3, 1), (5, 67), (1, 63), (2, 65), (7, 32),
                                 (3, 64), (1, 128), (2, 256), (9, 20), (4, 31)])
@pytest.mark.parametrize("gate", ["channel", "head", "log_bf16"])
def test_widths(H, d, gate):
    for dtype in (torch.bfloat16, torch.float32):
        c = _case([70, 0, 200, 31], H, d, dtype, gate, True, seed=H * 100 + d)
        dev, out = _check_prefill(c, dtype, gate, True)
        _check_backward(c, dev, out[2], gate, True)


@pytest.mark.parametrize("H,d", [(2, 1), (64, 1), (6, 5), (2, 640), (2, 128)])
def test_head_gate_widths(H, d):
    """Heads of an odd width in rows of an even one, where a lane takes one channel; more
    partial sums a head than one thread adds up."""
    c = _case([70, 0, 300, 31, 17], H, d, torch.bfloat16, "head", True, seed=H + d)
    dev, out = _check_prefill(c, torch.bfloat16, "head", False)
    got = _check_backward(c, dev, out[2], "head", False)
    again = _check_backward(c, dev, None, "head", False)
    end = c["cu_list"][-1]
    for name in got:
        rows = slice(None) if name == "dS0" else slice(0, end)
        assert torch.equal(got[name][rows], again[name][rows])


def test_many_sequences():
    """More sequences than a CTA checks by itself, most of them empty or one token."""
    r = np.random.RandomState(0)
    lens = [int(v) for v in r.choice([0, 0, 1, 1, 2, 5], 3000)]
    c = _case(lens, 1, 40, torch.float32, "channel", True)
    dev, out = _check_prefill(c, torch.float32, "channel", False)
    _check_backward(c, dev, out[2], "channel", False)


def test_long_memory_and_fast_decay():
    """Gates near one over thousands of tokens, and gates whose product over a chunk
    underflows to zero."""
    for mu, gate in ((9.0, "channel"), (9.0, "log_bf16"), (-6.0, "channel")):
        c = _case([3000, 1000], 1, 33, torch.float32, gate, True, mu=mu, seed=3)
        dev, out = _check_prefill(c, torch.float32, gate, False)
        _check_backward(c, dev, out[2], gate, False)


def test_gates_of_zero_and_one():
    c = _case([300, 150], 1, 64, torch.float32, "channel", True, seed=4)
    z = torch.rand(c["a"].shape, generator=torch.Generator().manual_seed(1))
    c["a"][z < 0.2] = 0.0
    c["a"][z > 0.7] = 1.0
    dev, out = _check_prefill(c, torch.float32, "channel", True)
    _check_backward(c, dev, out[2], "channel", True)


def test_no_state_given_and_no_final_gradient():
    c = _case([200, 90], 2, 64, torch.bfloat16, "channel", False, seed=5)
    dev, out = _check_prefill(c, torch.bfloat16, "channel", False, saved=False)
    c["dS_T"] = dev["dS_T"] = None
    _check_backward(c, dev, None, "channel", False)


def test_tokens_past_the_end_are_left_alone():
    """NaN in the tokens behind the last sequence changes nothing, and their rows of
    every output stay as they were."""
    for tail in (1, 150, 600):
        c = _case([100, 33], 2, 48, torch.float32, "channel", True, tail=tail, seed=6)
        for k in ("x", "a", "dy"):
            c[k][133:] = float("nan")
        dev, N, T = _cuda(c), 2, 133 + tail
        y = torch.full((T, 2, 48), 7.0, device="cuda")
        S_T = torch.empty(N, 2, 48, device="cuda")
        states = torch.empty(-(-T // 128), 2, 48, device="cuda")
        ws = torch.empty(kda.linrec_workspace_size(N, T, 2, 48), dtype=torch.uint8, device="cuda")
        kda.linrec_prefill_into(dev["x"], dev["a"], dev["S0"], dev["cu"], y, S_T, ws,
                                states=states)
        kda.device_status(ws)
        cu = c["cu_list"]
        x, a = _np(c["x"][:133]), _np(c["a"][:133])
        h, S_ref = ref.forward(x, a, _np(c["S0"]), cu)
        _, e, e_S = ref.forward_bound(x, a, _np(c["S0"]), cu, False, 2)
        _within(y[:133], h, e)
        _within(S_T, S_ref, e_S)
        assert (y[133:] == 7.0).all()
        assert (states[2:] == 0).all()
        g = {n: torch.full((T, 2, 48), 7.0, device="cuda") for n in ("dx", "dgate")}
        g["dS0"] = torch.empty(N, 2, 48, device="cuda")
        for st in (states, None):
            ws = torch.empty(kda.linrec_backward_workspace_size(N, T, 2, 48, with_states=st is not None),
                             dtype=torch.uint8, device="cuda")
            kda.linrec_backward_into(dev["x"], dev["a"], dev["S0"], dev["cu"], dev["dy"],
                                     dev["dS_T"], g, ws, states=st)
            kda.device_status(ws)
            args = (x, a, _np(c["S0"]), cu, _np(c["dy"][:133]), _np(c["dS_T"]), False, "channel")
            want, bound = ref.backward(*args), ref.backward_bound(*args, 2)
            _within(g["dx"][:133], want["dx"], bound["dx"])
            _within(g["dgate"][:133], want["dgate"], bound["dgate"])
            _within(g["dS0"], want["dS0"], bound["dS0"])
            assert (g["dx"][133:] == 7.0).all() and (g["dgate"][133:] == 7.0).all()


def test_a_sequence_that_is_not_finite_stays_alone():
    """inf and NaN in one sequence's inputs, states and gradients reach no other."""
    lens = [140, 60, 200, 5, 130]
    c = _case(lens, 1, 64, torch.float32, "channel", True, seed=7)
    dev = _cuda(c)
    cu = c["cu_list"]
    clean = kda.linrec_prefill(dev["x"], dev["a"], dev["S0"], dev["cu"], save_states=True)
    gclean = kda.linrec_backward(dev["x"], dev["a"], dev["S0"], dev["cu"], dev["dy"],
                                 dev["dS_T"], states=clean[2])
    dirty = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in dev.items()}
    for n, bad in ((1, float("inf")), (3, float("nan"))):
        dirty["x"][cu[n]:cu[n + 1]] = bad
        dirty["dy"][cu[n]:cu[n + 1]] = bad
        dirty["a"][cu[n]:cu[n + 1]] = bad
        dirty["S0"][n] = bad
        dirty["dS_T"][n] = bad
    out = kda.linrec_prefill(dirty["x"], dirty["a"], dirty["S0"], dirty["cu"], save_states=True)
    g = kda.linrec_backward(dirty["x"], dirty["a"], dirty["S0"], dirty["cu"], dirty["dy"],
                            dirty["dS_T"], states=out[2])
    for n in (0, 2, 4):
        s = slice(cu[n], cu[n + 1])
        assert torch.equal(out[0][s], clean[0][s]) and torch.equal(out[1][n], clean[1][n])
        for k in ("dx", "dgate"):
            assert torch.equal(g[k][s], gclean[k][s])
        assert torch.equal(g["dS0"][n], gclean["dS0"][n])


def test_state_in_place():
    c = _case([300, 0, 45], 2, 64, torch.bfloat16, "channel", True, seed=8)
    dev = _cuda(c)
    y, S_T = kda.linrec_prefill(dev["x"], dev["a"], dev["S0"], dev["cu"])
    S, y2 = dev["S0"].clone(), torch.empty_like(dev["x"])
    ws = torch.empty(kda.linrec_workspace_size(3, 345, 2, 64), dtype=torch.uint8, device="cuda")
    kda.linrec_prefill_into(dev["x"], dev["a"], S, dev["cu"], y2, S, ws)
    torch.cuda.synchronize()
    assert torch.equal(S, S_T) and torch.equal(y2, y)


def test_same_bits_every_time():
    """A wide and long batch, where the time axis is split over CTAs that run in any order."""
    c = _case([9000, 1, 5000, 77], 4, 128, torch.bfloat16, "channel", True, seed=9)
    dev = _cuda(c)
    first = None
    for _ in range(4):
        out = kda.linrec_prefill(dev["x"], dev["a"], dev["S0"], dev["cu"], save_states=True)
        g = kda.linrec_backward(dev["x"], dev["a"], dev["S0"], dev["cu"], dev["dy"],
                                dev["dS_T"], states=out[2])
        every = list(out) + [g["dx"], g["dgate"], g["dS0"]]
        if first is None:
            first = every
        for u, v in zip(first, every):
            assert torch.equal(u, v)


def test_no_sequences_and_no_tokens():
    x, a = torch.zeros(0, 2, 64, device="cuda"), torch.zeros(0, 2, 64, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, S = kda.linrec_prefill(x, a, None, cu, check_device_status=True)
    assert y.shape == (0, 2, 64) and S.shape == (0, 2, 64)
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    S0 = torch.randn(3, 2, 64, device="cuda")
    y, S, st = kda.linrec_prefill(x, a, S0, cu, save_states=True, check_device_status=True)
    assert torch.equal(S, S0)
    g = kda.linrec_backward(x, a, S0, cu, x, S0, states=st, check_device_status=True)
    assert torch.equal(g["dS0"], S0)
    # tokens, but no sequence: nothing is written
    x = torch.randn(300, 2, 64, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, ws = torch.full_like(x, 3.0), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    kda.linrec_prefill_into(x, torch.rand_like(x), None, cu, y, S0[:0].contiguous(), ws)
    kda.device_status(ws)
    assert (y == 3.0).all()


@pytest.mark.parametrize("bad", [[1, 50, 100], [0, 60, 40, 100], [0, 50, 101], [0, -5, 100]])
@pytest.mark.parametrize("N_extra", [0, 1500])
def test_bad_offsets_write_nothing(bad, N_extra):
    bad = bad + [bad[-1]] * N_extra
    T, H, d, N = 100, 1, 64, len(bad) - 1
    x, a = torch.randn(T, H, d, device="cuda"), torch.rand(T, H, d, device="cuda")
    cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
    y, S_T = torch.full_like(x, 5.0), torch.full((N, H, d), 5.0, device="cuda")
    states = torch.full((1, H, d), 5.0, device="cuda")
    ws = torch.empty(kda.linrec_workspace_size(N, T, H, d), dtype=torch.uint8, device="cuda")
    kda.linrec_prefill_into(x, a, None, cu, y, S_T, ws, states=states)
    with pytest.raises(kda.KdaError) as e:
        kda.device_status(ws)
    assert e.value.status == kda.ERR_DEVICE_INPUT
    g = dict(dx=torch.full_like(x, 5.0), dgate=torch.full_like(x, 5.0),
             dS0=torch.full((N, H, d), 5.0, device="cuda"))
    for st in (states, None):
        wb = torch.empty(kda.linrec_backward_workspace_size(N, T, H, d, with_states=st is not None),
                         dtype=torch.uint8, device="cuda")
        kda.linrec_backward_into(x, a, None, cu, x, None, g, wb, states=st)
        with pytest.raises(kda.KdaError) as e:
            kda.device_status(wb)
        assert e.value.status == kda.ERR_DEVICE_INPUT
    for t in (y, S_T, states, *g.values()):
        assert (t == 5.0).all()
    # the same workspace serves the next call
    good = torch.tensor([0, 40, 100], dtype=torch.int32, device="cuda")
    kda.linrec_prefill_into(x, a, None, good, y, S_T[:2].contiguous(), ws)
    kda.device_status(ws)


def test_captured_and_replayed():
    """A training step captured in a graph and replayed on new inputs, with dirt left in
    the workspace between replays."""
    c = _case([700, 0, 300], 2, 64, torch.bfloat16, "head", True, seed=10)
    c2 = _case([700, 0, 300], 2, 64, torch.bfloat16, "head", True, seed=11)
    dev, T, N = _cuda(c), 1000, 3
    y, S_T = torch.empty_like(dev["x"]), torch.empty_like(dev["S0"])
    states = torch.empty(8, 2, 64, device="cuda")
    g = dict(dx=torch.empty(T, 2, 64, device="cuda"), dgate=torch.empty(T, 2, device="cuda"),
             dS0=torch.empty(N, 2, 64, device="cuda"))
    ws = torch.empty(kda.linrec_workspace_size(N, T, 2, 64), dtype=torch.uint8, device="cuda")
    wb = torch.empty(kda.linrec_backward_workspace_size(N, T, 2, 64, gate="head"),
                     dtype=torch.uint8, device="cuda")

    def step():
        kda.linrec_prefill_into(dev["x"], dev["a"], dev["S0"], dev["cu"], y, S_T, ws,
                                states=states, gate="head")
        kda.linrec_backward_into(dev["x"], dev["a"], dev["S0"], dev["cu"], dev["dy"],
                                 dev["dS_T"], g, wb, states=states, gate="head")
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for case in (c2, c):
        for k, v in _cuda(case).items():
            if isinstance(v, torch.Tensor):
                dev[k].copy_(v)
        ws.fill_(255)
        wb.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        fresh = _cuda(case)
        o = kda.linrec_prefill(fresh["x"], fresh["a"], fresh["S0"], fresh["cu"], gate="head",
                               save_states=True)
        gr = kda.linrec_backward(fresh["x"], fresh["a"], fresh["S0"], fresh["cu"], fresh["dy"],
                                 fresh["dS_T"], states=o[2], gate="head")
        for u, v in zip((y, S_T, states, g["dx"], g["dgate"], g["dS0"]),
                        (*o, gr["dx"], gr["dgate"], gr["dS0"])):
            assert torch.equal(u, v)


def test_two_streams_at_once():
    c = _case([5000, 3000], 2, 128, torch.bfloat16, "channel", True, seed=12)
    dev = _cuda(c)
    want = kda.linrec_prefill(dev["x"], dev["a"], dev["S0"], dev["cu"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [kda.linrec_prefill(dev["x"], dev["a"], dev["S0"], dev["cu"], stream=streams[i % 2])
            for i in range(6)]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


@pytest.mark.parametrize("gate", ["channel", "head", "log_bf16"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,d", [(1, 1, 1), (3, 5, 67), (37, 4, 64), (256, 2, 128)])
def test_decode_step(B, H, d, dtype, gate):
    c = _case([1] * B, H, d, dtype, gate, True, seed=B)
    dev = _cuda(c)
    a = ref.expand_gate(_np(c["a"]), gate, (B, H, d))
    for complement in (False, True):
        S = dev["S0"].clone()
        y = kda.linrec_decode_step(dev["x"], dev["a"], S, gate=gate, complement=complement)
        h, _ = ref.forward(_np(c["x"]), a, _np(c["S0"]), c["cu_list"], complement)
        _, e, _ = ref.forward_bound(_np(c["x"]), a, _np(c["S0"]), c["cu_list"], complement,
                                    ULPS[gate])
        _within(S, h, e)
        _within(y, h, e, rounded=dtype == torch.bfloat16)
        # the states of the parents, two of them outside the table
        g = torch.Generator().manual_seed(B)
        rows = 5
        table = torch.randn(rows, H, d, generator=g)
        parents = torch.randint(0, rows, (B,), generator=g, dtype=torch.int32)
        parents[0] = -1
        parents[-1] = rows if B > 1 else -1
        start = torch.zeros(B, H, d)
        ok = (parents >= 0) & (parents < rows)
        start[ok] = table[parents[ok].long()]
        S_out, tab = torch.empty(B, H, d, device="cuda"), table.cuda()
        y = kda.linrec_decode_step(dev["x"], dev["a"], tab, parents=parents.cuda(),
                                   S_out=S_out, gate=gate, complement=complement)
        h, _ = ref.forward(_np(c["x"]), a, _np(start), c["cu_list"], complement)
        _, e, _ = ref.forward_bound(_np(c["x"]), a, _np(start), c["cu_list"], complement,
                                    ULPS[gate])
        _within(S_out, h, e)
        _within(y, h, e, rounded=dtype == torch.bfloat16)
        assert torch.equal(tab.cpu(), table)


def test_decode_continues_a_prefill():
    """Prefill of 140 tokens equals prefill of 137 and three decode steps."""
    c = _case([140, 140], 2, 64, torch.float32, "channel", True, seed=13)
    dev = _cuda(c)
    y, S_T = kda.linrec_prefill(dev["x"], dev["a"], dev["S0"], dev["cu"])
    keep = torch.cat([torch.arange(137), torch.arange(140, 277)]).cuda()
    cu = torch.tensor([0, 137, 274], dtype=torch.int32, device="cuda")
    _, S = kda.linrec_prefill(dev["x"][keep], dev["a"][keep], dev["S0"], cu)
    _, e, e_S = ref.forward_bound(_np(c["x"]), _np(c["a"]), _np(c["S0"]), c["cu_list"], False, 2)
    for j in range(3):
        rows = torch.tensor([137 + j, 277 + j]).cuda()
        o = kda.linrec_decode_step(dev["x"][rows], dev["a"][rows], S)
        assert (np.abs(_np(o) - _np(y[rows])) <= 2 * e[[137 + j, 277 + j]]).all()
    assert (np.abs(_np(S) - _np(S_T)) <= 2 * e_S).all()
