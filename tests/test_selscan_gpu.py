"""The selective scan on the GPU against its fp64 oracle: prefill, backward and decode step over
state sizes, groups, types, ragged and empty sequences, strided rows and cuts along the tokens.
Every output is held to the largest error that 32-bit arithmetic can leave
(``oracle.selscan``)."""
import numpy as np
import pytest
import torch

from gated_delta_rule_45_gb300 import kda
from layer_checks import LENS, cuda, np64, offsets, wide_rows, within
from oracle import selscan as ref

pytestmark = pytest.mark.gpu


def _case(lens, H, d, n, dtype, z=True, D=True, bias=True, S0=True, softplus=True, tail=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    cu, cut = offsets(lens)
    T, N = cu[-1] + tail, len(lens)
    return dict(x=rn(T, H, d).to(dtype),
                dt=(rn(T, H, d) - 1.0 if softplus else rn(T, H, d).abs() * 0.3).to(dtype),
                A=-torch.exp(rn(H, d, n)), B=rn(T, H, n).to(dtype), C=rn(T, H, n).to(dtype),
                D=rn(H, d) if D else None, z=rn(T, H, d).to(dtype) if z else None,
                dt_bias=0.3 * rn(H, d) if bias else None, S0=rn(N, H, d, n) if S0 else None,
                dy=rn(T, H, d).to(dtype), dS_T=rn(N, H, d, n), cu=cut, cu_list=cu,
                softplus=softplus)


def _oracle(c):
    keys = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "S0", "dy", "dS_T")
    return dict({k: np64(c[k]) for k in keys}, cu=c["cu_list"], softplus=c["softplus"])


def _kw(c):
    return dict(D=c["D"], z=c["z"], dt_bias=c["dt_bias"], softplus=c["softplus"])


def _ins(c):
    return tuple(c[k] for k in ("x", "dt", "A", "B", "C", "S0", "cu"))


def _representable(o):
    """Channels [H, d] whose values have a place in 32 bits.  A linear step may be negative, and
    then a decay is above 1: with rates of -exp(N(0, 1)) and steps of 0.3 (|N| + N) 57 tokens can
    take a state beyond 3.4e38 (test_forms without softplus and with a bias: 3.4e39 in 64 bits),
    where the header leaves the result open.  Such a channel is not compared."""
    fwd, back = ref.peak(o)
    top = float(np.finfo(np.float32).max)
    both = fwd * np.maximum(back, 1.0)        # products of a state and a gradient
    return (fwd < top) & (back < top) & (both < top / 1e6)


def _check(c, dev=None):
    dev = cuda(c) if dev is None else dev
    end, bf = c["cu_list"][-1], c["x"].dtype == torch.bfloat16
    o = _oracle(c)
    ok = _representable(o)
    if not ok.all():
        assert not c["softplus"]
        return _check_channels(c, dev, o, ok)
    y, S_T, states = kda.selscan_prefill(*_ins(dev), **_kw(dev), save_states=True,
                                         check_device_status=True)
    torch.cuda.synchronize()
    want, err = ref.forward(o)
    within("y", y[:end], want["y"][:end], err["y"][:end], bf)
    within("S_T", S_T, want["S_T"], err["S_T"])
    starts = set(c["cu_list"])
    at = [t for t in range(0, end, kda.SELSCAN_CHUNK) if t not in starts]
    within("states", states[[t // kda.SELSCAN_CHUNK for t in at]], want["before"][at],
           err["before"][at])
    got = kda.selscan_backward(*_ins(dev), dev["dy"], dev["dS_T"], **_kw(dev), states=states,
                               check_device_status=True)
    torch.cuda.synchronize()
    want, err = ref.backward(o)
    assert set(got) == set(want)
    for k in got:
        rows = slice(0, end) if want[k].shape[0] == c["x"].shape[0] and k in (
            "dx", "ddt", "dB", "dC", "dz") else slice(None)
        within(k, got[k][rows], want[k][rows], err[k][rows])
    return dev, y, S_T, states, got


def _check_channels(c, dev, o, ok):
    """The outputs of the channels that have a result, and the sums over channels of groups
    where all have."""
    assert ok.sum() >= ok.size / 2
    groups = ok.all(1)
    y, S_T, states = kda.selscan_prefill(*_ins(dev), **_kw(dev), save_states=True)
    got = kda.selscan_backward(*_ins(dev), dev["dy"], dev["dS_T"], **_kw(dev), states=states)
    torch.cuda.synchronize()
    want, err = ref.forward(o)
    t = torch.tensor(ok)
    within("y", y[:, t], want["y"][:, ok], err["y"][:, ok])
    within("S_T", S_T[:, t], want["S_T"][:, ok], err["S_T"][:, ok])
    want, err = ref.backward(o)
    for k in got:
        if k in ("dB", "dC"):
            at = (slice(None), groups)
        else:
            at = (slice(None), ok) if k in ("dx", "ddt", "dz", "dS0") else (ok,)
        pick = tuple(torch.tensor(a) if isinstance(a, np.ndarray) else a for a in at)
        within(k, got[k][pick], want[k][at], err[k][at])


@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill_and_backward(lens, dtype):
    _check(_case(LENS[lens], 1, 40, 16, dtype, S0=lens != "ragged", seed=len(lens)))


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9, 12, 16, 17, 24, 32, 33, 48, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_state_sizes(n, dtype):
    _check(_case([35, 0, 18], 2, 24, n, dtype, seed=n))


@pytest.mark.parametrize("H,d", [(1, 1), (3, 1), (1, 2), (2, 7), (3, 67), (1, 130), (2, 128), (1, 264)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_widths(H, d, dtype):
    for n in (4, 16):
        _check(_case([20, 45], H, d, n, dtype, tail=3, seed=d))


@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("D", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("softplus", [False, True])
def test_forms(z, D, bias, softplus):
    _check(_case([40, 17], 2, 16, 16, torch.float32, z, D, bias, S0=bias, softplus=softplus))


def _cut(c):
    """Whether the prefill's tokens are cut into segments: only then are there maps."""
    T, H, d = c["x"].shape
    return kda.selscan_workspace_size(len(c["cu_list"]) - 1, T, H, d, c["A"].shape[2]) > 256


@pytest.mark.parametrize("lens", [[400], [1, 300, 0, 64, 150, 2], [128, 128], [63, 0, 0, 450]])
@pytest.mark.parametrize("n", [4, 16, 32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_cut_along_the_tokens(lens, n, dtype):
    c = _case(lens, 1, 16, n, dtype, seed=n)
    assert _cut(c)
    dev, y, S_T, states, g = _check(c)
    # in place, and the states formed again
    S = dev["S0"].clone()
    ws = torch.empty(kda.selscan_workspace_size(len(lens), sum(lens), 1, 16, n), dtype=torch.uint8,
                     device="cuda")
    y2 = torch.empty_like(y)
    kda.selscan_prefill_into(*_ins(dict(dev, S0=S)), y2, S, ws, **_kw(dev))
    assert torch.equal(y, y2) and torch.equal(S, S_T)
    g2 = kda.selscan_backward(*_ins(dev), dev["dy"], dev["dS_T"], **_kw(dev))
    end = c["cu_list"][-1]
    assert all(torch.equal(g[k], g2[k]) for k in g)


@pytest.mark.parametrize("lens", [[0 if i % 7 == 3 else 80 for i in range(80)], [3, 0] * 700, [],
                                  [150] * 20 + [0] + [20] * 130])
def test_many_and_no_sequences(lens):
    """Cut along the tokens with more sequences than the join looks over for empty ones, more
    than a CTA checks or ranks by itself, and tokens that belong to none."""
    _check(_case(lens, 1, 16, 4, torch.float32, tail=7, seed=len(lens)))


def test_two_calls_at_once():
    """On two streams, from two threads, each with its own workspace."""
    import threading
    cs = [cuda(_case([300, 45], 1, 64, 16, torch.bfloat16, seed=s)) for s in (1, 2)]
    run = lambda c, **kw: kda.selscan_prefill(*_ins(c), **_kw(c), save_states=True, **kw)
    want = [run(c) for c in cs]
    back = [kda.selscan_backward(*_ins(c), c["dy"], c["dS_T"], **_kw(c), states=w[2])
            for c, w in zip(cs, want)]
    torch.cuda.synchronize()
    streams, got, grads = [torch.cuda.Stream() for _ in cs], [None, None], [None, None]

    def work(i):
        for _ in range(20):
            got[i] = run(cs[i], stream=streams[i])
            grads[i] = kda.selscan_backward(*_ins(cs[i]), cs[i]["dy"], cs[i]["dS_T"],
                                            **_kw(cs[i]), states=got[i][2], stream=streams[i])
    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in (0, 1):
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])
        assert all(torch.equal(grads[i][k], back[i][k]) for k in back[i])


def test_fast_and_slow_decays():
    c = _case([150, 300], 1, 16, 16, torch.float32, seed=2)
    c["A"][:, :4] = -1e-4
    c["A"][:, 4:8] = -60.0             # decays that leave nothing
    c["A"][:, 8] = 0.0
    c["dt"][10:20] += 30.0             # steps where softplus is the identity
    c["dt"][30:40] -= 25.0             # and where it is an exponential
    _check(c)


@pytest.mark.parametrize("lens", [[70, 33, 20], [500]])
@pytest.mark.parametrize("pads", [(16, 8), (8, 0), (1, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_rows(lens, pads, dtype):
    c = _case(lens, 2, 32, 16, dtype, seed=5)
    dev, y, S_T, states, g = _check(c)
    wide = dict(dev)
    for i, k in enumerate(("x", "dt", "B", "C", "z")):
        wide[k] = wide_rows(dev[k], pads[0], pads[1] * (i + 1))
    _, y2, S2, _, g2 = _check(c, wide)
    assert torch.equal(y, y2) and torch.equal(S_T, S2)
    # rows off the 16-byte grid add the sums over tokens and channels up in another order
    for k in g:
        assert torch.equal(g[k], g2[k]) or (pads[0] == 1 and k in ("dB", "dC", "dD", "ddt_bias")), k


@pytest.mark.parametrize("n", [3, 8, 16, 20, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_steps(n, dtype):
    """Steps against the oracle's scan of one token a sequence, from the states before."""
    B = 6
    c = _case([1] * B, 2, 35, n, dtype, seed=n)
    dev = cuda(c)
    o = _oracle(c)
    want, err = ref.forward(o)
    S = dev["S0"].clone()
    step = [dev[k] for k in ("x", "dt", "A", "B", "C")]
    y = kda.selscan_decode_step(*step, S, **_kw(dev))
    torch.cuda.synchronize()
    within("y", y, want["y"], err["y"], dtype == torch.bfloat16)
    within("S", S, want["S_T"], err["S_T"])
    wide = [wide_rows(t, 8, 16) if i != 2 else t for i, t in enumerate(step)]
    kw = dict(_kw(dev), z=wide_rows(dev["z"], 16, 8))
    S2 = dev["S0"].clone()
    assert torch.equal(kda.selscan_decode_step(*wide, S2, **kw), y) and torch.equal(S, S2)
    par = torch.tensor([0, 0, 5, -1, 6, 2], dtype=torch.int32, device="cuda")
    S_out = torch.empty_like(S)
    y2 = kda.selscan_decode_step(*step, dev["S0"], **_kw(dev), parents=par, S_out=S_out)
    moved = torch.stack([dev["S0"][p] if 0 <= p < B else torch.zeros_like(S[0])
                         for p in par.tolist()])
    y3 = kda.selscan_decode_step(*step, moved, **_kw(dev))
    assert torch.equal(y2, y3) and torch.equal(S_out, moved)


def test_rows_behind_the_last_sequence_are_left():
    for d in (16, 1000):               # cut along the tokens, and whole sequences
        c = cuda(_case([90, 70], 1, d, 16, torch.bfloat16, tail=40, seed=2))
        for k in ("x", "dt", "B", "C", "z", "dy"):
            c[k][160:] = float("nan")
        ws = torch.empty(max(kda.selscan_workspace_size(2, 200, 1, d, 16),
                             kda.selscan_backward_workspace_size(2, 200, 1, d, 16)),
                         dtype=torch.uint8, device="cuda")
        y, S_T = torch.full_like(c["x"], 7.0), torch.empty_like(c["S0"])
        states = torch.full((13, 1, d, 16), 7.0, device="cuda")
        kda.selscan_prefill_into(*_ins(c), y, S_T, ws, **_kw(c), states=states)
        assert (y[160:] == 7.0).all() and torch.isfinite(y.float()).all()
        assert (states[10:] == 7.0).all() and torch.isfinite(states).all()
        g = {k: torch.full_like(c[t], 7.0, dtype=torch.float32) for k, t in (
            ("dx", "x"), ("ddt", "dt"), ("dB", "B"), ("dC", "C"), ("dz", "z"), ("dA", "A"),
            ("dD", "D"), ("ddt_bias", "dt_bias"), ("dS0", "S0"))}
        kda.selscan_backward_into(*_ins(c), c["dy"], c["dS_T"], g, ws, **_kw(c), states=states)
        torch.cuda.synchronize()
        for k, t in g.items():
            assert torch.isfinite(t).all(), k
            if k in ("dx", "ddt", "dB", "dC", "dz"):
                assert (t[160:] == 7.0).all(), k


def test_values_stay_in_their_sequence():
    for d in (16, 1000):
        c = cuda(_case([50, 60, 70], 1, d, 16, torch.float32, seed=4))
        y, S_T, st = kda.selscan_prefill(*_ins(c), **_kw(c), save_states=True)
        g = kda.selscan_backward(*_ins(c), c["dy"], c["dS_T"], **_kw(c), states=st)
        for k in ("x", "dt", "B", "C", "z", "dy"):
            c[k][50:110] = float("nan")
        c["S0"][1], c["dS_T"][1] = float("nan"), float("inf")
        y2, S2, st = kda.selscan_prefill(*_ins(c), **_kw(c), save_states=True)
        g2 = kda.selscan_backward(*_ins(c), c["dy"], c["dS_T"], **_kw(c), states=st)
        for a, b in [(y, y2)] + [(g[k], g2[k]) for k in ("dx", "ddt", "dB", "dC", "dz")]:
            assert torch.equal(a[:50], b[:50]) and torch.equal(a[110:], b[110:])
        for a, b in ((S_T, S2), (g["dS0"], g2["dS0"])):
            assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("lens,d", [([4, 4], 16), ([200, 200], 16), ([2] * 1500, 8)])
def test_malformed_offsets_write_nothing(lens, d):
    c = cuda(_case(lens, 1, d, 4, torch.float32, seed=6))
    cu = c["cu"].clone()
    cu[1] = cu[2] + 1
    T, N = c["x"].shape[0], len(lens)
    ws = torch.empty(max(kda.selscan_workspace_size(N, T, 1, d, 4),
                         kda.selscan_backward_workspace_size(N, T, 1, d, 4, with_states=False)),
                     dtype=torch.uint8, device="cuda")
    y, S_T = torch.full_like(c["x"], 7.0), torch.full_like(c["S0"], 7.0)
    states = torch.full((-(-T // 16), 1, d, 4), 7.0, device="cuda")
    kda.selscan_prefill_into(*_ins(c)[:-1], cu, y, S_T, ws, **_kw(c), states=states)
    with pytest.raises(kda.KdaError):
        kda.device_status(ws)
    g = {k: torch.full_like(c[t], 7.0) for k, t in (
        ("dx", "x"), ("ddt", "dt"), ("dB", "B"), ("dC", "C"), ("dz", "z"), ("dA", "A"),
        ("dD", "D"), ("ddt_bias", "dt_bias"), ("dS0", "S0"))}
    for st in (states, None):
        kda.selscan_backward_into(*_ins(c)[:-1], cu, c["dy"], c["dS_T"], g, ws, **_kw(c), states=st)
        with pytest.raises(kda.KdaError):
            kda.device_status(ws)
    torch.cuda.synchronize()
    for t in (y, S_T, states, *g.values()):
        assert (t == 7.0).all()
    kda.selscan_prefill_into(*_ins(c), y, S_T, ws, **_kw(c))
    kda.device_status(ws)


@pytest.mark.parametrize("lens,d", [([700], 64), ([40] * 30, 512)])
def test_captured_on_another_stream_with_the_same_bits(lens, d):
    c = cuda(_case(lens, 1, d, 16, torch.bfloat16, seed=9))
    y, S_T, st = kda.selscan_prefill(*_ins(c), **_kw(c), save_states=True)
    g = kda.selscan_backward(*_ins(c), c["dy"], c["dS_T"], **_kw(c), states=st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y2, S2, st2 = kda.selscan_prefill(*_ins(c), **_kw(c), save_states=True)
        g2 = kda.selscan_backward(*_ins(c), c["dy"], c["dS_T"], **_kw(c), states=st2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(S_T, S2)
    assert all(torch.equal(g[k], g2[k]) for k in g)
    y3, _ = kda.selscan_prefill(*_ins(c), **_kw(c), stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, y3)
