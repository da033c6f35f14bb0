"""The gated linear recurrence and beam search without a GPU: every declared symbol is
exported, bad arguments are refused on the host before any CUDA call, and the Python
binding refuses wrong types, shapes and placements before it calls into the library."""
import ctypes
import os
import re

import pytest
import torch

from gated_delta_rule_45_gb300 import kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
M = 0x1000000   # fake buffers 16 MB apart; never dereferenced
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_45_gb300 import build
    build.build()
    return kda.load()


def test_every_declared_symbol_is_exported(lib):
    names = set()
    for h in ("linrec.h", "beam.h"):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", h)).read(), flags=re.S)
        names |= set(re.findall(r"\b((?:kda|linrec|beam)_[a-z_0-9]+)\s*\(", text))
    assert len(names) == 9 and "linrec_prefill" in names and "kda_decode_step_parents" in names
    for name in names:
        assert hasattr(lib, name), name


def _prefill(lib, **kw):
    a = dict(x=1 * M, gate=2 * M, fmt=0, S0=None, cu=3 * M, N=2, T=300, H=2, d=64, dtype=0,
             input=0, y=4 * M, S_T=5 * M, states=None, ws=6 * M, ws_bytes=1 << 20)
    a.update(kw)
    return lib.linrec_prefill(a["x"], a["gate"], a["fmt"], a["S0"], a["cu"], a["N"], a["T"],
                              a["H"], a["d"], a["dtype"], a["input"], a["y"], a["S_T"],
                              a["states"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), 1), (dict(T=-1), 1), (dict(H=0), 1), (dict(d=0), 1), (dict(dtype=4), 1),
    (dict(fmt=3), 1), (dict(input=2), 1), (dict(d=70000), 2), (dict(H=2048, d=1024), 2),
    (dict(T=2 ** 31 - 1), 2), (dict(N=2 ** 30 + 1), 2), (dict(T=2 ** 30, d=65536), 2),
    (dict(cu=None), 1), (dict(ws=None), 1), (dict(S_T=None), 1), (dict(x=None), 1),
    (dict(gate=None), 1), (dict(y=None), 1), (dict(ws_bytes=8), 1),
    (dict(x=1 * M + 4), 1), (dict(states=7 * M + 8), 1),
    (dict(y=1 * M), 1),                        # y is x
    (dict(y=2 * M + 1024), 1),                 # y inside the gate
    (dict(S0=5 * M + 64), 1),                  # S_T overlaps S0 without being it
    (dict(states=4 * M + 4096), 1),            # states inside y
    (dict(S_T=6 * M + 256), 1),                # S_T inside the workspace
])
def test_linrec_prefill_rejects_on_host(lib, kw, expect):
    assert _prefill(lib, **kw) == expect


def test_linrec_workspace_sizes(lib):
    f, g = lib.linrec_prefill_workspace_size, lib.linrec_backward_workspace_size
    assert f(3, 1000, 2, 67) > 0 and f(0, 0, 1, 1) > 0
    assert g(3, 1000, 2, 67, 1, 0) >= g(3, 1000, 2, 67, 1, 1) > 0
    for bad in [(-1, 10, 1, 1), (1, -1, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (1, 1, 2048, 1024)]:
        assert f(*bad) == 0 and g(*bad, 0, 1) == 0
    assert g(1, 1, 1, 1, 5, 1) == 0


def _backward(lib, **kw):
    a = dict(x=1 * M, gate=2 * M, fmt=0, S0=None, cu=3 * M, N=2, T=300, H=2, d=64, dtype=0,
             input=0, dy=4 * M, dS_T=5 * M, states=6 * M, dx=7 * M, dgate=8 * M, dS0=9 * M,
             ws=10 * M, ws_bytes=1 << 22)
    a.update(kw)
    return lib.linrec_backward(a["x"], a["gate"], a["fmt"], a["S0"], a["cu"], a["N"], a["T"],
                               a["H"], a["d"], a["dtype"], a["input"], a["dy"], a["dS_T"],
                               a["states"], a["dx"], a["dgate"], a["dS0"], a["ws"],
                               a["ws_bytes"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(fmt=9), 1), (dict(dtype=-1), 1), (dict(input=5), 1), (dict(d=70000), 2),
    (dict(dy=None), 1), (dict(dx=None), 1), (dict(dgate=None), 1), (dict(ws_bytes=16), 1),
    (dict(dx=7 * M + 8), 1), (dict(dx=1 * M), 1), (dict(dgate=7 * M + 256), 1),
    (dict(dS0=5 * M), 1), (dict(dgate=6 * M), 1), (dict(dx=10 * M), 1),
])
def test_linrec_backward_rejects_on_host(lib, kw, expect):
    assert _backward(lib, **kw) == expect


def _step(lib, **kw):
    a = dict(x=1 * M, gate=2 * M, fmt=0, S=3 * M, rows=4, parents=None, B=4, H=2, d=64, dtype=0,
             input=0, y=4 * M, S_out=5 * M)
    a.update(kw)
    return lib.linrec_decode_step(a["x"], a["gate"], a["fmt"], a["S"], a["rows"], a["parents"],
                                  a["B"], a["H"], a["d"], a["dtype"], a["input"], a["y"],
                                  a["S_out"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), 1), (dict(rows=5), 1), (dict(rows=-1), 1), (dict(x=None), 1), (dict(S=None), 1),
    (dict(y=None), 1), (dict(S_out=None), 1), (dict(S_out=5 * M + 4), 1),
    (dict(S_out=3 * M + 256), 1), (dict(y=3 * M), 1), (dict(y=5 * M), 1),
    (dict(parents=6 * M, S_out=3 * M), 1),     # beams cannot move in place
    (dict(parents=6 * M + 4), 1), (dict(fmt=7), 1), (dict(d=70000), 2),
    (dict(B=0, rows=0), 0),                    # empty: a no-op
])
def test_linrec_decode_rejects_on_host(lib, kw, expect):
    assert _step(lib, **kw) == expect


def _select(lib, **kw):
    a = dict(logits=1 * M, ld=None, scores=2 * M, fin=None, B=2, K=4, V=1000, n=8, eos=0,
             dtype=0, os=3 * M, op=4 * M, ot=5 * M, ws=6 * M, ws_bytes=1 << 20)
    a.update(kw)
    if a["ld"] is None:
        a["ld"] = a["V"]
    return lib.beam_select(a["logits"], a["ld"], a["scores"], a["fin"], a["B"], a["K"], a["V"],
                           a["n"], a["eos"], a["dtype"], a["os"], a["op"], a["ot"], a["ws"],
                           a["ws_bytes"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), 1), (dict(B=-1), 1), (dict(K=0), 1), (dict(V=0), 1), (dict(n=0), 1),
    (dict(V=2, K=2, n=5), 1),                  # fewer candidates than asked for
    (dict(K=33), 2), (dict(n=65), 2), (dict(V=1 << 21), 2), (dict(B=1 << 19, K=4), 2),
    (dict(ld=999), 1), (dict(ld=1001), 1),     # rows too short; rows off the 16-byte grid
    (dict(fin=7 * M, eos=1000), 1), (dict(fin=7 * M, eos=-1), 1),
    (dict(logits=None), 1), (dict(scores=None), 1), (dict(os=None), 1), (dict(op=None), 1),
    (dict(ot=None), 1), (dict(ws=None), 1), (dict(ws_bytes=16), 1),
    (dict(logits=1 * M + 2), 1), (dict(os=2 * M), 1), (dict(op=3 * M), 1),
    (dict(ot=1 * M + 64), 1), (dict(os=6 * M), 1),
    (dict(B=0), 0),
])
def test_beam_select_rejects_on_host(lib, kw, expect):
    assert _select(lib, **kw) == expect


def _reorder(lib, states, parents=9 * M, B=2, K=4):
    d = (kda._BeamState * max(1, len(states)))()
    for s, (data, n) in zip(d, states):
        s.data, s.row_bytes = data, n
    return lib.beam_reorder(ctypes.byref(d), len(states), parents, B, K, None)


def test_beam_reorder_rejects_on_host(lib):
    assert _reorder(lib, [(1 * M, 64)], K=0) == 1
    assert _reorder(lib, [(1 * M, 64)], B=-1) == 1
    assert _reorder(lib, [(1 * M, 64)], K=33) == 2
    assert _reorder(lib, [(1 * M, 64)], B=1 << 19) == 2
    assert _reorder(lib, [(1 * M, -4)]) == 1
    assert _reorder(lib, [(None, 64)]) == 1
    assert _reorder(lib, [(1 * M + 8, 64)]) == 1
    assert _reorder(lib, [(1 * M, 64)], parents=None) == 1
    assert _reorder(lib, [(1 * M, 64)], parents=9 * M + 4) == 1
    assert _reorder(lib, [(1 * M, 64), (1 * M + 256, 64)]) == 1   # two tensors overlap
    assert _reorder(lib, [(9 * M, 64)]) == 1                      # the parents' own memory
    assert _reorder(lib, [(1 * M, 1 << 41)]) == 2
    assert _reorder(lib, [(1 * M, 64)], B=0) == 0
    assert _reorder(lib, []) == 0


def test_decode_step_parents_rejects_on_host(lib):
    def call(**kw):
        a = dict(q=1 * M, k=2 * M, v=3 * M, al=4 * M, fmt=0, be=5 * M, S_in=6 * M, rows=3,
                 par=7 * M, S_out=8 * M, B=2, H=2, d_k=64, d_v=64, dtype=0, o=9 * M)
        a.update(kw)
        return lib.kda_decode_step_parents(a["q"], a["k"], a["v"], a["al"], a["fmt"], a["be"],
                                           a["S_in"], a["rows"], a["par"], a["S_out"], a["B"],
                                           a["H"], a["d_k"], a["d_v"], a["dtype"], a["o"], None)
    assert call(rows=-1) == 1
    assert call(par=None) == 1 and call(S_in=None) == 1 and call(S_out=None) == 1
    assert call(par=7 * M + 8) == 1 and call(S_in=6 * M + 4) == 1
    assert call(S_out=6 * M) == 1                 # in place
    assert call(S_out=6 * M + 3 * 2 * 64 * 64 * 4 - 16) == 1
    assert call(o=7 * M) == 1
    assert call(d_k=96) == 2 and call(fmt=4) == 1 and call(d_v=5000) == 2
    assert call(B=0, par=None, S_in=None, rows=0) == 0


# ---------------------------------------------------------------- the binding

F, BF, I = torch.float32, torch.bfloat16, torch.int32
T, H, D, N = 8, 2, 16, 2


def _z(*shape, dtype=F):
    return torch.zeros(*shape, dtype=dtype)


def _linrec(fn="prefill", **kw):
    a = dict(x=_z(T, H, D, dtype=BF), a=_z(T, H, D), S0=_z(N, H, D),
             cu=torch.tensor([0, 3, T], dtype=I), y=_z(T, H, D, dtype=BF), S_T=_z(N, H, D),
             ws=_z(4096, dtype=torch.uint8), states=_z(1, H, D), gate="channel",
             dy=_z(T, H, D, dtype=BF), dS=_z(N, H, D),
             grads=dict(dx=_z(T, H, D), dgate=_z(T, H, D), dS0=_z(N, H, D)))
    a.update(kw)
    if fn == "prefill":
        return kda.linrec_prefill_into(a["x"], a["a"], a["S0"], a["cu"], a["y"], a["S_T"],
                                       a["ws"], states=a["states"], gate=a["gate"])
    return kda.linrec_backward_into(a["x"], a["a"], a["S0"], a["cu"], a["dy"], a["dS"],
                                    a["grads"], a["ws"], states=a["states"], gate=a["gate"])


@pytest.mark.parametrize("fn", ["prefill", "backward"])
@pytest.mark.parametrize("bad,err", [
    (dict(x=_z(T, H, D, dtype=torch.float16)), TypeError),
    (dict(x=_z(T, H * D, dtype=BF)), ValueError),
    (dict(a=_z(T, H, D, dtype=BF)), TypeError),
    (dict(a=_z(T, H)), ValueError),
    (dict(gate="head"), ValueError),
    (dict(gate="log_bf16"), TypeError),
    (dict(S0=_z(N, H, D, dtype=BF)), TypeError),
    (dict(S0=_z(N + 1, H, D)), ValueError),
    (dict(cu=torch.tensor([0, 3, T])), TypeError),
    (dict(states=_z(2, H, D)), ValueError),
    (dict(), ValueError),                        # right, but on the host
])
def test_linrec_binding_rejects(fn, bad, err):
    with pytest.raises(err):
        _linrec(fn, **bad)


@pytest.mark.parametrize("bad,err", [
    (dict(y=_z(T, H, D)), TypeError), (dict(y=_z(T + 1, H, D, dtype=BF)), ValueError),
    (dict(S_T=_z(N, H, D, dtype=torch.float64)), TypeError), (dict(S_T=_z(1, H, D)), ValueError),
])
def test_linrec_prefill_binding_rejects_outputs(bad, err):
    with pytest.raises(err):
        _linrec("prefill", **bad)


@pytest.mark.parametrize("bad,err", [
    (dict(dy=_z(T, H, D)), TypeError), (dict(dS=_z(N, H, D, dtype=BF)), TypeError),
    (dict(grads=dict(dx=_z(T, H, D, dtype=BF), dgate=_z(T, H, D))), TypeError),
    (dict(grads=dict(dx=_z(T, H, D), dgate=_z(T, H))), ValueError),
])
def test_linrec_backward_binding_rejects_gradients(bad, err):
    with pytest.raises(err):
        _linrec("backward", **bad)


def test_linrec_decode_binding_rejects():
    x, a, S = _z(3, H, D), _z(3, H, D), _z(3, H, D)
    with pytest.raises(ValueError, match="CUDA"):
        kda.linrec_decode_step(x, a, S)
    with pytest.raises(ValueError):
        kda.linrec_decode_step(x, a, _z(4, H, D))
    with pytest.raises(TypeError):
        kda.linrec_decode_step(x, a, S, parents=torch.zeros(3, dtype=torch.int64), S_out=S)
    with pytest.raises(ValueError, match="S_out"):
        kda.linrec_decode_step(x, a, S, parents=torch.zeros(3, dtype=I))
    with pytest.raises(TypeError):
        kda.linrec_decode_step(x, a, _z(3, H, D, dtype=BF))


def test_decode_step_parents_binding_rejects():
    def call(**kw):
        B, dk, dv = 3, 16, 8
        t = dict(q=_z(B, H, dk), k=_z(B, H, dk), v=_z(B, H, dv), al=_z(B, H, dv), be=_z(B, H),
                 S=_z(5, H, dv, dk), p=torch.zeros(B, dtype=I), S2=_z(B, H, dv, dk))
        t.update(kw)
        return kda.decode_step_parents(t["q"], t["k"], t["v"], t["al"], t["be"], t["S"], t["p"],
                                       t["S2"])
    for bad, err in ((dict(), ValueError), (dict(p=torch.zeros(3)), TypeError),
                     (dict(p=torch.zeros(4, dtype=I)), ValueError),
                     (dict(S=_z(5, H, 8, 16, dtype=BF)), TypeError),
                     (dict(S2=_z(5, H, 8, 16)), ValueError), (dict(k=_z(3, H, 8)), ValueError),
                     (dict(v=_z(3, H, 8, dtype=BF)), TypeError)):
        with pytest.raises(err):
            call(**bad)


def test_beam_binding_rejects():
    lg, sc = _z(8, 50), _z(2, 4)
    for args, kw, err in (((lg, sc, 8), {}, ValueError),                       # on the host
                          ((lg.half(), sc, 8), {}, TypeError),
                          ((lg, sc.double(), 8), {}, TypeError),
                          ((_z(9, 50), sc, 8), {}, ValueError),
                          ((lg, sc, 8), dict(finished=_z(2, 4)), TypeError),
                          ((lg, sc, 8), dict(finished=_z(4, 2, dtype=torch.uint8)), ValueError),
                          ((_z(50, 8).t(), sc, 8), {}, ValueError),            # columns
                          ((lg, sc, 65), {}, kda.KdaError), ((lg, sc, 0), {}, kda.KdaError),
                          ((_z(66, 50), _z(2, 33), 8), {}, kda.KdaError)):
        with pytest.raises(err):
            kda.beam_select(*args, **kw)
    p = torch.zeros(8, dtype=I)
    for args, err in ((([_z(8, 3)], p, 4), ValueError), (([_z(7, 3)], p, 4), ValueError),
                      (([_z(8, 3)], p.long(), 4), TypeError), (([_z(8, 3)], p, 3), ValueError),
                      (([_z(8, 3)], p, 0), ValueError)):
        with pytest.raises(err):
            kda.beam_reorder(*args)
