"""The operators around a layer's recurrence without a GPU: every declared symbol is exported, bad
arguments are refused on the host before any CUDA call, and the Python binding refuses wrong
types, shapes, strides and placements before it calls into the library."""
import ctypes
import os
import re

import pytest
import torch

from gated_delta_rule_45_gb300 import kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
M = 0x1000000   # fake buffers 16 MB apart; never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_45_gb300 import build
    build.build()
    return kda.load()


def test_every_declared_symbol_is_exported(lib):
    names = set()
    for h in ("causalconv.h", "selscan.h", "groupnorm.h"):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", h)).read(), flags=re.S)
        names |= set(re.findall(r"\b((?:causalconv|selscan|groupnorm)_[a-z_0-9]+)\s*\(", text))
    assert len(names) == 13
    for name in names:
        assert hasattr(lib, name), name


# ---------------------------------------------------------------- causalconv

def _conv(lib, **kw):
    a = dict(x=1 * M, ldx=64, w=2 * M, b=3 * M, S0=None, cu=4 * M, N=2, T=300, D=64, W=4, dtype=0,
             act=1, y=5 * M, S_T=6 * M, ws=7 * M, ws_bytes=1 << 20)
    a.update(kw)
    return lib.causalconv_prefill(a["x"], a["ldx"], a["w"], a["b"], a["S0"], a["cu"], a["N"],
                                  a["T"], a["D"], a["W"], a["dtype"], a["act"], a["y"], a["S_T"],
                                  a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), 1), (dict(T=-1), 1), (dict(D=0), 1), (dict(W=0), 1), (dict(W=1), 2),
    (dict(W=5), 2), (dict(dtype=2), 1), (dict(act=2), 1), (dict(D=(1 << 20) + 1, ldx=1 << 21), 2),
    (dict(T=2 ** 31 - 1), 2), (dict(N=2 ** 30 + 1), 2), (dict(ldx=63), 1), (dict(ldx=1 << 40), 2),
    (dict(T=2 ** 23, D=2 ** 20, ldx=2 ** 20), 2), (dict(N=2 ** 17, D=2 ** 20, ldx=2 ** 20), 2),
    (dict(x=None), 1), (dict(w=None), 1), (dict(cu=None), 1), (dict(y=None), 1),
    (dict(S_T=None), 1), (dict(ws=None), 1), (dict(ws_bytes=8), 1), (dict(x=1 * M + 1), 1),
    (dict(w=2 * M + 4), 1), (dict(y=5 * M + 8), 1), (dict(S0=8 * M + 2), 1), (dict(y=1 * M), 1),
    (dict(S_T=5 * M + 1024), 1), (dict(S0=6 * M + 64), 1), (dict(y=2 * M), 1), (dict(y=7 * M), 1),
    (dict(ldx=1 << 16, y=1 * M + (299 << 17)), 1),      # y inside the last strided row
])
def test_conv_prefill_rejects_on_host(lib, kw, expect):
    assert _conv(lib, **kw) == expect


def _conv_back(lib, **kw):
    a = dict(x=1 * M, ldx=64, w=2 * M, b=3 * M, S0=None, cu=4 * M, N=2, T=300, D=64, W=4, dtype=0,
             act=1, dy=5 * M, dS_T=6 * M, dx=7 * M, dw=8 * M, db=9 * M, dS0=10 * M, ws=11 * M,
             ws_bytes=1 << 20)
    a.update(kw)
    return lib.causalconv_backward(a["x"], a["ldx"], a["w"], a["b"], a["S0"], a["cu"], a["N"],
                                   a["T"], a["D"], a["W"], a["dtype"], a["act"], a["dy"],
                                   a["dS_T"], a["dx"], a["dw"], a["db"], a["dS0"], a["ws"],
                                   a["ws_bytes"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(W=9), 2), (dict(act=-1), 1), (dict(dy=None), 1), (dict(dx=None), 1), (dict(dw=None), 1),
    (dict(ws_bytes=256), 1), (dict(dx=7 * M + 4), 1), (dict(dx=1 * M), 1), (dict(dw=7 * M), 1),
    (dict(db=8 * M + 64), 1), (dict(dS0=6 * M), 1), (dict(dS0=11 * M), 1), (dict(ldx=1), 1),
])
def test_conv_backward_rejects_on_host(lib, kw, expect):
    assert _conv_back(lib, **kw) == expect


def _conv_step(lib, **kw):
    a = dict(x=1 * M, ldx=64, w=2 * M, b=None, S=3 * M, rows=4, par=None, B=4, D=64, W=4, dtype=0,
             act=1, y=4 * M, S_out=5 * M)
    a.update(kw)
    return lib.causalconv_decode_step(a["x"], a["ldx"], a["w"], a["b"], a["S"], a["rows"],
                                      a["par"], a["B"], a["D"], a["W"], a["dtype"], a["act"],
                                      a["y"], a["S_out"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), 1), (dict(rows=-1), 1), (dict(rows=5), 1), (dict(x=None), 1), (dict(w=None), 1),
    (dict(S=None), 1), (dict(y=None), 1), (dict(S_out=None), 1), (dict(S_out=5 * M + 2), 1),
    (dict(S_out=3 * M + 64), 1), (dict(y=3 * M), 1), (dict(par=6 * M, S_out=3 * M), 1),
    (dict(par=6 * M + 4), 1), (dict(W=5), 2), (dict(B=0, rows=0, x=None), 0),
])
def test_conv_step_rejects_on_host(lib, kw, expect):
    assert _conv_step(lib, **kw) == expect


# ---------------------------------------------------------------- groupnorm

def _norm(lib, **kw):
    a = dict(x=1 * M, ldx=256, w=2 * M, b=3 * M, ph=1, z=4 * M, ldz=256, T=30, H=4, d=64, dtype=0,
             kind=1, act=1, eps=1e-5, y=5 * M)
    a.update(kw)
    return lib.groupnorm_forward(a["x"], a["ldx"], a["w"], a["b"], a["ph"], a["z"], a["ldz"],
                                 a["T"], a["H"], a["d"], a["dtype"], a["kind"], a["act"],
                                 a["eps"], a["y"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(d=0), 1), (dict(dtype=3), 1), (dict(kind=2), 1),
    (dict(act=3), 1), (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1),
    (dict(ph=2), 1), (dict(ldx=255), 1), (dict(ldz=255), 1), (dict(d=16385, H=1, ldx=1 << 15), 2),
    (dict(H=1 << 15, ldx=1 << 21, ldz=1 << 21), 2), (dict(ldx=1 << 40), 2), (dict(T=2 ** 31), 2),
    (dict(x=None), 1), (dict(y=None), 1), (dict(x=1 * M + 1), 1), (dict(z=4 * M + 1), 1),
    (dict(w=2 * M + 4), 1), (dict(y=5 * M + 2), 1), (dict(y=1 * M + 64), 1), (dict(y=2 * M), 1),
    (dict(ldx=512, y=1 * M), 1),               # in the place of strided rows
    (dict(T=0, x=None, y=None), 0),
])
def test_norm_forward_rejects_on_host(lib, kw, expect):
    assert _norm(lib, **kw) == expect


def _norm_back(lib, **kw):
    a = dict(x=1 * M, ldx=256, w=2 * M, b=3 * M, ph=4, z=4 * M, ldz=256, T=30, H=4, d=64, dtype=0,
             kind=1, act=1, eps=1e-5, dy=5 * M, dx=6 * M, dz=7 * M, dw=8 * M, db=9 * M, ws=10 * M,
             ws_bytes=1 << 24)
    a.update(kw)
    return lib.groupnorm_backward(a["x"], a["ldx"], a["w"], a["b"], a["ph"], a["z"], a["ldz"],
                                  a["T"], a["H"], a["d"], a["dtype"], a["kind"], a["act"],
                                  a["eps"], a["dy"], a["dx"], a["dz"], a["dw"], a["db"], a["ws"],
                                  a["ws_bytes"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dy=None), 1), (dict(dx=None), 1), (dict(z=None), 1),        # dz without a gate
    (dict(ws=None), 1), (dict(ws_bytes=64), 1), (dict(dx=6 * M + 4), 1), (dict(dx=5 * M), 1),
    (dict(dz=6 * M), 1), (dict(dw=2 * M), 1), (dict(db=8 * M), 1), (dict(dw=10 * M), 1),
    (dict(ph=3), 1), (dict(eps=-0.5), 1),
])
def test_norm_backward_rejects_on_host(lib, kw, expect):
    assert _norm_back(lib, **kw) == expect


# ---------------------------------------------------------------- selscan

def _rows(**kw):
    a = dict(x=1 * M, dt=2 * M, B=3 * M, C=4 * M, z=5 * M, ldx=64, lddt=64, ldB=32, ldC=32, ldz=64)
    a.update(kw)
    return kda._ScanRows(*(a[n] for n, _ in kda._ScanRows._fields_))


def _scan(lib, rows=None, **kw):
    a = dict(A=6 * M, D=7 * M, bias=8 * M, S0=None, cu=9 * M, N=2, T=300, H=2, d=32, n=16, dtype=0,
             step=1, y=10 * M, S_T=11 * M, states=None, ws=12 * M, ws_bytes=1 << 22)
    a.update(kw)
    r = _rows(**(rows or {}))
    return lib.selscan_prefill(ctypes.byref(r), a["A"], a["D"], a["bias"], a["S0"], a["cu"], a["N"],
                               a["T"], a["H"], a["d"], a["n"], a["dtype"], a["step"], a["y"],
                               a["S_T"], a["states"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), 1), (dict(T=-1), 1), (dict(H=0), 1), (dict(d=0), 1), (dict(n=0), 1),
    (dict(n=65), 2), (dict(dtype=5), 1), (dict(step=2), 1), (dict(d=1 << 20), 2),
    (dict(T=2 ** 31 - 1), 2), (dict(N=2 ** 30 + 1), 2), (dict(T=2 ** 30, H=1, d=2 ** 20), 2),
    (dict(rows=dict(x=None)), 1), (dict(rows=dict(dt=None)), 1), (dict(rows=dict(B=None)), 1),
    (dict(rows=dict(C=None)), 1), (dict(rows=dict(ldx=63)), 1), (dict(rows=dict(ldB=31)), 1),
    (dict(rows=dict(ldz=0)), 1), (dict(rows=dict(lddt=1 << 40)), 2), (dict(rows=dict(z=5 * M + 1)), 1),
    (dict(A=None), 1), (dict(cu=None), 1), (dict(y=None), 1), (dict(S_T=None), 1),
    (dict(ws=None), 1), (dict(ws_bytes=8), 1), (dict(A=6 * M + 4), 1), (dict(states=13 * M + 8), 1),
    (dict(y=1 * M), 1), (dict(S_T=6 * M), 1), (dict(S0=11 * M + 256), 1),
    (dict(states=10 * M + 4096), 1), (dict(S_T=12 * M), 1), (dict(y=8 * M), 1),
])
def test_scan_prefill_rejects_on_host(lib, kw, expect):
    assert _scan(lib, **kw) == expect


def _scan_back(lib, rows=None, grads=None, **kw):
    a = dict(A=6 * M, D=7 * M, bias=8 * M, S0=None, cu=9 * M, N=2, T=300, H=2, d=32, n=16, dtype=0,
             step=1, dy=10 * M, dS_T=11 * M, states=12 * M, ws=13 * M, ws_bytes=1 << 22)
    a.update(kw)
    g = dict(dx=20 * M, ddt=21 * M, dB=22 * M, dC=23 * M, dz=24 * M, dA=25 * M, dD=26 * M,
             ddt_bias=27 * M, dS0=28 * M)
    g.update(grads or {})
    r, g = _rows(**(rows or {})), kda._ScanGrads(*(g[n] for n, _ in kda._ScanGrads._fields_))
    return lib.selscan_backward(ctypes.byref(r), a["A"], a["D"], a["bias"], a["S0"], a["cu"],
                                a["N"], a["T"], a["H"], a["d"], a["n"], a["dtype"], a["step"],
                                a["dy"], a["dS_T"], a["states"], ctypes.byref(g), a["ws"],
                                a["ws_bytes"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(n=128), 2), (dict(dy=None), 1), (dict(ws_bytes=64), 1), (dict(rows=dict(z=None)), 1),
    (dict(grads=dict(dx=None)), 1), (dict(grads=dict(ddt=None)), 1), (dict(grads=dict(dB=None)), 1),
    (dict(grads=dict(dC=None)), 1), (dict(grads=dict(dA=None)), 1), (dict(grads=dict(dz=None)), 1),
    (dict(grads=dict(dx=20 * M + 4)), 1), (dict(grads=dict(ddt=20 * M)), 1),
    (dict(grads=dict(dS0=11 * M)), 1), (dict(grads=dict(dB=1 * M)), 1),
    (dict(grads=dict(dA=12 * M)), 1), (dict(grads=dict(dD=13 * M)), 1),
])
def test_scan_backward_rejects_on_host(lib, kw, expect):
    assert _scan_back(lib, **kw) == expect


def _scan_step(lib, rows=None, **kw):
    a = dict(A=6 * M, D=None, bias=None, S=7 * M, num=4, par=None, B=4, H=2, d=32, n=16, dtype=0,
             step=1, y=8 * M, S_out=9 * M)
    a.update(kw)
    r = _rows(**(rows or {}))
    return lib.selscan_decode_step(ctypes.byref(r), a["A"], a["D"], a["bias"], a["S"], a["num"],
                                   a["par"], a["B"], a["H"], a["d"], a["n"], a["dtype"],
                                   a["step"], a["y"], a["S_out"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), 1), (dict(num=-1), 1), (dict(num=3), 1), (dict(S=None), 1), (dict(y=None), 1),
    (dict(S_out=None), 1), (dict(A=None), 1), (dict(rows=dict(x=None)), 1),
    (dict(S_out=7 * M + 512), 1), (dict(y=9 * M), 1), (dict(y=7 * M), 1),
    (dict(par=10 * M, S_out=7 * M), 1), (dict(par=10 * M + 4), 1), (dict(n=65), 2),
    (dict(B=1 << 22, num=1 << 22, H=1, d=1 << 16, n=1, rows=dict(
        ldx=1 << 16, lddt=1 << 16, ldz=1 << 16)), 2),
    (dict(B=0, num=0), 0),
])
def test_scan_step_rejects_on_host(lib, kw, expect):
    assert _scan_step(lib, **kw) == expect


def test_workspace_sizes(lib):
    assert lib.causalconv_prefill_workspace_size(0, 0, 1, 2, 0) > 0
    assert lib.causalconv_prefill_workspace_size(3, 100, 64, 5, 0) == 0
    assert lib.causalconv_backward_workspace_size(3, 100, 64, 4) > 4 * 64 * 5 * 4
    assert lib.causalconv_backward_workspace_size(3, -1, 64, 4) == 0
    assert lib.selscan_prefill_workspace_size(0, 0, 1, 1, 1) > 0
    assert lib.selscan_prefill_workspace_size(1, 10, 1, 1, 65) == 0
    f = lib.selscan_backward_workspace_size
    assert f(2, 1000, 2, 67, 12, 0) > f(2, 1000, 2, 67, 12, 1) > 0
    assert f(2, 1000, 0, 67, 12, 1) == 0
    assert lib.groupnorm_backward_workspace_size(10, 4, 64) > 0
    assert lib.groupnorm_backward_workspace_size(0, 1, 1) > 0
    assert lib.groupnorm_backward_workspace_size(10, 4, 20000) == 0


# ---------------------------------------------------------------- the binding

F, BF, I = torch.float32, torch.bfloat16, torch.int32
T, H, D, N, NS = 8, 2, 16, 2, 4


def _z(*shape, dtype=F):
    return torch.zeros(*shape, dtype=dtype)


CUS = torch.tensor([0, 3, T], dtype=I)


@pytest.mark.parametrize("bad,err", [
    (dict(x=_z(T, H, D, dtype=torch.float16)), TypeError), (dict(x=_z(T)), ValueError),
    (dict(x=_z(D, T, H).permute(1, 2, 0)), ValueError), (dict(x=_z(1, H, D).expand(T, H, D)), ValueError),
    (dict(w=_z(H, D, 4, dtype=BF)), TypeError), (dict(w=_z(H, 4)), ValueError),
    (dict(b=_z(H * D)), ValueError), (dict(S0=_z(N, 3, H, D, dtype=BF)), TypeError),
    (dict(S0=_z(N, 4, H, D)), ValueError), (dict(cu=CUS.long()), TypeError),
    (dict(dy=_z(T, H, D, dtype=BF)), TypeError), (dict(dS=_z(N, 3, H, D, dtype=BF)), TypeError),
    (dict(), ValueError),                                    # right, but on the host
])
def test_conv_binding_rejects(bad, err):
    a = dict(x=_z(T, H, D), w=_z(H, D, 4), b=_z(H, D), S0=_z(N, 3, H, D), cu=CUS, dy=_z(T, H, D),
             dS=_z(N, 3, H, D))
    a.update(bad)
    with pytest.raises(err):
        kda.causalconv_backward(a["x"], a["w"], a["b"], a["S0"], a["cu"], a["dy"], a["dS"])
    if not {"dy", "dS"} & set(bad):
        with pytest.raises(err):
            kda.causalconv_prefill(a["x"], a["w"], a["b"], a["S0"], a["cu"])


def test_conv_step_binding_rejects():
    x, w, S = _z(3, H, D), _z(H, D, 4), _z(3, 3, H, D)
    for args, kw, err in (((x, w, None, S), {}, ValueError),
                          ((x, w, None, _z(4, 3, H, D)), {}, ValueError),
                          ((x, w, None, S.to(BF)), {}, TypeError),
                          ((x, w, None, S), dict(parents=torch.zeros(3, dtype=I)), ValueError),
                          ((x, w, None, S), dict(parents=torch.zeros(3), S_out=S), TypeError)):
        with pytest.raises(err):
            kda.causalconv_decode_step(*args, **kw)


def _scan_tensors(**kw):
    a = dict(x=_z(T, H, D), dt=_z(T, H, D), A=_z(H, D, NS), B=_z(T, H, NS), C=_z(T, H, NS),
             S0=_z(N, H, D, NS), cu=CUS, dy=_z(T, H, D), dS=None, D=_z(H, D), z=_z(T, H, D),
             bias=_z(H, D), states=None)
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,err", [
    (dict(x=_z(T, H * D)), ValueError), (dict(x=_z(T, H, D).half()), TypeError),
    (dict(dt=_z(T, H, D, dtype=BF)), TypeError), (dict(dt=_z(T, H, 1)), ValueError),
    (dict(A=_z(H, D)), ValueError), (dict(A=_z(H, D, NS).double()), TypeError),
    (dict(B=_z(T, 1, NS)), ValueError), (dict(C=_z(T, H, NS + 1)), ValueError),
    (dict(C=_z(T, NS, H).transpose(1, 2)), ValueError), (dict(z=_z(T, H, D, dtype=BF)), TypeError),
    (dict(D=_z(H)), ValueError), (dict(bias=_z(H, D, dtype=BF)), TypeError),
    (dict(S0=_z(N, H, D)), ValueError), (dict(cu=CUS.long()), TypeError),
    (dict(dy=_z(T, H, D, dtype=BF)), TypeError), (dict(dS=_z(1, H, D, NS)), ValueError),
    (dict(states=_z(2, H, D, NS)), ValueError), (dict(), ValueError),
])
def test_scan_binding_rejects(bad, err):
    a = _scan_tensors(**bad)
    with pytest.raises(err):
        kda.selscan_backward(a["x"], a["dt"], a["A"], a["B"], a["C"], a["S0"], a["cu"], a["dy"],
                             a["dS"], D=a["D"], z=a["z"], dt_bias=a["bias"], states=a["states"])
    if not {"dy", "dS", "states"} & set(bad):
        with pytest.raises(err):
            kda.selscan_prefill(a["x"], a["dt"], a["A"], a["B"], a["C"], a["S0"], a["cu"], D=a["D"],
                                z=a["z"], dt_bias=a["bias"])


def test_scan_step_binding_rejects():
    a = _scan_tensors()
    ins = (a["x"], a["dt"], a["A"], a["B"], a["C"])
    S = _z(T, H, D, NS)
    p = torch.zeros(T, dtype=I)
    for args, kw, err in (((S,), {}, ValueError), ((_z(T + 1, H, D, NS),), {}, ValueError),
                          ((S.to(BF),), {}, TypeError), ((S,), dict(parents=p), ValueError),
                          ((S,), dict(parents=p.long(), S_out=S), TypeError)):
        with pytest.raises(err):
            kda.selscan_decode_step(*ins, *args, **kw)


@pytest.mark.parametrize("args,kw,err", [
    ((_z(T, H * D),), {}, ValueError), ((_z(T, H, D).half(),), {}, TypeError),
    ((_z(T, H, D), _z(H)), {}, ValueError), ((_z(T, H, D), _z(D, dtype=BF)), {}, TypeError),
    ((_z(T, H, D), _z(D), _z(H, D)), {}, ValueError),
    ((_z(T, H, D),), dict(z=_z(T, H, D, dtype=BF)), TypeError),
    ((_z(T, H, D),), dict(act="relu"), ValueError), ((_z(T, H, D),), {}, ValueError),
    ((_z(T, D, H).transpose(1, 2),), {}, ValueError),
])
def test_norm_binding_rejects(args, kw, err):
    with pytest.raises(err):
        kda.groupnorm_forward(*args, **kw)
    x, w, b = (list(args) + [None, None])[:3]
    with pytest.raises(err):
        kda.groupnorm_backward(x, w, b, _z(T, H, D, dtype=x.dtype), **kw)
