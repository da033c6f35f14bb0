"""Selective state space scan: fp64 numpy reference, forward and backward.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Per (sequence, group, channel), one token at a time:

    s_t = softplus(dt_t + dt_bias) or dt_t + dt_bias,   a_t = exp(s_t A),
    h_t = a_t h_{t-1} + s_t x_t B_t,   y_t = (C_t . h_t + D x_t) silu(z_t)

Layouts as in ``include/selscan.h``: x, dt, z [T, H, d], B, C [T, H, n], A [H, d, n], D, dt_bias
[H, d], states [N, H, d, n].  ``forward`` and ``backward`` also return, element by element, the
largest error that 32-bit arithmetic leaves, by running the same lines on magnitudes and
errors.  A decay is off by `rho`: the error of the step size and the roundings of the rate and
of the exponent, all times the exponent, and 2^-22 of the exponential and its scale; where the
tokens are cut into segments the step sizes are summed first, which is off by at most one
rounding a token of the exponent.
"""
from __future__ import annotations

import numpy as np

from . import causalconv as cc

U32 = cc.U32
DEEP = 96          # additions that a sum over channels or values is deep, at most
EX2 = 2.0 ** -22   # of the exponential


def _steps(c):
    """Step sizes, their slope by dt, and their relative error: one addition, the exponential's
    argument and value, the series and its division."""
    v = c["dt"].astype(np.float64)
    ev = np.zeros_like(v)
    if c.get("dt_bias") is not None:
        ev = U32 * np.abs(v + c["dt_bias"])
        v = v + c["dt_bias"]
    if not c["softplus"]:
        return v, np.ones_like(v), ev, 0.0 * v, v
    s = np.logaddexp(v, 0.0)
    sig = cc.sigmoid(v)
    # the slope is at most the step itself times 1.45 for small steps, and 1
    es = np.minimum(1.0, 1.45 * s) * ev + s * (EX2 + 16 * U32)
    return s, sig, es, sig * cc.sigmoid_rel(v) + 0.25 * ev, v


def _rho(c, s, es):
    T = c["x"].shape[0]
    arg = np.abs(c["A"]) * np.abs(s)[..., None]
    return np.abs(c["A"]) * es[..., None] + arg * (3 + T) * U32 + 2 * EX2 + 6 * U32


def _states(c):
    """(before [T,..n], after, their errors), and S_T with its error."""
    x, B, A, cu = (np.asarray(c[k], np.float64) if k != "cu" else c[k] for k in ("x", "B", "A", "cu"))
    T, H, d = x.shape
    N, n = len(cu) - 1, A.shape[2]
    s, sig, es, esig, v = _steps(c)
    rho = _rho(c, s, es)
    a = np.exp(s[..., None] * A)
    u = (s * x)[..., None] * B[:, :, None]
    eu = (es * np.abs(x))[..., None] * np.abs(B)[:, :, None] + 3 * U32 * np.abs(u)
    S_T = np.zeros((N, H, d, n)) if c.get("S0") is None else np.array(c["S0"], np.float64)
    eS = np.zeros_like(S_T)
    before, after = np.zeros((T, H, d, n)), np.zeros((T, H, d, n))
    eb, ea = np.zeros_like(before), np.zeros_like(before)
    mag = np.abs(S_T)
    for q in range(N):
        h, e, m = S_T[q], eS[q], mag[q]
        for t in range(cu[q], cu[q + 1]):
            before[t], eb[t] = h, e
            e = a[t] * (e + rho[t] * m) + eu[t]
            m = a[t] * m + np.abs(u[t])
            e = e + 2 * U32 * m
            h = a[t] * h + u[t]
            after[t], ea[t] = h, e
        S_T[q], eS[q] = h, e
    return dict(x=x, B=B, A=A, C=np.asarray(c["C"], np.float64), s=s, sig=sig, es=es, esig=esig, v=v,
                rho=rho, a=a, u=u, eu=eu, before=before, after=after, eb=eb, ea=ea, S_T=S_T, eS=eS)


def _raw(c, f):
    """C . h + D x and its error."""
    raw = np.einsum("thdn,thn->thd", f["after"], f["C"])
    aC = np.abs(f["C"])
    err = np.einsum("thdn,thn->thd", f["ea"] + DEEP * U32 * np.abs(f["after"]), aC)
    if c.get("D") is not None:
        raw = raw + c["D"] * f["x"]
        err = err + 2 * U32 * (np.abs(c["D"] * f["x"]) + np.abs(raw))
    return raw, err


def forward(c):
    """Returns ({y, S_T, before}, their largest errors); y's before its rounding."""
    f = _states(c)
    raw, err = _raw(c, f)
    if c.get("z") is not None:
        z = np.asarray(c["z"], np.float64)
        g = cc.silu(z)
        err = err * np.abs(g) + np.abs(raw) * cc.silu_error(z, 0.0) + U32 * np.abs(raw * g)
        raw = raw * g
    return {"y": raw, "S_T": f["S_T"], "before": f["before"]}, \
        {"y": err, "S_T": f["eS"], "before": f["eb"]}


def peak(c):
    """Largest value [H, d] that a channel's states, the gradients that come back through them
    or their products take: above the range of 32 bits the recurrence has no result there."""
    f = _states(c)
    top = np.maximum(np.abs(f["after"]).max((0, 3), initial=0.0),
                     np.abs(f["S_T"]).max((0, 3), initial=0.0))
    back = 0.0 * top
    dr = np.abs(np.asarray(c["dy"], np.float64))
    for q in range(len(c["cu"]) - 1):
        R = 0.0 if c.get("dS_T") is None else np.abs(c["dS_T"][q])
        for t in range(c["cu"][q + 1] - 1, c["cu"][q] - 1, -1):
            R = f["a"][t] * (dr[t][..., None] * np.abs(f["C"][t])[:, None] + R)
            back = np.maximum(back, R.max(-1))
    return top, back


def backward(c):
    """Gradients of sum(dy y) + sum(dS_T S_T) and their largest errors."""
    f = _states(c)
    x, B, A, C, s, a = (f[k] for k in ("x", "B", "A", "C", "s", "a"))
    cu, N = c["cu"], len(c["cu"]) - 1
    T, H, d = x.shape
    dr = np.asarray(c["dy"], np.float64)
    edr = np.zeros_like(dr)
    g, e = {}, {}
    if c.get("z") is not None:
        z = np.asarray(c["z"], np.float64)
        raw, eraw = _raw(c, f)
        g["dz"] = dr * raw * cc.silu_grad(z)
        e["dz"] = np.abs(dr) * (np.abs(raw) * cc.silu_grad_error(z, 0.0) +
                                np.abs(cc.silu_grad(z)) * eraw) + 3 * U32 * np.abs(g["dz"])
        edr = np.abs(dr) * cc.silu_error(z, 0.0) + U32 * np.abs(dr * cc.silu(z))
        dr = dr * cc.silu(z)
    end = cu[-1]
    dr, edr = dr.copy(), edr.copy()
    dr[end:], edr[end:] = 0.0, 0.0
    r = np.zeros_like(f["S_T"]) if c.get("dS_T") is None else np.array(c["dS_T"], np.float64)
    er, mr = np.zeros_like(r), np.abs(r)
    G, eG = np.zeros_like(f["before"]), np.zeros_like(f["before"])
    for q in range(N):
        R, E, M = r[q], er[q], mr[q]
        for t in range(cu[q + 1] - 1, cu[q] - 1, -1):
            own = dr[t][..., None] * C[t][:, None]
            G[t] = own + R
            M = M + np.abs(own)
            eG[t] = E + edr[t][..., None] * np.abs(C[t])[:, None] + 2 * U32 * M
            E = a[t] * (eG[t] + f["rho"][t] * M + U32 * M)
            R = a[t] * G[t]
            M = a[t] * M
        r[q], er[q] = R, E
    aG = np.abs(G)
    u = s * x
    eu = f["es"] * np.abs(x) + U32 * np.abs(u)
    deep = DEEP * U32
    g["dS0"], e["dS0"] = r, er
    g["dB"] = np.einsum("thdn,thd->thn", G, u)
    e["dB"] = np.einsum("thdn,thd->thn", eG + deep * aG, np.abs(u)) + \
        np.einsum("thdn,thd->thn", aG, eu)
    g["dC"] = np.einsum("thdn,thd->thn", f["after"], dr)
    aft = np.abs(f["after"])
    e["dC"] = np.einsum("thdn,thd->thn", f["ea"] + deep * aft, np.abs(dr)) + \
        np.einsum("thdn,thd->thn", aft, edr)
    w = G * a * f["before"]
    ew = a * (eG * np.abs(f["before"]) + aG * f["eb"]) + np.abs(w) * (f["rho"] + 3 * U32)
    tokens = (max(1, end) + 16) * U32
    g["dA"] = np.einsum("thdn,thd->hdn", w, s)
    e["dA"] = np.einsum("thdn,thd->hdn", ew + tokens * np.abs(w), np.abs(s)) + \
        np.einsum("thdn,thd->hdn", np.abs(w), f["es"])
    gb = np.einsum("thdn,thn->thd", G, B)
    egb = np.einsum("thdn,thn->thd", eG + deep * aG, np.abs(B))
    wa = (w * A).sum(-1)
    ewa = ((ew + (deep + 2 * U32) * np.abs(w)) * np.abs(A)).sum(-1)
    ds = x * gb + wa
    eds = np.abs(x) * egb + ewa + 2 * U32 * (np.abs(x * gb) + np.abs(wa))
    g["ddt"] = ds * f["sig"]
    e["ddt"] = eds * f["sig"] + np.abs(ds) * f["esig"] + U32 * np.abs(g["ddt"])
    g["dx"] = s * gb
    e["dx"] = np.abs(s) * egb + f["es"] * np.abs(gb) + 2 * U32 * np.abs(g["dx"])
    if c.get("D") is not None:
        g["dx"] = g["dx"] + c["D"] * dr
        e["dx"] = e["dx"] + np.abs(c["D"]) * edr + 2 * U32 * np.abs(c["D"] * dr)
        g["dD"] = (dr * x).sum(0)
        e["dD"] = ((edr + tokens * np.abs(dr)) * np.abs(x)).sum(0)
    if c.get("dt_bias") is not None:
        g["ddt_bias"] = g["ddt"][:end].sum(0)
        e["ddt_bias"] = (e["ddt"] + tokens * np.abs(g["ddt"]))[:end].sum(0)
    return g, e
