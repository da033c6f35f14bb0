"""Gated linear recurrence: fp64 numpy reference, forward and backward.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Per (sequence, head, channel): h_t = a_t h_{t-1} + u_t, u_t = x_t or
(1 - a_t) x_t, one token at a time.  ``backward`` is the reverse mode of that
line.  ``forward_bound`` and ``backward_bound`` run the same lines on
magnitudes: the largest error that 32-bit arithmetic of the recurrence, in any
grouping along the sequence, can leave in each output.

Layouts as in ``include/linrec.h``; x, dy, states any float type, the gate per
channel (``expand_gate``).
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24   # largest relative error of one rounding to fp32


def expand_gate(gate, layout: str, shape):
    """The gate per channel [T, H, d] in fp64 from its stored layout."""
    g = np.asarray(gate, dtype=np.float64)
    if layout == "log_bf16":
        return np.exp(g)
    if layout == "head":
        return np.broadcast_to(g[..., None], shape).copy()
    return g


def forward(x, a, S0, cu, complement=False):
    """Returns (h [T, H, d], S_T [N, H, d]); tokens past cu[-1] get 0."""
    x = np.asarray(x, dtype=np.float64)
    u = (1.0 - a) * x if complement else x
    N = len(cu) - 1
    h = np.zeros_like(x)
    S_T = np.zeros((N,) + x.shape[1:]) if S0 is None else np.array(S0, dtype=np.float64)
    for n in range(N):
        for t in range(cu[n], cu[n + 1]):
            S_T[n] = a[t] * S_T[n] + u[t]
            h[t] = S_T[n]
    return h, S_T


def chunk_states(h, cu, chunk):
    """State that reaches token i * chunk (0 where it starts a sequence or is past the last)."""
    T = h.shape[0]
    out = np.zeros((-(-T // chunk),) + h.shape[1:])
    starts = set(cu[:-1])
    for i in range(out.shape[0]):
        t = i * chunk
        if 0 < t < cu[-1] and t not in starts:
            out[i] = h[t - 1]
    return out


def backward(x, a, S0, cu, dy, dS_T=None, complement=False, layout="channel"):
    """Gradients of sum(dy * y) + sum(dS_T * S_T): dx, dgate (in the gate's layout), dS0."""
    x = np.asarray(x, dtype=np.float64)
    dy = np.asarray(dy, dtype=np.float64)
    h, _ = forward(x, a, S0, cu, complement)
    N = len(cu) - 1
    r = np.zeros((N,) + x.shape[1:]) if dS_T is None else np.array(dS_T, dtype=np.float64)
    dx, da = np.zeros_like(x), np.zeros_like(x)
    for n in range(N):
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            g = dy[t] + r[n]
            prev = h[t - 1] if t > cu[n] else (0.0 if S0 is None else np.asarray(S0[n], np.float64))
            dx[t] = (1.0 - a[t]) * g if complement else g
            da[t] = g * (prev - x[t]) if complement else g * prev
            r[n] = a[t] * g
    dgate = da.sum(-1) if layout == "head" else a * da if layout == "log_bf16" else da
    return {"dx": dx, "dgate": dgate, "dS0": r}


def _magnitudes(u, a, S, cu, ulps):
    """For h = a h + u: m (the same with magnitudes) and e, the error bound.  A step rounds
    its result once and the products of gates it joins once more each way; `ulps` more
    roundings are in the gate and the input themselves.  Each is at most U32 of m_t, and
    an error made at one token decays with the state."""
    m, e = np.zeros_like(u), np.zeros_like(u)
    Sm, Se = np.abs(S), np.zeros_like(S)
    for n in range(len(cu) - 1):
        for t in range(cu[n], cu[n + 1]):
            Sm[n] = np.abs(a[t]) * Sm[n] + np.abs(u[t])
            Se[n] = np.abs(a[t]) * Se[n] + (2 + ulps) * U32 * Sm[n]
            m[t], e[t] = Sm[n], Se[n]
    return m, e, Sm, Se


def forward_bound(x, a, S0, cu, complement, ulps):
    """(m, e [T, H, d], e of S_T): see ``_magnitudes``."""
    x = np.asarray(x, dtype=np.float64)
    u = np.abs((1.0 - a) * x if complement else x)
    S = np.zeros((len(cu) - 1,) + x.shape[1:]) if S0 is None else np.array(S0, np.float64)
    m, e, _, Se = _magnitudes(u, a, S, cu, ulps)
    return m, e, Se


def backward_bound(x, a, S0, cu, dy, dS_T, complement, layout, ulps):
    """Largest error of each gradient, as ``backward`` returns them."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    m, e, _ = forward_bound(x, a, S0, cu, complement, ulps)
    T, N = x.shape[0], len(cu) - 1
    # r_t = a_t (dy_t + r_{t+1}): the same recurrence on reversed tokens
    end = cu[-1]
    rcu = [end - c for c in cu[::-1]]
    S = np.zeros((N,) + x.shape[1:]) if dS_T is None else np.array(dS_T, np.float64)[::-1].copy()
    ar = a[:end][::-1]
    ur = np.abs(ar * np.asarray(dy, np.float64)[:end][::-1])
    rm, re, _, Se = _magnitudes(ur, ar, S, rcu, ulps + 1)
    gm, ge = np.zeros_like(x), np.zeros_like(x)
    ends = {cu[n + 1] - 1: n for n in range(N) if cu[n + 1] > cu[n]}
    prev_m, prev_e = np.zeros_like(x), np.zeros_like(x)
    for t in range(end):
        if t in ends:
            rmt, ret = (np.zeros(x.shape[1:]) if dS_T is None
                        else np.abs(np.asarray(dS_T[ends[t]], np.float64))), 0.0
        else:
            rmt, ret = rm[end - 2 - t], re[end - 2 - t]
        gm[t] = np.abs(np.asarray(dy[t], np.float64)) + rmt
        ge[t] = ret + U32 * gm[t]
        if t not in set(cu[:-1]):
            prev_m[t], prev_e[t] = m[t - 1], e[t - 1]
    if S0 is not None:
        for n in range(N):
            if cu[n + 1] > cu[n]:
                prev_m[cu[n]] = np.abs(np.asarray(S0[n], np.float64))
    na = np.abs(1.0 - a) if complement else np.ones_like(a)
    dx = na * ge + (1 + ulps) * U32 * na * gm
    f_m, f_e = prev_m + (x if complement else 0.0), prev_e + U32 * (prev_m + x)
    da = gm * f_e + ge * f_m + 2 * U32 * gm * f_m
    if layout == "log_bf16":
        da = np.abs(a) * (da + (1 + ulps) * U32 * gm * f_m)
    elif layout == "head":
        da = da.sum(-1) + x.shape[-1] * U32 * (gm * f_m).sum(-1)
    return {"dx": dx, "dgate": da, "dS0": Se[::-1]}
