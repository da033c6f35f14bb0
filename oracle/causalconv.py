"""Short causal convolution: fp64 numpy reference, forward and backward.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Per (sequence, channel): v_t = b + sum_j w_j x_{t-W+1+j}, y_t = v_t or silu(v_t), one token at
a time.  Layouts as in ``include/causalconv.h`` with the channels flat: x [T, D], w [D, W], b
[D], states [N, W-1, D].  The ``*_bound`` functions give, element by element, the largest error
that 32-bit arithmetic leaves: u = 2^-24 for a rounding, and for the sigmoid the published
error of the fast exponential (2 + 1.173 |v| units in the last place) and of the fast division
(2 units).
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24   # largest relative error of one rounding to fp32


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def silu(v):
    return v * sigmoid(v)


def silu_grad(v):
    s = sigmoid(v)
    return s * (1.0 + v * (1.0 - s))


def sigmoid_rel(v):
    """Relative error of 1 / (1 + e^-v): the exponential's, as far as it counts, one addition,
    one division, and one product behind it."""
    return (2.0 + 1.2 * np.abs(v)) * 2 * U32 * (1.0 - sigmoid(v)) + 8 * U32


def silu_error(v, ev):
    """Error of silu(v) for an argument that is off by ev (its slope is at most 1.1)."""
    return 1.1 * ev + np.abs(silu(v)) * sigmoid_rel(v) + 1e-36


def silu_grad_error(v, ev):
    """Error of silu'(v) (its slope is at most 0.5)."""
    s = sigmoid(v)
    return 0.5 * ev + np.abs(s * (1.0 + v * (1.0 - 2.0 * s))) * sigmoid_rel(v) + \
        6 * U32 * s * (1.0 + np.abs(v) * (1.0 - s)) + np.abs(v) * s * s * sigmoid_rel(v) + 1e-36


def _history(x, S0, cu, W):
    """Each token's W inputs [T, W, D], and the final states."""
    N, D = len(cu) - 1, x.shape[1]
    S0 = np.zeros((N, W - 1, D)) if S0 is None else np.asarray(S0, np.float64)
    win, S_T = np.zeros((x.shape[0], W, D)), np.zeros((N, W - 1, D))
    for n in range(N):
        past = [S0[n, j] for j in range(W - 1)]
        for t in range(cu[n], cu[n + 1]):
            past.append(x[t])
            for j in range(W):
                win[t, j] = past[len(past) - W + j]
        for j in range(W - 1):
            S_T[n, j] = past[len(past) - (W - 1) + j]
    return win, S_T


def forward(x, w, b, S0, cu, act=True):
    """Returns (y [T, D], S_T [N, W-1, D]) and the largest error of y before its rounding."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    win, S_T = _history(x, S0, cu, w.shape[1])
    v = np.einsum("twd,dw->td", win, w)
    mag = np.einsum("twd,dw->td", np.abs(win), np.abs(w))
    if b is not None:
        v, mag = v + b, mag + np.abs(b)
    ev = (w.shape[1] + 1) * U32 * mag
    return (silu(v) if act else v), S_T, (silu_error(v, ev) if act else ev)


def backward(x, w, b, S0, cu, dy, dS_T=None, act=True):
    """Gradients of sum(dy y) + sum(dS_T S_T) (dx, dw, db, dS0) and the largest errors."""
    x, w, dy = (np.asarray(a, np.float64) for a in (x, w, dy))
    W, N, D = w.shape[1], len(cu) - 1, x.shape[1]
    win, _ = _history(x, S0, cu, W)
    v = np.einsum("twd,dw->td", win, w)
    mag = np.einsum("twd,dw->td", np.abs(win), np.abs(w))
    if b is not None:
        v, mag = v + b, mag + np.abs(b)
    ev = (W + 1) * U32 * mag
    dv = dy * silu_grad(v) if act else dy
    edv = np.abs(dy) * (silu_grad_error(v, ev) if act else 0.0) + U32 * np.abs(dv)
    end = cu[-1]
    dv[end:], edv[end:] = 0.0, 0.0
    dx, edx = np.zeros_like(x), np.zeros_like(x)
    dS0, eS0 = np.zeros((N, W - 1, D)), np.zeros((N, W - 1, D))
    for n in range(N):
        L = cu[n + 1] - cu[n]
        col, ecol = np.zeros((W - 1 + L, D)), np.zeros((W - 1 + L, D))
        mcol = np.zeros((W - 1 + L, D))
        for t in range(L):
            for j in range(W):
                col[t + j] += w[:, j] * dv[cu[n] + t]
                mcol[t + j] += np.abs(w[:, j] * dv[cu[n] + t])
                ecol[t + j] += np.abs(w[:, j]) * edv[cu[n] + t]
        if dS_T is not None:
            col[L:] += dS_T[n]
            mcol[L:] += np.abs(dS_T[n])
        ecol += (W + 2) * U32 * mcol
        dS0[n], eS0[n] = col[:W - 1], ecol[:W - 1]
        dx[cu[n]:cu[n + 1]], edx[cu[n]:cu[n + 1]] = col[W - 1:], ecol[W - 1:]
    # a sum over the tokens is at most as many additions deep as there are tokens
    deep = (max(1, end) + 16) * U32
    grads = {"dx": dx, "dS0": dS0, "dw": np.einsum("td,twd->dw", dv[:end], win[:end]),
             "db": dv.sum(0)}
    bounds = {"dx": edx, "dS0": eS0,
              "dw": np.einsum("td,twd->dw", edv[:end] + deep * np.abs(dv[:end]),
                              np.abs(win[:end])),
              "db": (edv + deep * np.abs(dv)).sum(0)}
    return grads, bounds
