"""Gated group norm of the heads: fp64 numpy reference, forward and backward.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Per (token, head): m = mean(x) or 0, r = 1 / sqrt(mean((x - m)^2) + eps), v = w (x - m) r + b, y =
v act(z) or act(v).  Layouts as in ``include/groupnorm.h``: x, z, dy [T, H, d], w, b [d] or
[H, d].  ``forward`` and ``backward`` also return, element by element, the largest error that
32-bit arithmetic leaves; sums over a head are at most DEEP additions deep.
"""
from __future__ import annotations

import numpy as np

from . import causalconv as cc

U32 = cc.U32
DEEP = 96


def _act(v, act):
    """act(v), its slope, and for an argument off by ev the errors of both."""
    if act == "silu":
        return cc.silu(v), cc.silu_grad(v), lambda ev: cc.silu_error(v, ev), \
            lambda ev: cc.silu_grad_error(v, ev)
    if act == "sigmoid":
        s = cc.sigmoid(v)
        return s, s * (1 - s), lambda ev: 0.25 * ev + s * cc.sigmoid_rel(v) + 1e-36, \
            lambda ev: 0.1 * ev + s * (1 - s) * 4 * U32 + \
            s * np.abs(1 - 2 * s) * cc.sigmoid_rel(v) + U32 * s + 1e-36
    one = np.ones_like(v)
    return v, one, lambda ev: ev, lambda ev: 0.0 * one


def _norm(x, w, b, center, eps):
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    m = x.mean(-1, keepdims=True) if center else np.zeros_like(x[..., :1])
    em = (DEEP + 1) * U32 * np.abs(x).mean(-1, keepdims=True) if center else 0.0
    xc = x - m
    exc = em + (U32 * np.abs(xc) if center else 0.0) + np.zeros_like(x)
    q = (xc * xc).sum(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = 1.0 / np.sqrt(q / d + eps)
        rel = 0.5 * ((2 * np.abs(xc) * exc + exc * exc).sum(-1, keepdims=True) + DEEP * U32 * q) / \
            (q + d * eps) + 4 * U32
    xh = xc * r
    exh = exc * r + np.abs(xh) * (rel + U32)
    w = 1.0 if w is None else np.asarray(w, np.float64)
    b = 0.0 if b is None else np.asarray(b, np.float64)
    v = w * xh + b
    return xh, exh, r, rel, w, v, np.abs(w) * exh + 2 * U32 * (np.abs(w * xh) + np.abs(b))


def forward(x, w, b, z, act, center, eps):
    """Returns y and its largest error before the rounding to its type."""
    xh, _, _, _, _, v, ev = _norm(x, w, b, center, eps)
    if z is None:
        y, _, err, _ = _act(v, act)
        return y, err(ev)
    f, _, err, _ = _act(np.asarray(z, np.float64), act)
    return v * f, np.abs(f) * ev + np.abs(v) * err(0.0) + U32 * np.abs(v * f)


def backward(x, w, b, z, act, center, eps, dy):
    """Returns (dx, dz, dw, db) and their largest errors, as dicts."""
    dy = np.asarray(dy, np.float64)
    xh, exh, r, rel, wv, v, ev = _norm(x, w, b, center, eps)
    d, T = dy.shape[-1], dy.shape[0]
    g, e = {}, {}
    if z is None:
        _, slope, _, serr = _act(v, act)
        dv = dy * slope
        edv = np.abs(dy) * serr(ev) + U32 * np.abs(dv)
    else:
        f, slope, ferr, serr = _act(np.asarray(z, np.float64), act)
        dv = dy * f
        edv = np.abs(dy) * ferr(0.0) + U32 * np.abs(dv)
        g["dz"] = dy * v * slope
        e["dz"] = np.abs(dy) * (np.abs(v) * serr(0.0) + np.abs(slope) * ev) + 3 * U32 * np.abs(g["dz"])
    gv = dv * wv
    egv = np.abs(wv) * edv + U32 * np.abs(gv)
    mean = lambda a: a.mean(-1, keepdims=True)
    s1 = mean(gv * xh)
    es1 = mean(egv * np.abs(xh) + np.abs(gv) * exh) + (DEEP + 2) * U32 * mean(np.abs(gv * xh))
    s2 = mean(gv) if center else 0.0 * s1
    es2 = mean(egv) + (DEEP + 2) * U32 * mean(np.abs(gv)) if center else 0.0 * s1
    inner = gv - xh * s1 - s2
    mag = np.abs(gv) + np.abs(xh * s1) + np.abs(s2)
    g["dx"] = r * inner
    e["dx"] = r * (egv + np.abs(xh) * es1 + np.abs(s1) * exh + es2 + 4 * U32 * mag) + \
        np.abs(r * inner) * (rel + U32)
    deep = (T * dy.shape[1] + 16) * U32
    for name, val, err in (("dw", dv * xh, edv * np.abs(xh) + np.abs(dv) * exh), ("db", dv, edv)):
        par = w if name == "dw" else b
        if par is None:
            continue
        over = (0, 1) if np.ndim(par) == 1 else (0,)
        g[name] = val.sum(over)
        e[name] = (err + deep * np.abs(val)).sum(over)
    return g, e
