"""Beam search over states: fp64 numpy reference of the selection and the moves.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

``select``: the value of candidate (beam k, token v) is
scores[k] + logits[k, v] - log sum_w exp(logits[k, w]); a finished beam has the
one candidate (k, eos) at scores[k]; every other candidate of it is -inf.  The
best come first, equal values by k V + v.  NaN counts as -inf, +inf as the
largest finite float.
"""
from __future__ import annotations

import numpy as np


def _tame(x):
    x = np.asarray(x, dtype=np.float64)
    big = float(np.finfo(np.float32).max)
    return np.minimum(np.where(np.isnan(x), -np.inf, x), big)


def candidates(logits, scores, finished=None, eos=0):
    """Values of all candidates of one request: logits [K, V], scores [K] -> [K, V]."""
    x, sc = _tame(logits), _tame(scores)
    K, V = x.shape
    out = np.full((K, V), -np.inf)
    for k in range(K):
        if finished is not None and finished[k]:
            out[k, eos] = sc[k]
            continue
        top = x[k].max()
        if top == -np.inf or sc[k] == -np.inf:
            continue
        out[k] = sc[k] + (x[k] - (top + np.log(np.exp(x[k] - top).sum())))
    return out


def select(logits, scores, num_out, finished=None, eos=0):
    """logits [B K, V], scores [B, K] -> (values [B, n] fp64, parents, tokens [B, n])."""
    B, K = scores.shape
    V = logits.shape[1]
    vals, par, tok = [], [], []
    for b in range(B):
        c = candidates(logits[b * K:(b + 1) * K], scores[b],
                       None if finished is None else finished[b], eos).reshape(-1)
        pick = np.argsort(-c, kind="stable")[:num_out]
        vals.append(c[pick])
        par.append(b * K + pick // V)
        tok.append(pick % V)
    return np.array(vals), np.array(par), np.array(tok)


def reorder(state, parents, K):
    """Row i becomes the old row parents[i]; an entry outside the request leaves its row."""
    out = state.copy()
    for i, p in enumerate(parents):
        base = i // K * K
        if base <= p < base + K:
            out[i] = state[p]
    return out
