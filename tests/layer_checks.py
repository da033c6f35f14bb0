"""Shared by the tests of the operators around a layer's recurrence."""
import numpy as np
import torch

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2

LENS = {
    "one_token": [1],
    "short": [2, 1, 3, 0, 2],
    "tile": [32],
    "tile_and_one": [33],
    "several_tiles": [200],
    "ragged": [3, 0, 70, 1, 0, 0, 97, 32, 16, 2],
    "all_empty": [0, 0, 0],
    "none": [],
    "many_short": [1, 2, 0, 3, 1] * 30,
}


def offsets(lens):
    """(host list, int32 tensor)"""
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu, torch.tensor(cu, dtype=torch.int32)


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def cuda(c):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def within(name, got, want, bound, rounded=False):
    """Every element within its bound, plus half a step of bf16 where it was rounded; below
    the smallest normal number a rounding is absolute."""
    got, want = np64(got), np.asarray(want)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.isfinite(got).all(), name
    tol = np.asarray(bound) + 2.0 ** -126
    if rounded:
        tol = tol * (1 + BF16_HALF) + BF16_HALF * np.abs(want)
    off = np.abs(got - want) - tol
    bad = off > 0
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} beyond, worst by {off.max():.3g} " \
        f"at {np.unravel_index(off.argmax(), off.shape)}"


def wide_rows(t, left, right):
    """The same rows inside wider ones: `left` and `right` elements of NaN around each."""
    T = t.shape[0]
    w = t[0].numel() if T else 0
    big = torch.full((T, left + w + right), float("nan"), dtype=t.dtype, device=t.device)
    big[:, left:left + w] = t.reshape(T, -1)
    return big[:, left:left + w].view(t.shape) if t.dim() == 2 else \
        big[:, left:left + w].unflatten(1, t.shape[1:])
