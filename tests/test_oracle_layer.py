"""The oracles of the operators around a layer's recurrence (CPU): library routines, closed forms
and central differences of every gradient."""
import numpy as np
import pytest
import torch

from oracle import causalconv as cc
from oracle import groupnorm as gn
from oracle import linrec
from oracle import selscan as ss

CU = [0, 4, 4, 5, 7, 12]


def _differences(loss, tensors, grads, eps=1e-6, picks=12):
    r = np.random.RandomState(7)
    for name, t in tensors.items():
        flat, got = t.reshape(-1), np.asarray(grads[name]).reshape(-1)
        for i in r.permutation(flat.size)[:picks]:
            keep = flat[i]
            flat[i] = keep + eps
            up = loss()
            flat[i] = keep - eps
            down = loss()
            flat[i] = keep
            want = (up - down) / (2 * eps)
            assert abs(got[i] - want) <= 2e-7 * max(1.0, abs(want)), (name, i, got[i], want)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act", [False, True])
def test_conv_is_the_library_routine(W, act):
    r = np.random.RandomState(W)
    x, w, b = r.randn(9, 5), r.randn(5, W), r.randn(5)
    S0 = r.randn(1, W - 1, 5)
    y, S_T, _ = cc.forward(x, w, b, S0, [0, 9], act)
    full = torch.tensor(np.concatenate([S0[0], x]).T[None])
    v = torch.nn.functional.conv1d(full, torch.tensor(w)[:, None], torch.tensor(b), groups=5)
    v = torch.nn.functional.silu(v) if act else v
    np.testing.assert_allclose(y, v[0].T.numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_array_equal(S_T[0], np.concatenate([S0[0], x])[-(W - 1):])


def test_conv_short_sequences_keep_the_state():
    S0 = np.arange(6.0).reshape(2, 3, 1)
    _, S_T, _ = cc.forward(np.array([[9.0]]), np.ones((1, 4)), None, S0, [0, 0, 1], False)
    np.testing.assert_array_equal(S_T[:, :, 0], [[0, 1, 2], [4, 5, 9]])


@pytest.mark.parametrize("act", [False, True])
def test_conv_gradients_match_differences(act):
    r = np.random.RandomState(3)
    N, W, D = len(CU) - 1, 4, 3
    t = dict(dx=r.randn(CU[-1] + 1, D), dw=r.randn(D, W), db=r.randn(D), dS0=r.randn(N, W - 1, D))
    dy, dS = r.randn(CU[-1] + 1, D), r.randn(N, W - 1, D)

    def loss():
        y, S_T, _ = cc.forward(t["dx"], t["dw"], t["db"], t["dS0"], CU, act)
        return (dy * y)[:CU[-1]].sum() + (dS * S_T).sum()

    g, e = cc.backward(t["dx"], t["dw"], t["db"], t["dS0"], CU, dy, dS, act)
    _differences(loss, t, g)
    assert all((e[k] >= 0).all() and e[k].shape == g[k].shape for k in g)


@pytest.mark.parametrize("center", [False, True])
def test_norm_is_the_library_routine(center):
    r = np.random.RandomState(1)
    x, w, b = r.randn(6, 3, 8), r.randn(3, 8), r.randn(3, 8)
    y, _ = gn.forward(x, w, b, None, "none", center, 1e-5)
    tx = torch.tensor(x)
    if center:
        want = torch.nn.functional.group_norm(tx.reshape(6, 24), 3, torch.tensor(w.reshape(-1)),
                                              torch.tensor(b.reshape(-1)), 1e-5).reshape(6, 3, 8)
    else:
        want = tx / torch.sqrt((tx ** 2).mean(-1, keepdim=True) + 1e-5) * torch.tensor(w) + \
            torch.tensor(b)
    np.testing.assert_allclose(y, want.numpy(), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("center,shape", [(False, (4,)), (True, (3, 4))])
def test_norm_gradients_match_differences(act, gated, center, shape):
    r = np.random.RandomState(2)
    t = dict(dx=r.randn(5, 3, 4), dw=r.randn(*shape), db=r.randn(*shape))
    if gated:
        t["dz"] = r.randn(5, 3, 4)
    dy = r.randn(5, 3, 4)

    def loss():
        return (dy * gn.forward(t["dx"], t["dw"], t["db"], t.get("dz"), act, center, 1e-3)[0]).sum()

    g, e = gn.backward(t["dx"], t["dw"], t["db"], t.get("dz"), act, center, 1e-3, dy)
    assert set(g) == set(t)
    _differences(loss, t, g)
    assert all((e[k] >= 0).all() for k in g)


def _scan_case(softplus=True, gated=True, seed=0):
    r = np.random.RandomState(seed)
    T, H, d, n, N = CU[-1] + 1, 2, 3, 4, len(CU) - 1
    return dict(x=r.randn(T, H, d), dt=r.randn(T, H, d) * 0.5 + (0 if softplus else 1.0),
                A=-np.exp(r.randn(H, d, n)), B=r.randn(T, H, n), C=r.randn(T, H, n),
                D=r.randn(H, d), dt_bias=r.randn(H, d) * 0.2, z=r.randn(T, H, d) if gated else None,
                S0=r.randn(N, H, d, n), cu=CU, softplus=softplus, dy=r.randn(T, H, d),
                dS_T=r.randn(N, H, d, n))


def test_scan_of_one_value_is_the_gated_recurrence():
    """n = 1, B = C = 1, no skip: h_t = exp(s A) h + s x, the linear recurrence's own oracle."""
    c = _scan_case(softplus=False, gated=False)
    c["A"], c["S0"] = c["A"][..., :1], c["S0"][..., :1]
    c["B"] = c["C"] = np.ones(c["B"].shape[:2] + (1,))
    c["D"] = c["dt_bias"] = None
    f, _ = ss.forward(c)
    s = c["dt"]
    h, S_T = linrec.forward(s * c["x"], np.exp(s * c["A"][..., 0]), c["S0"][..., 0], CU)
    np.testing.assert_allclose(f["y"][:CU[-1]], h[:CU[-1]], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(f["S_T"][..., 0], S_T, rtol=1e-12, atol=1e-12)


def test_scan_constant_input_has_its_limit():
    """A constant step, input and projection: h -> s x B / (1 - exp(s A))."""
    T = 400
    one = np.ones((T, 1, 1))
    c = dict(x=2 * one, dt=0.5 * one, A=-np.ones((1, 1, 1)), B=3 * one, C=one, cu=[0, T],
             softplus=False)
    f, _ = ss.forward(c)
    np.testing.assert_allclose(f["y"][-1, 0, 0], 0.5 * 2 * 3 / (1 - np.exp(-0.5)), rtol=1e-12)


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_scan_gradients_match_differences(softplus, gated):
    c = _scan_case(softplus, gated)
    names = ["x", "dt", "A", "B", "C", "D", "dt_bias", "S0"] + (["z"] if gated else [])

    def loss():
        f, _ = ss.forward(c)
        return (c["dy"] * f["y"])[:CU[-1]].sum() + (c["dS_T"] * f["S_T"]).sum()

    g, e = ss.backward(c)
    assert set(g) == {"d" + k for k in names}
    for name in g:   # rows past the last sequence count for nothing
        if g[name].shape[0] == CU[-1] + 1:
            g[name][CU[-1]:] = 0.0
        assert e[name].shape == g[name].shape and (e[name] >= 0).all()
    _differences(loss, {"d" + k: c[k] for k in names}, g)
