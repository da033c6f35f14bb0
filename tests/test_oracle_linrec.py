"""The gated linear recurrence's oracle (CPU): closed forms, finite differences of every
gradient, and the chunk states; and the beam oracle against a plain enumeration."""
import numpy as np
import pytest

from oracle import beam, linrec


def _case(seed, cu, H=2, d=3, S0=True):
    r = np.random.RandomState(seed)
    T, N = cu[-1], len(cu) - 1
    return (r.randn(T, H, d), 1 / (1 + np.exp(-r.randn(T, H, d) - 1)),
            r.randn(N, H, d) if S0 else None, r.randn(T, H, d), r.randn(N, H, d))


def test_constant_gate_closed_form():
    """a constant, x = 1: h_t = a^t S0 + (1 - a^t) / (1 - a); the complement's limit is 1."""
    a, T = 0.9, 40
    g = np.full((T, 1, 1), a)
    S0 = np.full((1, 1, 1), 2.0)
    h, S_T = linrec.forward(np.ones((T, 1, 1)), g, S0, [0, T])
    k = np.arange(1, T + 1)
    np.testing.assert_allclose(h[:, 0, 0], a ** k * 2.0 + (1 - a ** k) / (1 - a), rtol=1e-13)
    assert S_T[0, 0, 0] == h[-1, 0, 0]
    h, _ = linrec.forward(np.ones((T, 1, 1)), g, S0, [0, T], complement=True)
    np.testing.assert_allclose(h[:, 0, 0], a ** k * 2.0 + (1 - a ** k), rtol=1e-13)


def test_gate_zero_forgets_and_one_sums():
    x = np.arange(1.0, 7.0).reshape(6, 1, 1)
    h, _ = linrec.forward(x, np.zeros_like(x), np.full((1, 1, 1), 9.0), [0, 6])
    np.testing.assert_array_equal(h, x)
    h, _ = linrec.forward(x, np.ones_like(x), None, [0, 6])
    np.testing.assert_array_equal(h, np.cumsum(x, 0))


@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("layout", ["channel", "head", "log_bf16"])
def test_gradients_match_differences(complement, layout):
    cu = [0, 4, 4, 5, 9]
    x, a, S0, dy, dS = _case(1, cu)
    if layout == "head":
        a = np.broadcast_to(a[..., :1], a.shape).copy()
    got = linrec.backward(x, a, S0, cu, dy, dS, complement, layout)

    def loss(x, a, S0):
        h, S_T = linrec.forward(x, a, S0, cu, complement)
        return (dy * h).sum() + (dS * S_T).sum()

    eps, r = 1e-6, np.random.RandomState(2)
    vx, vs = r.randn(*x.shape), r.randn(*S0.shape)
    va = r.randn(*(a.shape[:2] if layout == "head" else a.shape))
    step = {"channel": lambda s: a + s * va, "head": lambda s: a + s * va[..., None],
            "log_bf16": lambda s: a * np.exp(s * va)}[layout]
    num = {"dx": (loss(x + eps * vx, a, S0) - loss(x - eps * vx, a, S0)) / (2 * eps),
           "dgate": (loss(x, step(eps), S0) - loss(x, step(-eps), S0)) / (2 * eps),
           "dS0": (loss(x, a, S0 + eps * vs) - loss(x, a, S0 - eps * vs)) / (2 * eps)}
    for name, v in (("dx", vx), ("dgate", va), ("dS0", vs)):
        # central differences: 1e-16 / eps of the loss plus eps^2, both near 1e-9
        assert abs((got[name] * v).sum() - num[name]) <= 1e-7 * (1 + abs(num[name])), name


def test_bounds_cover_32_bit_arithmetic():
    """The recurrence in fp32, token by token, stays within the bounds."""
    cu = [0, 30, 30, 97]
    x, a, S0, dy, dS = (None if v is None else v.astype(np.float32)
                        for v in _case(3, cu))
    h, _ = linrec.forward(x, a.astype(np.float64), S0, cu)
    _, e, _ = linrec.forward_bound(x, a.astype(np.float64), S0, cu, False, 0)
    s, worst = np.zeros_like(S0), 0.0
    s[:] = S0
    for n in range(len(cu) - 1):
        for t in range(cu[n], cu[n + 1]):
            s[n] = a[t] * s[n] + x[t]
            worst = max(worst, float((np.abs(s[n] - h[t]) / e[t]).max()))
    assert 0 < worst <= 1


def test_chunk_states():
    cu = [0, 4, 7, 20, 20]
    x, a, S0, _, _ = _case(4, cu)
    h, _ = linrec.forward(np.concatenate([x, x[:3]]), np.concatenate([a, a[:3]]), S0, cu)
    s = linrec.chunk_states(h, cu, 4)
    assert s.shape[0] == 6
    assert not s[0].any() and not s[1].any() and not s[5].any()   # starts, and past the end
    np.testing.assert_array_equal(s[2], h[7])
    np.testing.assert_array_equal(s[4], h[15])


def test_beam_select_matches_enumeration():
    r = np.random.RandomState(5)
    logits, scores = r.randn(6, 7), r.randn(2, 3)
    fin = np.array([[0, 1, 0], [0, 0, 0]])
    v, p, t = beam.select(logits, scores, 9, fin, eos=4)
    for b in range(2):
        every = []
        for k in range(3):
            z = np.exp(logits[b * 3 + k])
            for w in range(7):
                if fin[b, k]:
                    every.append((scores[b, k] if w == 4 else -np.inf, k * 7 + w))
                else:
                    every.append((scores[b, k] + np.log(z[w] / z.sum()), k * 7 + w))
        every.sort(key=lambda c: (-c[0], c[1]))
        assert [c[1] for c in every[:9]] == [(p[b, i] - b * 3) * 7 + t[b, i] for i in range(9)]
        np.testing.assert_allclose(v[b], [c[0] for c in every[:9]], rtol=1e-12)


def test_beam_select_dead_rows_and_reorder():
    logits = np.array([[1.0, np.nan, -np.inf], [-np.inf] * 3, [np.inf, 0.0, 2.0]])
    v, p, t = beam.select(logits, np.array([[-1.0, 0.0, -np.inf]]), 4)
    assert list(zip(p[0], t[0])) == [(0, 0), (0, 1), (0, 2), (1, 0)]
    assert v[0, 0] == -1.0 and np.isneginf(v[0, 1:]).all()
    s = np.arange(12.0).reshape(6, 2)
    got = beam.reorder(s, [1, 1, 0, 5, 2, -3], 3)
    np.testing.assert_array_equal(got[:, 0], [2, 2, 0, 10, 8, 10])
