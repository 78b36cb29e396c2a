"""The 64-bit references against differences and against each other (CPU)."""
import numpy as np
import pytest

import mixer_oracle as M


def _case(rng, b, L, H, G, dk, dv):
    return (rng.standard_normal((b, L, G, dk)),
            rng.standard_normal((b, L, G, dk)),
            rng.standard_normal((b, L, H, dv)),
            -np.abs(rng.standard_normal((b, L, H))) * 0.3)


@pytest.mark.parametrize("lengths", [None, [0, 4]])
def test_gradients_are_the_differences(lengths):
    rng = np.random.default_rng(3)
    b, L, H, G, dk, dv = 2, 5, 4, 2, 3, 2
    q, k, v, g = _case(rng, b, L, H, G, dk, dv)
    h0 = rng.standard_normal((b, H, dk, dv))
    dy = rng.standard_normal(v.shape)
    dh = rng.standard_normal(h0.shape)
    scale = 0.7
    grads = M.backward(q, k, v, g, scale, dy, h0, dh, lengths)

    def loss(**kw):
        a = dict(q=q, k=k, v=v, g=g, h0=h0)
        a.update(kw)
        y, S = M.forward(a["q"], a["k"], a["v"], a["g"], scale, a["h0"],
                         lengths)
        return (y * dy).sum() + (S * dh).sum()

    for name, ref, key in (("q", q, "dq"), ("k", k, "dk"), ("v", v, "dv"),
                           ("g", g, "dg"), ("h0", h0, "dh0")):
        for _ in range(12):
            at = tuple(rng.integers(0, n) for n in ref.shape)
            e = np.zeros_like(ref)
            e[at] = 1e-5
            diff = (loss(**{name: ref + e}) - loss(**{name: ref - e})) / 2e-5
            # central differences: h^2 times third derivatives, and 2^-53 / h
            assert abs(diff - grads[key][at]) <= 1e-7 * (1 + abs(diff)), (
                name, at)


def test_the_decay_restarts_the_state():
    rng = np.random.default_rng(4)
    q, k, v, g = _case(rng, 1, 8, 2, 1, 3, 4)
    g[0, 5] = -np.inf
    h0 = np.full((1, 2, 3, 4), np.nan)
    g0 = g.copy()
    g0[0, 0] = -np.inf
    y, S = M.forward(q, k, v, g0, 1.0, h0)
    assert np.all(np.isfinite(y)) and np.all(np.isfinite(S))
    tail, S2 = M.forward(q[:, 5:], k[:, 5:], v[:, 5:],
                         np.where(np.isinf(g[:, 5:]), 0.0, g[:, 5:]), 1.0)
    np.testing.assert_array_equal(y[:, 5:], tail)
    np.testing.assert_array_equal(S, S2)


def test_norm_gradients_are_the_differences():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 7)) + 2
    w, bias = rng.standard_normal(7), rng.standard_normal(7)
    dy, ds = rng.standard_normal(x.shape), rng.standard_normal(x.shape)
    s, mean, rstd, _ = M.norm_forward(x, None, w, bias, 1e-5, None)
    dx, dw, db = M.norm_backward(dy, s, mean, rstd, w, ds)

    def loss(x, w, bias):
        s, _, _, y = M.norm_forward(x, None, w, bias, 1e-5, None)
        return (y * dy).sum() + (s * ds).sum()

    for i in range(3):
        for j in range(7):
            e = np.zeros_like(x)
            e[i, j] = 1e-5
            d = (loss(x + e, w, bias) - loss(x - e, w, bias)) / 2e-5
            assert abs(d - dx[i, j]) <= 1e-7 * (1 + abs(d))
    for j in range(7):
        e = np.zeros(7)
        e[j] = 1e-5
        assert abs((loss(x, w + e, bias) - loss(x, w - e, bias)) / 2e-5
                   - dw[j]) <= 1e-7 * (1 + abs(dw[j]))
        assert abs((loss(x, w, bias + e) - loss(x, w, bias - e)) / 2e-5
                   - db[j]) <= 1e-7 * (1 + abs(db[j]))
