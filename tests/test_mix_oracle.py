"""The lapmix oracle against itself: closed forms, and its gradients against central
differences of its forward."""

import numpy as np
import pytest

from oracle import lapmix_oracle as O


def _inputs(B=2, H=2, N=7, d=3, seed=0):
    r = np.random.default_rng(seed)
    return (r.standard_normal((B, H, N, d)), r.standard_normal((B, H, N, d)) - 0.5,
            r.standard_normal((B, H, d)), r.standard_normal((B, H, N, d)), r.standard_normal((B, H, d)))


def test_constant_gate_is_a_geometric_sum():
    N, f = 12, 0.75
    x = np.ones((1, 1, N, 1))
    g = np.full_like(x, np.log(f))
    got = O.scan(x, g, log_gate=True)["y"][0, 0, :, 0]
    np.testing.assert_allclose(got, (1 - f ** np.arange(1, N + 1)) / (1 - f), rtol=1e-14)
    coupled = O.scan(x, g, log_gate=True, coupled=True)["y"][0, 0, :, 0]
    np.testing.assert_allclose(coupled, 1 - f ** np.arange(1, N + 1), rtol=1e-14)


def test_gate_of_minus_infinity_starts_anew():
    x, g, h0, _, _ = _inputs()
    for log_gate in (False, True):
        cut = g.copy()
        cut[:, :, 4] = -np.inf
        y = O.scan(x, cut, h0, log_gate=log_gate)["y"]
        tail = O.scan(x[:, :, 5:], g[:, :, 5:], x[:, :, 4], log_gate=log_gate)["y"]
        np.testing.assert_array_equal(y[:, :, 5:], tail)


@pytest.mark.parametrize("log_gate", [False, True])
@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("lengths", [None, [5, 1], [0, 7]])
def test_scan_gradients_against_differences(log_gate, coupled, lengths):
    """Central differences with step 1e-5: their own error is about 1e-10 (third derivatives and
    rounding), well below the 1e-7 asked for."""
    x, g, h0, dy, dhN = _inputs()

    def loss(x, g, h0):
        r = O.scan(x, g, h0, lengths, log_gate, coupled)
        return (r["y"] * dy).sum() + (r["hN"] * dhN).sum()

    got = O.scan_backward(x, g, dy, h0, dhN, lengths, log_gate, coupled)
    for name, t in (("dx", x), ("dg", g), ("dh0", h0)):
        num = np.empty_like(t)
        for at in np.ndindex(t.shape):
            keep, e = t[at], 1e-5
            t[at] = keep + e
            up = loss(x, g, h0)
            t[at] = keep - e
            num[at] = (up - loss(x, g, h0)) / (2 * e)
            t[at] = keep
        np.testing.assert_allclose(got[name], num, atol=1e-7, err_msg=name)


def test_norm_gradients_against_differences():
    r = np.random.default_rng(1)
    s, w, dy, ds = r.standard_normal((3, 9)), r.standard_normal(9), r.standard_normal((3, 9)), r.standard_normal((3, 9))

    def loss(s, w):
        return (O.norm(s, w, 1e-3)[0] * dy).sum() + (ds * s).sum()

    dr, dw, _, _ = O.norm_backward(dy, s, w, 1e-3, ds)
    for got, t in ((dr, s), (dw, w)):
        num = np.empty_like(t)
        for at in np.ndindex(t.shape):
            keep, e = t[at], 1e-5
            t[at] = keep + e
            up = loss(s, w)
            t[at] = keep - e
            num[at] = (up - loss(s, w)) / (2 * e)
            t[at] = keep
        np.testing.assert_allclose(got, num, atol=1e-7)


def test_norm_rows_have_unit_mean_square():
    r = np.random.default_rng(2)
    y, _ = O.norm(r.standard_normal((4, 50)) * 7, np.ones(50), 1e-12)
    np.testing.assert_allclose((y * y).mean(1), 1.0, rtol=1e-10)


def test_float32_evaluation_stays_within_the_bounds():
    """A float32 run of the recurrence, token by token, lies within e_y of float64."""
    x, g, h0, _, _ = (t.astype(np.float32) for t in _inputs(1, 1, 400, 8, seed=3))
    ref = O.scan(x.astype(np.float64), g.astype(np.float64), h0.astype(np.float64))
    h, one = h0, np.float32(1)
    for n in range(400):
        h = one / (one + np.exp(-g[:, :, n])) * h + x[:, :, n]
        assert np.all(np.abs(h - ref["y"][:, :, n]) <= ref["e_y"][:, :, n])
    assert np.all(ref["e_y"] <= 1e-4)
