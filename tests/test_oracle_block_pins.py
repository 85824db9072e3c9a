"""Pins of oracle/block_ref.py: published known answers of the generator,
hand-derived norm rows, and gradients against central differences."""

import numpy as np
import pytest

from oracle import block_ref as B


def test_philox_known_answers():
    """The known-answer vectors of the generator's authors (Random123)."""
    f = 0xFFFFFFFF
    cases = [
        ((0, 0, 0, 0), (0, 0),
         (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
        ((f, f, f, f), (f, f),
         (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
        ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344),
         (0xA4093822, 0x299F31D0),
         (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]
    for c, k, want in cases:
        got = tuple(int(w[0]) for w in B.philox4x32(c, k))
        assert got == want


def test_dropout_draw_order_and_rate():
    d = B.dropout_draws(16, 5, (7 << 32) + 9)
    w = B.philox4x32([1, 0, 9, 7], [5, 0])
    assert d[8] == int(w[0][0]) & 0xFFFF and d[9] == int(w[0][0]) >> 16
    assert d[15] == int(w[3][0]) >> 16
    # a shifted window of the same stream
    np.testing.assert_array_equal(B.dropout_draws(8, 5, (7 << 32) + 9, 8),
                                  d[8:])
    x = np.ones(1 << 16)
    y, keep = B.dropout(x, None, 0.25, 3, 4)
    # binomial: 6 sigma of 65536 draws at p = 1/4 is 0.0101
    assert abs(keep.mean() - 0.75) < 0.0102
    assert set(np.unique(y)) == {0.0, 4.0 / 3.0}
    assert B.dropout(x, x, 1.0, 3, 4)[0].max() == 1.0
    assert B.dropout(x, None, 0.0, 3, 4)[1].all()


def test_norm_by_hand():
    # row (1, 2, 3, 6): mean 3, centred (-2, -1, 0, 3), variance 14/4
    x = np.array([[1.0, 2.0, 3.0, 6.0]])
    g, b = np.array([1.0, 2.0, 1.0, 1.0]), np.array([0.0, 0.0, 5.0, 0.0])
    y, mean, rstd = B.norm_forward(x, g, b, 0.0, rms=False)
    r = np.sqrt(2.0 / 7.0)
    np.testing.assert_allclose(y, [[-2 * r, -2 * r, 5.0, 3 * r]], rtol=1e-15)
    assert mean[0] == 3.0 and abs(rstd[0] - r) < 1e-15
    # RMS: mean square 50/4
    y, _, rstd = B.norm_forward(x, g, None, 0.0, rms=True)
    np.testing.assert_allclose(rstd, [np.sqrt(4.0 / 50.0)], rtol=1e-15)
    np.testing.assert_allclose(y[0, 1], 4 * np.sqrt(0.08), rtol=1e-15)


def _diff(fun, arr, v, h=1e-5):
    return (fun(arr + h * v) - fun(arr - h * v)) / (2 * h)


@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradient_is_the_difference_quotient(rms):
    r = np.random.default_rng(0)
    x, dy = r.normal(size=(3, 8)) + 0.5, r.normal(size=(3, 8))
    g, b = r.normal(size=8), None if rms else r.normal(size=8)
    dx, dg, db = B.norm_backward(dy, x, g, 1e-3, rms)
    L = lambda x_, g_, b_: float(  # noqa: E731
        (B.norm_forward(x_, g_, b_, 1e-3, rms)[0] * dy).sum())
    v = r.normal(size=x.shape)
    assert abs(_diff(lambda t: L(t, g, b), x, v) - (dx * v).sum()) < 1e-8
    v = r.normal(size=8)
    assert abs(_diff(lambda t: L(x, t, b), g, v) - (dg * v).sum()) < 1e-8
    if not rms:
        assert abs(_diff(lambda t: L(x, g, t), b, v) - (db * v).sum()) < 1e-8


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_ffn_gradient_is_the_difference_quotient(act):
    r = np.random.default_rng(1)
    x, dy = r.normal(size=(3, 4)), r.normal(size=(3, 4))
    w_gu, w2 = r.normal(size=(10, 4)), r.normal(size=(4, 5))

    def L(x_, wg_, w2_):
        return float((B.ffn_forward(act, x_, wg_, w2_)[0] * dy).sum())

    _, a, u, s = B.ffn_forward(act, x, w_gu, w2)
    dx, dwg, dw2 = B.ffn_backward(act, dy, x, w_gu, w2, a, u, s)
    for arr, grad, fun in ((x, dx, lambda t: L(t, w_gu, w2)),
                           (w_gu, dwg, lambda t: L(x, t, w2)),
                           (w2, dw2, lambda t: L(x, w_gu, t))):
        v = r.normal(size=arr.shape)
        assert abs(_diff(fun, arr, v) - (grad * v).sum()) < 1e-7


def test_activation_values():
    assert B.activation("silu", np.array(0.0))[0] == 0.0
    np.testing.assert_allclose(B.activation("silu", np.array([1.0]))[0],
                               1 / (1 + np.exp(-1.0)), rtol=1e-15)
    # tanh GELU: 0.8411919906 at 1 (0.5 (1 + tanh(0.8411...)))
    z = np.sqrt(2 / np.pi) * 1.044715
    np.testing.assert_allclose(B.activation("gelu_tanh", np.array([1.0]))[0],
                               0.5 * (1 + np.tanh(z)), rtol=1e-15)
    for act in ("silu", "gelu_tanh"):
        v, g = B.activation(act, np.array([-80.0, 80.0]))
        np.testing.assert_allclose(v, [0.0, 80.0], atol=1e-30)
        np.testing.assert_allclose(g, [0.0, 1.0], atol=1e-30)
