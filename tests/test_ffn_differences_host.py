"""The check of gradients against differences (ffn_differences.py) on the CPU
oracle: it passes the formulas' gradients as they are and rounded where the
kernels round, and fails each gradient with a piece missing."""

import numpy as np
import pytest

import ffn_differences as FD
from oracle import block_ref as B

T, D, F = 40, 64, 96


def _bf16(a):
    """Round to nearest even on 8 significant bits."""
    m, e = np.frexp(a)
    return np.ldexp(np.rint(m * 256.0) / 256.0, e)


def _case():
    rng = np.random.default_rng(5)
    n = lambda *s: _bf16(rng.normal(size=s))  # noqa: E731
    return dict(x=n(T, D), w_gu=_bf16(n(2 * F, D) * 1.2 * D ** -0.5),
                w2=_bf16(n(D, F) * F ** -0.5), dy=n(T, D))


def _grads(act, N, rnd):
    _, a, u, _ = B.ffn_forward(act, N["x"], N["w_gu"], N["w2"])
    s = rnd(B.activation(act, a)[0] * u)
    a, u = rnd(a), rnd(u)
    h, slope = B.activation(act, a)
    ds = N["dy"] @ N["w2"]
    dab = rnd(np.concatenate((ds * u * slope, ds * h), axis=1))
    return [rnd(dab @ N["w_gu"]), rnd(dab.T @ N["x"]), rnd(N["dy"].T @ s)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_the_formulas_pass(act):
    N = _case()
    assert FD.worst(act, N, _grads(act, N, lambda a: a))[0] < 1e-3
    off, where = FD.worst(act, N, _grads(act, N, _bf16))
    assert off <= 1.0, where


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("i,name", enumerate(["dx", "dw_gu", "dw2"]))
def test_a_missing_piece_fails(act, i, name):
    N = _case()
    good = _grads(act, N, _bf16)
    rows = good[i].shape[0]
    half = {"first half": slice(0, rows // 2),
            "last half": slice(rows // 2, rows),
            "last quarter": slice(rows - rows // 4, rows),
            "last eighth": slice(rows - rows // 8, rows)}
    for what, sl in half.items():
        for axis in (0, 1):
            bad = [g.copy() for g in good]
            if axis == 0:
                bad[i][sl] = 0.0
            else:
                n = bad[i].shape[1]
                bad[i][:, n - n // (2 if "half" in what else 4):] = 0.0
            off, _ = FD.worst(act, N, bad)
            assert off > 1.0, (name, what, axis)
    # four of the tokens left out of a weight gradient's sum
    if i:
        bad = list(good)
        bad[i] = _grads(act, {**N, **{k: N[k][:-4] for k in ("x", "dy")}},
                        _bf16)[i]
        assert FD.worst(act, N, bad)[0] > 1.0
