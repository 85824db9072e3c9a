"""moe_layer_fwd where test_gpu_layer_few.py's sizes do not reach, held to its
bounds."""

import pytest
import torch

import test_gpu_layer_few as L

gpu = pytest.mark.gpu


def to_one_expert_each(c, hot=3):
    """Logits that give token t the expert t % hot."""
    c.logits = torch.full((c.T, c.E), -9.0, device="cuda:0")
    t = torch.arange(c.T, device="cuda:0")
    c.logits[t, t % hot] = 2.0
    return t


@gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 2, 4, 7, 20, 64])
@pytest.mark.parametrize("f", [128, 384, 640, 896])
def test_a_nan_scale_stays_in_its_row(T, mx, f):
    """A NaN in the first blocks of a row of w2 (MXFP8: a NaN scale) is no
    part of the row before it, wherever f ends in a load."""
    c = L.Case(T, 256, f, 4, 1, mx=mx, seed=8)
    t = to_one_expert_each(c)
    want = c.run().clone()
    rows = (1, 8, 16, 30, 128, 255)
    for i, r in enumerate(rows):
        if mx:
            c.s[1][0, r, i % 4] = 255
        else:
            c.w[1][0, r, 32 * (i % 4)] = float("nan")
    got = c.run()
    bad = torch.zeros(T, 256, dtype=torch.bool, device="cuda:0")
    for r in rows:
        bad[t % 3 == 0, r] = True
    assert torch.equal(got[~bad], want[~bad])
    assert not torch.isfinite(got[bad]).any()


@gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,first", [(1, 0), (1, 1), (1, 3), (4, 0), (7, 0),
                                     (20, 0), (64, 0)])
def test_values_of_s_past_the_end_of_bf16(T, first, mx):
    """One value of S a token, times rows of w2 of +-2^-100 and 0: an infinite
    one gives infinities (and NaN at 0), as a single product would; one between
    bf16's largest value and fp32's gives 2^28 (1 - 2^-10); S itself is off by
    12 u and held to 2^-16, y rounds to 2^-8."""
    dev = torch.device("cuda:0")
    c = L.Case(T, 128, 128, 2, 1, mx=mx, seed=1)
    c.logits = torch.tensor([[1.0, -1.0]], device=dev).repeat(T, 1)
    a = [2.0 ** 70, 2.0 ** 64 * (1 + 2.0 ** -5), 2.0, 2.0 ** 64]
    u = [2.0 ** 70, 2.0 ** 64 * (1 - 2.0 ** -5), 3.0, -2.0 ** 80]
    kind = [(t + first) % 4 for t in range(T)]
    c.x.zero_()
    for t, i in enumerate(kind):
        c.x[t, 0], c.x[t, 1] = a[i], u[i]
    for w in c.w:
        w.zero_()
    one, minus = (0x38, 0xB8) if mx else (1.0, -1.0)
    c.w[0][0, 0, 0] = one               # gate reads x[0], up x[1]
    c.w[0][0, 128, 1] = one
    if mx:
        c.s[0].fill_(127)
        c.s[1].fill_(27)
    else:
        one, minus = 2.0 ** -100, -2.0 ** -100
    c.w[1][0, ::2, 0], c.w[1][0, 1::2, 0] = one, minus
    c.w[1][0, 7, 0] = 0
    y = c.run().double()
    sign = torch.ones(128, dtype=torch.float64, device=dev)
    sign[1::2] = -1
    sign[7] = 0
    live = sign != 0
    for t, i in enumerate(kind):
        if i in (0, 3):
            want = sign * (1 if i == 0 else -1) * float("inf")
            assert torch.equal(y[t][live], want[live]), i
            assert torch.isnan(y[t, 7])
        else:
            S = (torch.tensor(a[i], dtype=torch.float64).sigmoid() * a[i] *
                 u[i])
            want = sign * float(S) * 2.0 ** -100
            tol = (2.0 ** -8 + 2.0 ** -15) * want.abs()
            assert ((y[t] - want).abs() <= tol).all(), i
