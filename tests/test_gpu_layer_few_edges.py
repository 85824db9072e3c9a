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
