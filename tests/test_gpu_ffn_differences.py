"""moe_ffn_bwd's gradients against central differences of the float64 forward,
over blocks of rows and columns (ffn_differences.py, where the tolerance is
derived), in the weight-streaming and the tile forms."""

import pytest
import torch

import ffn_differences as FD
import test_gpu_ffn as G

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("act", G.ACTS)
@pytest.mark.parametrize("T,d,f", [(40, 64, 96), (9, 136, 72), (65, 72, 264),
                                   (200, 136, 264), (700, 72, 104)])
def test_ffn_gradients_against_differences(T, d, f, act):
    g = G.Guarded()
    D = G._data(T, d, f, seed=T)
    _, ab, s = G._run(act, D, T, d, f, False, g)
    grads = G._bwd(act, D, T, d, f, False, g, ab, s)
    N = {k: G.h64(v) for k, v in D.items()}
    off, where = FD.worst(act, N, [G.h64(t) for t in grads])
    print(f"{off:.3f} of the tolerance at {where}")
    assert off <= 1.0, where
