"""Parity of the dense feed-forward block's kernel instances that the sizes of
test_gpu_ffn.py do not take (test_ffn_forms_host.py holds that together they
take all): the step, and each gradient alone, in a launch of its own.  Bounds
as derived there."""

import pytest
import torch

import test_gpu_ffn as G
from ffn_form_sizes import SIZES

gpu = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_expert_top_amd import moe


@gpu
@pytest.mark.parametrize("act", G.ACTS)
@pytest.mark.parametrize("T,d,f", SIZES)
def test_ffn_form(T, d, f, act):
    if T * d * f > 10 ** 9:       # references on the GPU, mean-square bounds
        G.test_ffn_large_products(T, d, f, act)
        return
    g = G.Guarded()
    D = G._data(T, d, f, seed=T + f)
    y, ab, s = G._run(act, D, T, d, f, True, g)
    step = G._bwd(act, D, T, d, f, True, g, ab, s)
    alone = (g.new(T, d), g.new(2 * f, d), g.new(d, f))
    for i in range(3):
        o = [t if j == i else None for j, t in enumerate(alone)]
        moe.moe_ffn_bwd(G._act(act), D["dy"], D["x"], D["w_gu"], D["w2"], ab,
                        s, D["dx_add"] if i == 0 else None, *o,
                        G._ws(moe.MOE_ENTRY_FFN_BWD, T, d, f, g))
    torch.cuda.synchronize()
    g.check()
    N = {k: G.h64(v) for k, v in D.items()}
    G._check_fwd(act, N, True, y, ab, s, d, f)
    for got in (step, alone):
        G._check_bwd(act, N, True, ab, s, *got, T, d, f)
