"""Refusals of the operators around the expert layer that need tensors on a
GPU; nothing is launched."""

import pytest
import torch

gpu = pytest.mark.gpu
BF = torch.bfloat16

if torch.cuda.is_available():
    from mixture_experts_expert_top_amd import moe


@gpu
def test_ffn_without_a_workspace_is_refused():
    T, d, f = 4, 64, 128
    z = lambda *s: torch.zeros(*s, dtype=BF, device="cuda:0")  # noqa: E731
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_ffn_fwd(0, z(T, d), z(2 * f, d), z(d, f), None, None, None,
                        z(T, d), None)
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_ffn_bwd(0, z(T, d), z(T, d), z(2 * f, d), z(d, f),
                        z(T, 2 * f), z(T, f), None, z(T, d), None, None, None)
