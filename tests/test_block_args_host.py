"""Further argument checks of the norm and feed-forward entries that need no
GPU (fake device pointers; every call is refused before a launch)."""

import pytest
import torch

from mixture_experts_expert_top_amd import moe

L = moe.lib


@pytest.mark.parametrize("d", [9, 12, 20, 4100, 16380])
def test_norm_workspace_of_a_refused_width_is_0(d):
    """The width's own call is refused, so it has no workspace either."""
    assert L.moe_workspace_bytes(moe.MOE_ENTRY_NORM_BWD, 0, 4, 1, 1, d, 0) == 0
    assert L.moe_workspace_bytes(moe.MOE_ENTRY_NORM_BWD, 0, 4, 1, 1,
                                 d // 8 * 8, 0) > 0


def test_ffn_binding_without_a_workspace_is_a_refusal():
    """No AttributeError: the call goes on to the other checks, the last of
    them the library's, which requires a workspace."""
    T, d, f = 4, 64, 128
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_ffn_fwd(0, bf(T, d), bf(2 * f, d), bf(d, f), None, None,
                        None, bf(T, d), None)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_ffn_bwd(0, bf(T, d), bf(T, d), bf(2 * f, d), bf(d, f),
                        bf(T, 2 * f), bf(T, f), None, bf(T, d), None, None,
                        None)
