"""layer.AdamW and the gradients methods where no kernel has to run: tables
are replaced by the rows that they would be made of."""

import pytest
import torch

from mixture_experts_expert_top_amd import layer, moe

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def tables(monkeypatch):
    monkeypatch.setattr(moe, "adamw_table", lambda rows: rows)
    monkeypatch.setattr(moe, "grad_table", lambda grads: grads)


def test_copies_of_weights_that_require_gradients_hold_no_graph(tables):
    """The fp32 copy is data: no node of the weight's autograd graph lives as
    long as the optimizer does."""
    w = torch.nn.Parameter(torch.randn(6, 8).to(BF))
    opt = layer.AdamW([(w, torch.zeros_like(w))])
    row = opt.rows[0]
    assert row["master"].dtype == F32
    assert torch.equal(row["master"], w.detach().float())
    for n in ("master", "m", "v"):
        assert row[n].grad_fn is None and not row[n].requires_grad, n


@pytest.mark.parametrize("norm,f_shared,but,word", [
    (moe.MOE_NORM_LAYER, 16, "sw_gu", "sw_gu"),
    (moe.MOE_NORM_LAYER, 16, "sw2", "sw2"),
    (moe.MOE_NORM_RMS, 16, None, "beta"), (moe.MOE_NORM_RMS, 0, None, "beta")])
def test_a_blocks_gradients_go_with_its_weights(norm, f_shared, but, word):
    """Weights that the block has no gradient for, and gradients without their
    weights, are refused as forward does it."""
    path = layer.MoEPath(4, 16, 8, 2, 1, device="cpu")
    block = layer.MoEBlock(path, norm=norm, f_shared=f_shared)
    w = dict(gamma=torch.zeros(16), w_gu=torch.zeros(2, 16, 16, dtype=BF),
             w2=torch.zeros(2, 16, 8, dtype=BF), beta=torch.zeros(16),
             sw_gu=torch.zeros(32, 16, dtype=BF),
             sw2=torch.zeros(16, 16, dtype=BF))
    if but:
        w[but] = None
    with pytest.raises(ValueError, match=word):
        block.gradients(**w)
    w = {n: t for n, t in w.items() if n not in ("beta", "sw_gu", "sw2")}
    if not f_shared:
        assert len(block.gradients(**w)) == 3
