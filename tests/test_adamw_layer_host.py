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
