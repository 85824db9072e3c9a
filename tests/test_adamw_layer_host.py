"""layer.AdamW and the gradients methods where no kernel has to run: tables
are replaced by the rows that they would be made of."""

import io

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


def _optimizer(moments, master=True, shapes=((6, 8), (300,)), **kw):
    ws = [torch.randn(*s).to(BF) for s in shapes] + [torch.randn(5)]
    return layer.AdamW([(w, torch.zeros_like(w)) for w in ws],
                       moments=moments, master=master, **kw)


@pytest.mark.parametrize("moments", [moe.MOE_MOMENTS_FP32,
                                     moe.MOE_MOMENTS_FP8])
@pytest.mark.parametrize("master", [True, False])
def test_state_through_a_file(tables, moments, master):
    a, b = (_optimizer(moments, master, lr=lr) for lr in (1e-3, 5e-2))
    a.steps.fill_(12)
    for r in a.rows:
        for n in ("m", "v"):
            r[n].view(torch.uint8).random_(0, 100)
            if moments == moe.MOE_MOMENTS_FP8:
                r[n + "_scale"].uniform_()
    f = io.BytesIO()
    torch.save(a.state_dict(), f)
    f.seek(0)
    at = [t.data_ptr() for r in b.rows for t in r.values()
          if torch.is_tensor(t)]
    b.load_state_dict(torch.load(f, weights_only=True))
    assert at == [t.data_ptr() for r in b.rows for t in r.values()
                  if torch.is_tensor(t)]
    assert int(b.steps) == 12 and torch.equal(b.lr, a.lr)
    kept = ("m", "v") + ("m_scale", "v_scale") * moments
    for x, y in zip(a.rows, b.rows):
        assert ("master" in y) == (master and y["p"].dtype == BF)
        for n in kept + ("master",) * ("master" in y):
            assert torch.equal(x[n].view(torch.uint8), y[n].view(torch.uint8))
        assert not torch.equal(x["p"], y["p"])      # weights are their owner's


def test_state_of_something_else_is_refused(tables):
    """Before anything is copied."""
    a = _optimizer(moe.MOE_MOMENTS_FP8)
    before = [r["m"].clone() for r in a.rows]
    for b in (_optimizer(moe.MOE_MOMENTS_FP32),
              _optimizer(moe.MOE_MOMENTS_FP8, master=False),
              _optimizer(moe.MOE_MOMENTS_FP8, shapes=((6, 8),)),
              _optimizer(moe.MOE_MOMENTS_FP8, shapes=((6, 8), (301,))),
              _optimizer(moe.MOE_MOMENTS_FP8, shapes=((8, 6), (300,)))):
        for r in b.rows:
            r["m"].view(torch.uint8).fill_(1)
        b.steps.fill_(5)
        with pytest.raises(ValueError):
            a.load_state_dict(b.state_dict())
        assert int(a.steps) == 0
        assert all(torch.equal(r["m"].view(torch.uint8), m.view(torch.uint8))
                   for r, m in zip(a.rows, before))


@pytest.mark.parametrize("kw,word", [
    (dict(moments=2), "moments"), (dict(moments=None), "moments"),
    (dict(betas=(1.0, 0.95)), "betas"), (dict(betas=(0.9, -0.1)), "betas"),
    (dict(betas=(0.9, float("nan"))), "betas"), (dict(eps=0.0), "eps"),
    (dict(eps=2.0), "eps"), (dict(eps=1e-13, moments=1), "eps"),
    (dict(eps=float("nan")), "eps")])
def test_adamw_refuses_when_it_is_made(tables, kw, word):
    """What every step of it would be refused for, after the step had been
    counted."""
    w = torch.zeros(8, dtype=BF)
    with pytest.raises(ValueError, match=word):
        layer.AdamW([(w, torch.zeros_like(w))], **kw)


def test_adamw_takes_the_ends_of_its_ranges(tables):
    w = torch.zeros(8, dtype=BF)
    for kw in (dict(betas=(0.0, 0.0), eps=1.0), dict(eps=1e-20),
               dict(eps=1e-12, moments=1)):
        layer.AdamW([(w, torch.zeros_like(w))], **kw)
