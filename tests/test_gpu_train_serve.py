"""The two ends of an expert layer together, as a program uses them: a block
is trained with clipped AdamW steps (eager and captured, moments in 32 and in
8 bits), its weights are quantized, and it serves single tokens through
MoEDecode."""

import numpy as np
import pytest
import torch

from mixture_experts_expert_top_amd import inputs as I
from oracle import optim_ref as R

gpu = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
T, D, F, E, K, FS = 48, 256, 128, 6, 2, 64

if torch.cuda.is_available():
    from mixture_experts_expert_top_amd import moe
    from mixture_experts_expert_top_amd.layer import (AdamW, MoEBlock,
                                                      MoEDecode, MoEPath,
                                                      MoEPathMX, StepGraph)


def weights(seed=0):
    dev = torch.device("cuda:0")
    mk = lambda s, i, sc, dt=BF: I.make_tensor(  # noqa: E731
        s, seed=seed * 17 + i, scale=sc, dtype=dt, device=dev)
    return dict(gamma=1 + mk((D,), 0, 0.1, F32), beta=mk((D,), 1, 0.1, F32),
                w_gu=mk((E, 2 * F, D), 2, 0.06), w2=mk((E, D, F), 3, 0.06),
                w_g=mk((E, D), 4, D ** -0.5), bias=mk((E,), 5, 0.1, F32),
                sw_gu=mk((2 * FS, D), 6, 0.06), sw2=mk((D, FS), 7, 0.06))


class Training:
    def __init__(self, path, moments, **kw):
        dev = torch.device("cuda:0")
        self.w = weights()
        self.block = MoEBlock(path, norm=moe.MOE_NORM_LAYER, f_shared=FS)
        self.x = I.make_tensor((T, D), seed=70, device=dev)
        self.dy = I.make_tensor((T, D), seed=71, device=dev)
        self.opt = AdamW(self.block.gradients(**self.w), lr=2e-3,
                         moments=moments, max_norm=1.0, **kw)

    def backward(self):
        w = self.w
        self.block.forward(self.x, **w)
        self.block.backward(self.dy, w["gamma"], w["w_gu"], w["w2"],
                            w["sw_gu"], w["sw2"])

    def step(self):
        self.backward()
        self.opt.step()


def _path(mx):
    dev = torch.device("cuda:0")
    return (MoEPathMX if mx else MoEPath)(T, D, F, E, K, device=dev)


@gpu
@pytest.mark.parametrize("moments", [0, 1], ids=["fp32", "fp8"])
@pytest.mark.parametrize("master", [True, False])
def test_step_on_a_blocks_gradients(moments, master):
    """The norm and the new weights are those of the gradients that the
    block's backward left."""
    t = Training(_path(False), moments, master=master)
    t.backward()
    rows = t.opt.rows
    assert len(rows) == 8
    g = [r["g"].double().cpu().numpy().reshape(-1) for r in rows]
    p = [(r.get("master", r["p"])).double().cpu().numpy().reshape(-1)
         for r in rows]
    t.opt.step()
    norm = R.grad_norm(g)
    assert abs(float(t.opt.norm.double()) - norm) <= 1e-7 * norm
    c = R.clip_factor(norm, 1.0)
    assert c < 1.0
    lr = float(t.opt.lr.double())
    for r, gi, pi in zip(rows, g, p):
        m, v = R.moments(np.zeros_like(gi), np.zeros_like(gi), gi * c, 0.9,
                         0.95)
        wd = r["weight_decay"]
        want = R.parameter(pi, m, np.sqrt(v), 1, lr, 0.9, 0.95, 1e-8, wd)
        got = r.get("master", r["p"]).double().cpu().numpy().reshape(-1)
        half = 2.0 ** -8 if r.get("master", r["p"]).dtype == BF else 2.0 ** -24
        # the update itself to 60 roundings, then p's own
        assert np.all(np.abs(got - want) <=
                      60 * 2.0 ** -24 * lr + 2 * half * np.abs(want))
        if "master" in r:
            assert torch.equal(r["p"], r["master"].to(BF))
        moved = got != pi
        assert moved[gi != 0].mean() > (0.99 if half < 1e-3 else 0.5)


@gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("moments", [0, 1], ids=["fp32", "fp8"])
def test_captured_training_equals_eager(mx, moments):
    """Forward, backward, norm and step as one graph, replayed between eager
    work, against the same steps one by one, bit for bit."""
    a, b = (Training(_path(mx), moments) for _ in range(2))
    g = StepGraph(a.step)          # two steps to warm up, none by capturing
    for _ in range(2):
        b.step()
    for i in range(4):
        dy = I.make_tensor((T, D), seed=90 + i, device="cuda:0")
        a.dy.copy_(dy)
        b.dy.copy_(dy)
        g.replay()
        b.step()
        torch.cuda.synchronize()
        assert int(a.opt.steps) == int(b.opt.steps) == 3 + i
        for x, y in zip(a.opt.rows, b.opt.rows):
            for n in x:
                if torch.is_tensor(x[n]):
                    assert torch.equal(x[n].view(torch.uint8),
                                       y[n].view(torch.uint8)), (i, n)


@gpu
def test_a_step_without_a_finite_norm_is_left_out():
    t = Training(_path(False), 0)
    t.step()
    before = [r["p"].clone() for r in t.opt.rows]
    t.backward()
    t.block.path.dw2.view(-1)[5] = float("inf")
    t.opt.step()
    assert int(t.opt.steps) == 1
    assert all(torch.equal(r["p"], b) for r, b in zip(t.opt.rows, before))
    t.step()
    assert int(t.opt.steps) == 2
    assert not torch.equal(t.opt.rows[3]["p"], before[3])


def _serve_reference(w, x, quantized):
    """The block's output for x from its formulas in float64, with the
    weights as served."""
    x = x.double()
    n = torch.nn.functional.layer_norm(x, (D,), w["gamma"].double(),
                                       w["beta"].double(), 1e-5)
    n = n.to(BF).double()
    z = n @ w["w_g"].double().t() + w["bias"].double()
    idx = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :K]
    p = torch.softmax(torch.gather(z, 1, idx), 1)
    y = torch.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(K):
            e = int(idx[t, j])
            if quantized:
                w1, w2 = (torch.exp2(s[e].double() - 127)[..., None] *
                          c[e].view(torch.float8_e4m3fn).double().view(
                              *s[e].shape, 32) for c, s in quantized)
                w1, w2 = w1.flatten(1), w2.flatten(1)
            else:
                w1, w2 = w["w_gu"][e].double(), w["w2"][e].double()
            a, u = w1[:F] @ n[t], w1[F:] @ n[t]
            y[t] += p[t, j] * (w2 @ (a * torch.sigmoid(a) * u))
    sg = n @ w["sw_gu"].double().t()
    s = sg[:, :FS] * torch.sigmoid(sg[:, :FS]) * sg[:, FS:]
    return x + y + s @ w["sw2"].double().t()


@gpu
@pytest.mark.parametrize("tokens", [1, 5, 40])
@pytest.mark.parametrize("mx", [False, True])
def test_trained_block_serves_tokens(tokens, mx):
    """Three training steps, then the block around MoEDecode on its weights
    (bf16, or quantized once), against float64 within 2e-2 of the output's
    rms (four bf16 roundings on the way: n, the experts' y, the sum with the
    dense block, the output), and against the block around MoEPath."""
    dev = torch.device("cuda:0")
    t = Training(_path(False), 0)
    for _ in range(3):
        t.step()
    w = t.w
    prec = moe.MOE_MXFP8 if mx else moe.MOE_BF16
    path = MoEDecode(tokens, D, F, E, K, prec=prec, device=dev)
    block = MoEBlock(path, norm=moe.MOE_NORM_LAYER, f_shared=FS)
    q = [MoEDecode.quantize(w[n]) for n in ("w_gu", "w2")] if mx else None
    served = {**w, "w_gu": q[0], "w2": q[1]} if mx else w
    for seed in range(3):
        x = I.make_tensor((tokens, D), seed=200 + seed, device=dev)
        y = block.forward(x, **served)
        want = _serve_reference(w, x, q)
        rms = float(want.square().mean().sqrt())
        assert float((y.double() - want).abs().max()) <= 2e-2 * rms
        if not mx:
            long = MoEPath(tokens, D, F, E, K, device=dev)
            other = MoEBlock(long, norm=moe.MOE_NORM_LAYER, f_shared=FS)
            z = other.forward(x, **w)
            assert torch.equal(path.topk_idx, long.topk_idx)
            assert float((y.double() - z.double()).abs().max()) <= 2e-2 * rms


@gpu
def test_a_captured_decode_step_follows_its_input():
    dev = torch.device("cuda:0")
    w = weights(3)
    path = MoEDecode(1, D, F, E, K, device=dev)
    block = MoEBlock(path, norm=moe.MOE_NORM_LAYER, f_shared=FS)
    x = I.make_tensor((1, D), seed=1, device=dev)
    g = StepGraph(lambda: block.forward(x, **w))
    other = MoEBlock(MoEDecode(1, D, F, E, K, device=dev),
                     norm=moe.MOE_NORM_LAYER, f_shared=FS)
    for i in range(4):
        x.copy_(I.make_tensor((1, D), seed=300 + i, device=dev))
        g.replay()
        want = other.forward(x, **w)
        torch.cuda.synchronize()
        assert torch.equal(block.y, want)


@gpu
def test_refusals():
    dev = torch.device("cuda:0")
    with pytest.raises(ValueError):
        MoEDecode(65, D, F, E, K, device=dev)
    with pytest.raises(ValueError):
        MoEDecode(1, D, F, E, E + 1, device=dev)
    w = weights()
    path = MoEDecode(2, D, F, E, K, device=dev)
    block = MoEBlock(path, norm=moe.MOE_NORM_LAYER, f_shared=FS)
    x = I.make_tensor((2, D), seed=1, device=dev)
    block.forward(x, **w)
    with pytest.raises(NotImplementedError):
        block.backward(x.clone(), w["gamma"], w["w_gu"], w["w2"], w["sw_gu"],
                       w["sw2"])
    with pytest.raises(ValueError):
        path.forward(I.make_tensor((3, D), seed=1, device=dev), w["w_gu"],
                     w["w2"], w_g=w["w_g"])
    with pytest.raises(ValueError):
        AdamW([(w["w2"].cpu(), w["w2"].cpu())])
    with pytest.raises(ValueError):
        AdamW([])


@gpu
@pytest.mark.parametrize("bad", [0.0, -1.0, float("nan"), float("inf")])
def test_adamw_refuses_a_norm_to_clip_to(bad):
    w = torch.zeros(8, dtype=BF, device="cuda:0")
    with pytest.raises(ValueError, match="max_norm"):
        AdamW([(w, torch.zeros_like(w))], max_norm=bad)


@gpu
@pytest.mark.parametrize("moments", [0, 1], ids=["fp32", "fp8"])
def test_training_goes_on_from_a_stored_state(moments):
    """Three steps, store, two more: another program that loads the weights
    and the state makes the same two, bit for bit, also by a step captured
    before it loaded them."""
    a, b = Training(_path(False), moments), Training(_path(False), moments)
    g = StepGraph(b.step)
    for _ in range(3):
        a.step()
    state = {k: v.clone() if torch.is_tensor(v) else
             [{n: t.clone() for n, t in w.items()} for w in v]
             for k, v in a.opt.state_dict().items()}
    for n, w in b.w.items():
        w.copy_(a.w[n])
    b.opt.load_state_dict(state)
    for i in range(2):
        a.step()
        if i:
            g.replay()
        else:
            b.step()
        torch.cuda.synchronize()
        assert int(a.opt.steps) == int(b.opt.steps) == 4 + i
        for x, y in zip(a.opt.rows, b.opt.rows):
            for n in x:
                if torch.is_tensor(x[n]):
                    assert torch.equal(x[n].view(torch.uint8),
                                       y[n].view(torch.uint8)), (i, n)
