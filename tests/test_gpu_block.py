"""The residual block around the expert layer (MoEBlock): norm, routed
experts, dense feed-forward block, dropout and residual sum run together,
forward and backward, against the float64 oracles chained the same way.

Tolerances: every intermediate that the block keeps in bf16 (n, the experts'
output, the feed-forward block's sum, dz, the experts' dx, dn, and inside
each part its AB, S and [dA dU]) carries a relative rounding of at most h =
2^-8, independent between elements.  y's branch passes 4 roundings (n, the
part's AB/S, the part's output, the sum), its gradients at most 7 in a row
(n, AB, S or dAB, dz, dx, dn, the result), each amplified by at most the
norm's and the activations' unit-size slopes; their mean square is bounded by
sqrt(7) h of the output's own, and 4 h is allowed.  The oracle routes with the
kernel's own choices (topk_idx), since a rounding of n may reorder two close
scores.
"""

import numpy as np
import pytest
import torch

from mixture_experts_expert_top_amd import inputs as I
from oracle import block_ref as B

gpu = pytest.mark.gpu
H = 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32

if torch.cuda.is_available():
    from mixture_experts_expert_top_amd import moe
    from mixture_experts_expert_top_amd.layer import (MoEBlock, MoEPath,
                                                      MoEPathMX, StageTimers,
                                                      StepGraph)


def h64(t):
    return t.double().cpu().numpy()


def _inputs(T, d, f, E, fs, xt, seed, rms):
    dev = torch.device("cuda:0")
    mk = lambda shape, k, s=1.0, dt=BF: I.make_tensor(  # noqa: E731
        shape, seed=seed * 13 + k, scale=s, dtype=dt, device=dev)
    return dict(
        x=mk((T, d), 0, dt=xt), gamma=1 + mk((d,), 1, 0.1, F32),
        beta=None if rms else mk((d,), 2, 0.1, F32),
        w_g=mk((E, d), 3, d ** -0.5), w_gu=mk((E, 2 * f, d), 4, d ** -0.5),
        w2=mk((E, d, f), 5, f ** -0.5), dy=mk((T, d), 6, dt=xt),
        sw_gu=mk((2 * fs, d), 7, d ** -0.5) if fs else None,
        sw2=mk((d, fs), 8, fs ** -0.5) if fs else None,
        rng=torch.tensor([77, 5], dtype=torch.int64, device=dev))


def _step(blk, D, p, delta=3):
    y = blk.forward(D["x"], D["gamma"], D["w_gu"], D["w2"], beta=D["beta"],
                    w_g=D["w_g"], sw_gu=D["sw_gu"], sw2=D["sw2"], p=p,
                    rng=D["rng"] if p else None, delta=delta)
    dx = blk.backward(D["dy"], D["gamma"], D["w_gu"], D["w2"],
                      sw_gu=D["sw_gu"], sw2=D["sw2"])
    return y, dx


def _reference(D, idx, k, act, rms, p, eps, aux_coef, delta=3):
    """The block in float64, one expert and token at a time."""
    N = {n: (None if t is None else h64(t)) for n, t in D.items()}
    X, DY = N["x"], N["dy"]
    T, d = X.shape
    E = N["w_g"].shape[0]
    n, _, _ = B.norm_forward(X, N["gamma"], N["beta"], eps, rms)
    L = n @ N["w_g"].T
    ch = np.take_along_axis(L, idx, axis=1)
    w = np.exp(ch - ch.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    z = np.zeros((T, d))
    keep_e = []
    for e in range(E):
        t, j = np.nonzero(idx == e)
        y, a, u, s = B.ffn_forward("silu", n[t], N["w_gu"][e], N["w2"][e])
        z[t] += w[t, j][:, None] * y
        keep_e.append((t, j, y, a, u, s))
    shared = N["sw_gu"] is not None
    if shared:
        y, sa, su, ss = B.ffn_forward(act, n, N["sw_gu"], N["sw2"])
        z += y
    drop, keep = B.dropout(z, None, p, 77, 5 + delta)
    out = {"y": X + drop}
    scale = 65536.0 / (65536 - np.floor(p * 65536 + 0.5))
    dz = np.where(keep, DY, 0.0) * scale
    dn = np.zeros((T, d))
    dp = np.zeros(idx.shape)
    dwg, dw2 = np.zeros_like(N["w_gu"]), np.zeros_like(N["w2"])
    for e, (t, j, y, a, u, s) in enumerate(keep_e):
        dp[t, j] = (dz[t] * y).sum(axis=1)
        g = w[t, j][:, None] * dz[t]
        dxe, dwg[e], dw2[e] = B.ffn_backward("silu", g, n[t], N["w_gu"][e],
                                             N["w2"][e], a, u, s)
        dn[t] += dxe
    dl = np.zeros((T, E))
    sm = (w * dp).sum(axis=1, keepdims=True)
    np.put_along_axis(dl, idx, w * (dp - sm), axis=1)
    P = np.exp(L - L.max(axis=1, keepdims=True))
    P /= P.sum(axis=1, keepdims=True)
    fe = np.bincount(idx.ravel(), minlength=E) / idx.size
    dl += aux_coef * E / T * P * (fe - (P * fe).sum(axis=1, keepdims=True))
    dn += dl @ N["w_g"]
    out.update(dw_gu=dwg, dw2=dw2, dw_g=dl.T @ n)
    if shared:
        dxs, out["dsw_gu"], out["dsw2"] = B.ffn_backward(
            act, dz, n, N["sw_gu"], N["sw2"], sa, su, ss)
        dn += dxs
    out["dx"], out["dgamma"], dbeta = B.norm_backward(
        dn, X, N["gamma"], eps, rms, DY)
    if not rms:
        out["dbeta"] = dbeta
    return out


def _rms_err(got, ref):
    return float(np.sqrt(np.mean((h64(got) - ref) ** 2) / np.mean(ref ** 2)))


CASES = [
    # T, d, f, E, k, f_shared, act, norm rms, stream fp32, p
    (64, 64, 96, 4, 2, 128, 0, True, False, 0.1),
    (200, 136, 72, 5, 2, 200, 1, False, True, 0.25),
    (33, 128, 64, 8, 3, 0, 0, True, True, 0.0),
    (1, 64, 64, 4, 1, 64, 0, False, False, 0.0),
]


@gpu
@pytest.mark.parametrize("T,d,f,E,k,fs,act,rms,f32,p", CASES)
def test_block_against_oracle(T, d, f, E, k, fs, act, rms, f32, p):
    dev = torch.device("cuda:0")
    D = _inputs(T, d, f, E, fs, F32 if f32 else BF, T + d, rms)
    path = MoEPath(T, d, f, E, k, device=dev)
    blk = MoEBlock(path, norm=moe.MOE_NORM_RMS if rms else moe.MOE_NORM_LAYER,
                   f_shared=fs, act=act, stream_fp32=f32)
    y, dx = _step(blk, D, p)
    torch.cuda.synchronize()
    assert y.dtype == dx.dtype == D["x"].dtype
    ref = _reference(D, path.topk_idx.cpu().numpy().astype(np.int64), k,
                     "gelu_tanh" if act else "silu", rms, p, blk.eps,
                     path.aux_coef)
    got = dict(y=y, dx=dx, dgamma=blk.dgamma, dw_gu=path.dw_gu,
               dw2=path.dw2, dw_g=path.dw_g)
    if not rms:
        got["dbeta"] = blk.dbeta
    if fs:
        got.update(dsw_gu=blk.dsw_gu, dsw2=blk.dsw2)
    # one token routed to one expert leaves the router nothing to learn: its
    # gradient is a difference of equal numbers
    if k == 1:
        got.pop("dw_g")
    errs = {n: _rms_err(t, ref[n]) / H for n, t in got.items()}
    print({n: f"{e:.2f} h" for n, e in errs.items()})
    assert all(e <= 4.0 for e in errs.values()), errs


@gpu
@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
def test_block_graph_timers_and_rng(mx):
    """A captured step equals the eager one at the same generator state, and
    advances with it; timing the stages changes nothing."""
    dev = torch.device("cuda:0")
    T, d, f, E, k, fs = 150, 128, 128, 4, 2, 136
    D = _inputs(T, d, f, E, fs, BF, 4, True)
    path = (MoEPathMX if mx else MoEPath)(T, d, f, E, k, device=dev)
    blk = MoEBlock(path, f_shared=fs)
    names = ["y", "dx", "dgamma", "dsw_gu", "dsw2"]

    def snap():
        torch.cuda.synchronize()
        return [getattr(blk, n).clone() for n in names] + [
            path.dw_gu.clone(), path.dw2.clone()]

    def step():
        _step(blk, D, 0.2)

    refs = []
    for i in range(3):
        D["rng"].copy_(torch.tensor([77, 5 + i]))
        step()
        refs.append(snap())
    assert not torch.equal(refs[0][0], refs[1][0])
    D["rng"].copy_(torch.tensor([77, 5]))
    timers = StageTimers()
    blk.forward(D["x"], D["gamma"], D["w_gu"], D["w2"], w_g=D["w_g"],
                sw_gu=D["sw_gu"], sw2=D["sw2"], p=0.2, rng=D["rng"], delta=3,
                timers=timers)
    blk.backward(D["dy"], D["gamma"], D["w_gu"], D["w2"], sw_gu=D["sw_gu"],
                 sw2=D["sw2"], timers=timers)
    got = snap()
    assert all(torch.equal(a, b) for a, b in zip(got, refs[0]))
    assert {"norm_fwd", "ffn_fwd", "dropout_fwd", "dropout_bwd", "ffn_bwd",
            "norm_bwd"} <= set(timers.mean_ms())
    g = StepGraph(step)
    other = torch.randn(256, 256, device=dev)
    for i in range(3):
        D["rng"].copy_(torch.tensor([77, 5 + i]))
        for n in names:
            getattr(blk, n).zero_()
        other = other @ other.t() / 256.0
        torch.cuda.synchronize()
        g.replay()
        got = snap()
        assert all(torch.equal(a, b) for a, b in zip(got, refs[i])), i


@gpu
def test_block_refusals():
    dev = torch.device("cuda:0")
    path = MoEPath(16, 64, 64, 4, 2, device=dev)
    D = _inputs(16, 64, 64, 4, 64, BF, 1, True)
    blk = MoEBlock(path, f_shared=64)
    with pytest.raises(ValueError, match="rng"):
        blk.forward(D["x"], D["gamma"], D["w_gu"], D["w2"], w_g=D["w_g"],
                    sw_gu=D["sw_gu"], sw2=D["sw2"], p=0.1)
    with pytest.raises(ValueError, match="sw_gu"):
        blk.forward(D["x"], D["gamma"], D["w_gu"], D["w2"], w_g=D["w_g"])
    with pytest.raises(ValueError, match="bf16"):
        MoEBlock(MoEPath(16, 64, 64, 4, 2, device=dev, y_fp32=True))


@gpu
def test_tensors_on_different_devices_are_refused():
    dev = torch.device("cuda:0")
    x = torch.zeros(4, 64, dtype=BF, device=dev)
    y, gamma = torch.empty_like(x), torch.ones(64)
    with pytest.raises(ValueError, match="different devices"):
        moe.moe_norm_fwd(0, x, gamma, None, 1e-5, y)
    with pytest.raises(ValueError, match="different devices"):
        moe.moe_dropout(x, None, 0.1, torch.zeros(2, dtype=torch.int64), 0, y)
    # a view that starts off a 16-byte boundary is refused by the library
    flat = torch.zeros(4 * 64 + 8, dtype=BF, device=dev)
    with pytest.raises(moe.MoeError, match="aligned"):
        moe.moe_norm_fwd(0, flat[4:4 + 256].view(4, 64), gamma.to(dev), None,
                         1e-5, y)


@gpu
def test_calls_at_the_same_time_on_two_streams():
    """Two steps of different data, each with its own buffers and workspaces,
    issued in turn on two streams: the bits of each run alone."""
    dev = torch.device("cuda:0")
    T, d, f = 200, 264, 1032
    sets = []
    for seed in (1, 2):
        mk = lambda shape, k, s=1.0, dt=BF: I.make_tensor(  # noqa: E731
            shape, seed=seed * 17 + k, scale=s, dtype=dt, device=dev)
        new = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device=dev)  # noqa
        ws = lambda e: new(max(16, moe.moe_workspace_bytes(  # noqa: E731
            e, 0, T, 1, 1, d, f)), dt=torch.uint8)
        sets.append(dict(
            x=mk((T, d), 0), gamma=mk((d,), 1, dt=F32), dy=mk((T, d), 2),
            wg=mk((2 * f, d), 3, d ** -0.5), w2=mk((d, f), 4, f ** -0.5),
            n=new(T, d), rstd=new(T, dt=F32), ab=new(T, 2 * f), s=new(T, f),
            y=new(T, d), dn=new(T, d), dwg=new(2 * f, d), dw2=new(d, f),
            dx=new(T, d), dg=new(d, dt=F32), wf=ws(moe.MOE_ENTRY_FFN_FWD),
            wb=ws(moe.MOE_ENTRY_FFN_BWD), wn=ws(moe.MOE_ENTRY_NORM_BWD),
            rng=torch.tensor([seed, 3], dtype=torch.int64, device=dev)))

    def step(b, st=None):
        moe.moe_norm_fwd(1, b["x"], b["gamma"], None, 1e-5, b["n"], None,
                         b["rstd"], stream=st)
        moe.moe_ffn_fwd(0, b["n"], b["wg"], b["w2"], None, b["ab"], b["s"],
                        b["y"], b["wf"], stream=st)
        moe.moe_dropout(b["y"], b["x"], 0.2, b["rng"], 1, b["y"], stream=st)
        moe.moe_ffn_bwd(0, b["dy"], b["n"], b["wg"], b["w2"], b["ab"],
                        b["s"], None, b["dn"], b["dwg"], b["dw2"], b["wb"],
                        stream=st)
        moe.moe_norm_bwd(1, b["dn"], b["x"], b["gamma"], None, b["rstd"],
                         b["dy"], b["dx"], b["dg"], None, b["wn"], stream=st)

    outs = ["y", "dn", "dwg", "dw2", "dx", "dg"]
    for b in sets:
        step(b)
    torch.cuda.synchronize()
    refs = [[b[n].clone() for n in outs] for b in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, st in zip(sets, streams):
            step(b, st)
    torch.cuda.synchronize()
    for b, ref in zip(sets, refs):
        assert all(torch.equal(b[n], r) for n, r in zip(outs, ref))


@gpu
def test_block_on_its_own_output():
    """x may be the block's last y: the forward is that of a copy; the
    backward, whose x is gone, is refused, as is one without a forward, and
    an x in the path's own output."""
    dev = torch.device("cuda:0")
    path = MoEPath(33, 64, 64, 4, 2, device=dev)
    D = _inputs(33, 64, 64, 4, 64, BF, 1, True)
    blk = MoEBlock(path, f_shared=64)

    def fwd(x):
        return blk.forward(x, D["gamma"], D["w_gu"], D["w2"], w_g=D["w_g"],
                           sw_gu=D["sw_gu"], sw2=D["sw2"], p=0.25,
                           rng=D["rng"])

    def bwd():
        return blk.backward(D["dy"], D["gamma"], D["w_gu"], D["w2"],
                            sw_gu=D["sw_gu"], sw2=D["sw2"])
    with pytest.raises(ValueError, match="forward"):
        bwd()
    once = fwd(D["x"]).clone()
    twice = fwd(once).clone()
    bwd()
    assert torch.equal(fwd(D["x"]), once)
    assert torch.equal(fwd(blk.y), twice)
    with pytest.raises(ValueError, match="this block's y"):
        bwd()
    with pytest.raises(ValueError, match="path's y"):
        fwd(path.y)
    fwd(D["x"])
    bwd()
