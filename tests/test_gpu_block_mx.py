"""MoEBlock around MoEPathMX (MXFP8, and MXFP4 activations) against the
MX-emulating float64 oracle and the block's own, forward and backward.

The experts are compared on the block's own bf16 n and dz (each first held to
the oracle's within its rounding): a rounding of n may move an MX code by a
whole step, which is no error of the block.  The routing is the kernel's own
(topk_idx).

Tolerance, in relative root mean square: the MX layer by itself is held to
1e-2 of its oracle (test_gpu_mx_layer.py), and the block adds at most four
roundings to bf16 in a row, each at most h = 2^-8 and of root mean square at
most h / sqrt(3), independent of it: sqrt(1e-2^2 + 4 h^2 / 3) = 1.1e-2.  The
branch's share of y and dx is what is compared, the stream taken off again;
a bf16 stream's own rounding, at most h of y (dx), is added."""

import numpy as np
import pytest
import torch

import test_gpu_block as K
from oracle import block_ref as B
from oracle import moe_mx as X

gpu = pytest.mark.gpu
H = K.H
TOL = (1e-4 + 4 * H * H / 3) ** 0.5

if torch.cuda.is_available():
    from mixture_experts_expert_top_amd import moe
    from mixture_experts_expert_top_amd.layer import MoEBlock, MoEPathMX

CASES = [
    # T, d, f, E, k, f_shared, act, norm rms, stream fp32, p, fp4 activations
    (64, 128, 128, 4, 2, 136, 0, True, False, 0.1, False),
    (300, 256, 384, 5, 2, 200, 1, False, True, 0.25, False),
    (150, 128, 256, 8, 3, 0, 0, True, True, 0.0, False),
    (300, 256, 384, 5, 2, 200, 0, True, False, 0.2, True),
]


def _rms(a):
    return float(np.sqrt(np.mean(np.square(a))))


def _router_grad(n, w_g, idx, p, dp, aux_coef):
    """d/dlogits of the renormalized top-k weights and the balancing loss."""
    T, E = n.shape[0], w_g.shape[0]
    dl = np.zeros((T, E))
    np.put_along_axis(
        dl, idx, p * (dp - (p * dp).sum(axis=1, keepdims=True)), axis=1)
    L = n @ w_g.T
    P = np.exp(L - L.max(axis=1, keepdims=True))
    P /= P.sum(axis=1, keepdims=True)
    fe = np.bincount(idx.ravel(), minlength=E) / idx.size
    return dl + aux_coef * E / T * P * (
        fe - (P * fe).sum(axis=1, keepdims=True))


@gpu
@pytest.mark.parametrize("T,d,f,E,k,fs,act,rms,f32,p,fp4", CASES)
def test_mx_block_against_oracle(T, d, f, E, k, fs, act, rms, f32, p, fp4):
    dev = torch.device("cuda:0")
    D = K._inputs(T, d, f, E, fs, K.F32 if f32 else K.BF, T + d, rms)
    path = MoEPathMX(T, d, f, E, k, device=dev, act_fp4=fp4)
    blk = MoEBlock(path, norm=moe.MOE_NORM_RMS if rms else moe.MOE_NORM_LAYER,
                   f_shared=fs, act=act, stream_fp32=f32)
    y, dx = K._step(blk, D, p)
    torch.cuda.synchronize()
    N = {n: (None if t is None else K.h64(t)) for n, t in D.items()}
    x, dy, n, dz = N["x"], N["dy"], K.h64(blk.n), K.h64(blk.dz)
    off = {}                       # error over its tolerance

    def hold(name, got, ref, tol):
        off[name] = _rms(K.h64(got) - ref) / (tol * _rms(ref))

    nref, _, _ = B.norm_forward(x, N["gamma"], N["beta"], blk.eps, rms)
    hold("n", blk.n, nref, H)
    drop_dy, keep = B.dropout(dy, None, p, 77, 5 + 3)
    hold("dz", blk.dz, drop_dy, H)

    idx = path.topk_idx.cpu().numpy().astype(np.int64)
    ch = np.take_along_axis(n @ N["w_g"].T, idx, axis=1)
    w = np.exp(ch - ch.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    fwd = X.experts_forward_mx(n, idx, w, N["w_gu"], N["w2"], fp4)
    z = fwd["y"]
    an = "gelu_tanh" if act else "silu"
    if fs:
        sy, sa, su, ss = B.ffn_forward(an, n, N["sw_gu"], N["sw2"])
        z = z + sy
    hold("z", path.y, z, TOL)
    branch, _ = B.dropout(z, None, p, 77, 5 + 3)
    off["y"] = _rms(K.h64(y) - x - branch) / (
        TOL * _rms(branch) + (0 if f32 else H) * _rms(x + branch))

    bwd = X.moe_backward_mx(fwd, dz, N["w_gu"], N["w2"])
    dl = _router_grad(n, N["w_g"], idx, w, bwd["dp"], path.aux_coef)
    dn = bwd["dx"] + dl @ N["w_g"]
    hold("dw_gu", path.dw_gu, bwd["dw_gu"], TOL)
    hold("dw2", path.dw2, bwd["dw2"], TOL)
    hold("dw_g", path.dw_g, dl.T @ n, TOL)
    if fs:
        sdx, dsw_gu, dsw2 = B.ffn_backward(an, dz, n, N["sw_gu"], N["sw2"],
                                           sa, su, ss)
        dn = dn + sdx
        hold("dsw_gu", blk.dsw_gu, dsw_gu, TOL)
        hold("dsw2", blk.dsw2, dsw2, TOL)
    hold("dn", path.dx, dn, TOL)
    dxb, dgamma, dbeta = B.norm_backward(dn, x, N["gamma"], blk.eps, rms)
    off["dx"] = _rms(K.h64(dx) - dy - dxb) / (
        TOL * _rms(dxb) + (0 if f32 else H) * _rms(dy + dxb))
    hold("dgamma", blk.dgamma, dgamma, TOL)
    if not rms:
        hold("dbeta", blk.dbeta, dbeta, TOL)
    print({a: f"{v:.2f}" for a, v in off.items()})
    assert all(v <= 1.0 for v in off.values()), off
