"""GPU parity of moe_ffn_fwd / moe_ffn_bwd (through the C-ABI) against the
float64 oracle.

Element by element (u = 2^-24, h = 2^-8 half a bf16 step, all magnitudes from
the float64 values): a sum of n fp32 products is off by at most
2 n u sum|a||b| in any order; act and its slope are off by at most 2^-15
relative and 2^-16 absolute (hardware exponential and reciprocal, the
exponential's argument scaled by 4 u |z|) and act's slope is at most 1.13, so
  * AB: 2 d u |x||w_gu|^T + h |AB|;
  * S, held in bf16 for the second product:
    eS = 1.13 |U| eA + |act| eU + 2^-15 |S| + h |S|;
  * y: sum eS |w2| + 2 f u sum |S||w2| + h |y| + u |y_add|.
The backward is compared on the kernel's own saved (bf16) AB and S:
  * eDS = 2 d u |dy||w2|, [dA dU] = eDS (1.13 |U|, |act|) + 2^-15 |[dA dU]|
    + 2^-16 |dS U| (the slope's absolute error) + h |[dA dU]|;
  * dx: sum eDAB |w_gu| + 4 f u sum |DAB||w_gu| + h |dx| + u |dx_add|;
  * dw_gu: sum_t eDAB |x| + 2 T u sum |DAB||x| + h |dw_gu|;
  * dw2: 2 T u sum |dy||S| + h |dw2|.
Those add every rounding at its worst, so the outputs that pass through a
rounded intermediate are also held in the mean square: independent roundings
of relative size <= h in the terms and in the result give at most
sqrt(2) h of the sum's own mean square; 1.6 h is allowed.
"""

import numpy as np
import pytest
import torch

from mixture_experts_expert_top_amd import inputs as I
from oracle import block_ref as B

gpu = pytest.mark.gpu
U = 2.0 ** -24
H = 2.0 ** -8
BF = torch.bfloat16
ACTS = ["silu", "gelu_tanh"]

if torch.cuda.is_available():
    from mixture_experts_expert_top_amd import moe


def h64(t):
    return t.double().cpu().numpy()


def _act(name):
    return moe.MOE_ACT_SILU if name == "silu" else moe.MOE_ACT_GELU_TANH


def _data(T, d, f, seed, wscale=None):
    dev = torch.device("cuda:0")
    mk = lambda shape, k, s=1.0: I.make_tensor(  # noqa: E731
        shape, seed=seed * 11 + k, scale=s, device=dev)
    w = 1.2 / np.sqrt(d) if wscale is None else wscale
    return dict(x=mk((T, d), 0), w_gu=mk((2 * f, d), 1, w),
                w2=mk((d, f), 2, 1.0 / np.sqrt(f)), y_add=mk((T, d), 3),
                dy=mk((T, d), 4), dx_add=mk((T, d), 5))


class Guarded:
    """Tensors inside larger buffers filled with a pattern."""

    def __init__(self):
        self.bufs = []

    def new(self, *shape, dtype=BF):
        n, pad = int(np.prod(shape)), 256
        fill = 173 if dtype == torch.uint8 else -77.0
        b = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda:0")
        self.bufs.append((b, n, pad, fill))
        return b[pad:pad + n].view(*shape)

    def check(self):
        for b, n, pad, fill in self.bufs:
            assert (b[:pad] == fill).all() and (b[pad + n:] == fill).all()


def _ws(entry, T, d, f, g):
    return g.new(moe.moe_workspace_bytes(entry, 0, T, 1, 1, d, f),
                 dtype=torch.uint8)


def _check(name, got, ref, bound, rms=False):
    g = h64(got)
    assert np.isfinite(g).all(), name
    worst = float(np.max(np.abs(g - ref) / np.maximum(bound, 1e-300)))
    q = float(np.sqrt(np.mean((g - ref) ** 2) /
                      max(np.mean(ref ** 2), 1e-300)))
    print(f"{name}: max|err|/bound = {worst:.3f}, rms {q / H:.3f} h")
    assert worst <= 1.0, name
    if rms and ref.size >= 4096:
        assert q <= 1.6 * H, name


def _run(act, D, T, d, f, add, g, save=True):
    ab, s = (g.new(T, 2 * f), g.new(T, f)) if save else (None, None)
    y = g.new(T, d)
    moe.moe_ffn_fwd(_act(act), D["x"], D["w_gu"], D["w2"],
                    D["y_add"] if add else None, ab, s, y,
                    _ws(moe.MOE_ENTRY_FFN_FWD, T, d, f, g))
    return y, ab, s


def _bwd(act, D, T, d, f, add, g, ab, s):
    dx, dwg, dw2 = g.new(T, d), g.new(2 * f, d), g.new(d, f)
    moe.moe_ffn_bwd(_act(act), D["dy"], D["x"], D["w_gu"], D["w2"], ab, s,
                    D["dx_add"] if add else None, dx, dwg, dw2,
                    _ws(moe.MOE_ENTRY_FFN_BWD, T, d, f, g))
    return dx, dwg, dw2


def _check_fwd(act, N, add, y, ab, s, d, f):
    X, WG, W2 = N["x"], N["w_gu"], N["w2"]
    YA = N["y_add"] if add else 0.0
    ry, ra, ru, rs = B.ffn_forward(act, X, WG, W2, YA if add else None)
    rab = np.concatenate((ra, ru), axis=1)
    eab = 2 * d * U * (np.abs(X) @ np.abs(WG).T)
    if ab is not None:
        _check("ab", ab, rab, eab + H * (np.abs(rab) + eab))
    hv = np.abs(B.activation(act, ra)[0])
    es = 1.13 * np.abs(ru) * eab[:, :f] + hv * eab[:, f:] + 2.0 ** -15 * \
        np.abs(rs)
    es = es + H * (np.abs(rs) + es)
    if s is not None:
        _check("s", s, rs, es)
    W2a = np.abs(W2).T
    e = es @ W2a + 2 * f * U * (np.abs(rs) @ W2a) + U * np.abs(YA)
    _check("y", y, ry, e + H * (np.abs(ry) + e), rms=True)


def _check_bwd(act, N, add, ab, s, dx, dwg, dw2, T, d, f):
    X, WG, W2, DY = N["x"], N["w_gu"], N["w2"], N["dy"]
    DA = N["dx_add"] if add else None
    A, Uu, S = h64(ab)[:, :f], h64(ab)[:, f:], h64(s)
    rdx, rdg, rd2 = B.ffn_backward(act, DY, X, WG, W2, A, Uu, S, DA)
    hv, slope = B.activation(act, A)
    ds = DY @ W2
    eds = 2 * d * U * (np.abs(DY) @ np.abs(W2))
    dab = np.concatenate((ds * Uu * slope, ds * hv), axis=1)
    e = np.concatenate((eds * 1.13 * np.abs(Uu) +
                        2.0 ** -16 * np.abs(ds * Uu), eds * np.abs(hv)),
                       axis=1) + 2.0 ** -15 * np.abs(dab)
    e = e + H * (np.abs(dab) + e)
    WGa, Xa, Da = np.abs(WG), np.abs(X), np.abs(dab)
    b = e @ WGa + 4 * f * U * (Da @ WGa) + (U * np.abs(DA) if add else 0.0)
    _check("dx", dx, rdx, b + H * (np.abs(rdx) + b), rms=True)
    b = e.T @ Xa + 2 * T * U * (Da.T @ Xa)
    _check("dw_gu", dwg, rdg, b + H * (np.abs(rdg) + b), rms=True)
    b = 2 * T * U * (np.abs(DY).T @ np.abs(S))
    _check("dw2", dw2, rd2, b + H * (np.abs(rd2) + b))


# the weight-streaming form (T <= 64, small weights: one, two and four token blocks, each
# with its last block full and not), tiles of either width, split and whole
# reductions, widths inside and across tiles and k-steps
SIZES = [(1, 8, 8), (1, 2048, 1408), (2, 16, 24), (5, 264, 520),
         (16, 136, 40), (17, 520, 264), (31, 128, 4104), (33, 72, 104),
         (48, 4104, 136), (64, 256, 264), (64, 64, 4096), (65, 8, 8),
         (65, 40, 136), (100, 264, 72), (128, 128, 64), (130, 520, 392),
         (257, 1032, 776), (300, 2048, 1408), (1100, 520, 1416),
         (1500, 2056, 136), (4, 264, 136), (8, 4104, 4104), (12, 136, 520),
         (20, 4096, 5632), (40, 2048, 2816)]


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,d,f", SIZES)
def test_ffn_parity(T, d, f, act):
    g = Guarded()
    add = (T + d) % 3 != 0
    D = _data(T, d, f, seed=T + d + f)
    y, ab, s = _run(act, D, T, d, f, add, g)
    y2, _, _ = _run(act, D, T, d, f, add, g, save=False)
    dx, dwg, dw2 = _bwd(act, D, T, d, f, add, g, ab, s)
    torch.cuda.synchronize()
    g.check()
    assert torch.equal(y, y2)
    N = {k: h64(v) for k, v in D.items()}
    _check_fwd(act, N, add, y, ab, s, d, f)
    _check_bwd(act, N, add, ab, s, dx, dwg, dw2, T, d, f)


@gpu
@pytest.mark.parametrize("T", [3, 64, 65, 200, 1024])
def test_ffn_integers_are_exact(T):
    """Small integers: every product and sum is an integer below 2^24, so the
    first product (and with it dS and dW2's own sums) has one right answer:
    AB and dw2 to the bit."""
    d, f = 104, 72
    gen = torch.Generator().manual_seed(T)
    ri = lambda *s: torch.randint(-2, 3, s, generator=gen).to(  # noqa: E731
        "cuda:0").to(BF)
    D = dict(x=ri(T, d), w_gu=ri(2 * f, d), w2=ri(d, f), dy=ri(T, d))
    g = Guarded()
    y, ab, s = _run("silu", D, T, d, f, False, g)
    assert torch.equal(ab.double().cpu(), (
        D["x"].double() @ D["w_gu"].double().t()).to(BF).double().cpu())
    s_int = ri(T, f)
    dx, dwg, dw2 = _bwd("silu", D, T, d, f, False, g, ab, s_int)
    assert torch.equal(dw2.double().cpu(), (
        D["dy"].double().t() @ s_int.double()).to(BF).double().cpu())
    g.check()


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_ffn_saturated_gates_are_finite(act):
    """Gates far on either side: act -> 0 or the gate itself, the slope -> 0
    or 1, no NaN from an overflowing polynomial or exponential."""
    T, d, f = 2, 8, 16
    x = torch.zeros(T, d, dtype=BF, device="cuda:0")
    x[:, 0] = 1.0
    big = [1e4, 1e13, 1e19, 3e19, 1e30]
    gate = torch.tensor([s * v for v in big for s in (1, -1)] +
                        [0.0, -0.0, 30.0, -30.0, 90.0, -90.0])
    w_gu = torch.zeros(2 * f, d, dtype=BF, device="cuda:0")
    w_gu[:f, 0] = gate.to(BF).to("cuda:0")
    w_gu[f:, 0] = 2.0 ** -20
    w2 = torch.zeros(d, f, dtype=BF, device="cuda:0")
    w2[0] = 1.0
    dy = torch.zeros(T, d, dtype=BF, device="cuda:0")
    dy[:, 0] = 1.0
    g = Guarded()
    D = dict(x=x, w_gu=w_gu, w2=w2, dy=dy)
    y, ab, s = _run(act, D, T, d, f, False, g)
    dx, dwg, dw2 = _bwd(act, D, T, d, f, False, g, ab, s)
    gv = w_gu[:f, 0].double().cpu()
    want = torch.where(gv > 0, gv, torch.zeros(())) * 2.0 ** -20
    far = gv.abs() > 50
    got = s[0].double().cpu()
    assert torch.allclose(got[far], want[far], rtol=H, atol=1e-30)
    assert torch.isfinite(dwg).all() and torch.isfinite(dx).all()
    # dA = dS U slope: slope 1 or 0
    dg = dwg[:f, 0].double().cpu() / T
    assert torch.allclose(dg[far], (gv[far] > 0).double() * 2.0 ** -20,
                          rtol=2 * H, atol=1e-30)


@gpu
def test_ffn_optional_outputs_and_alias():
    T, d, f = 96, 136, 200
    D = _data(T, d, f, seed=2)
    g = Guarded()
    y, ab, s = _run("silu", D, T, d, f, True, g)
    dx, dwg, dw2 = _bwd("silu", D, T, d, f, True, g, ab, s)
    ws = _ws(moe.MOE_ENTRY_FFN_FWD, T, d, f, g)
    wsb = _ws(moe.MOE_ENTRY_FFN_BWD, T, d, f, g)
    acc = D["y_add"].clone()
    moe.moe_ffn_fwd(0, D["x"], D["w_gu"], D["w2"], acc, None, None, acc, ws)
    assert torch.equal(acc, y)
    acc = D["dx_add"].clone()
    a = (D["w_gu"], D["w2"], ab)
    moe.moe_ffn_bwd(0, D["dy"], None, *a, None, acc, acc, None, None, wsb)
    assert torch.equal(acc, dx)
    o = g.new(2 * f, d)
    moe.moe_ffn_bwd(0, D["dy"], D["x"], *a, None, None, None, o, None, wsb)
    assert torch.equal(o, dwg)
    o = g.new(d, f)
    moe.moe_ffn_bwd(0, D["dy"], None, *a, s, None, None, None, o, wsb)
    assert torch.equal(o, dw2)
    g.check()


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_ffn_gradient_against_differences(act):
    """Directional derivatives of the float64 forward against the kernel's
    gradients.  The gradients carry bf16 roundings of AB, S, [dA dU] and of
    themselves: each at most h relative on terms whose signs are random, so
    the inner product with a random direction is off by a few h of
    |grad||v| / sqrt(size) * sqrt(size); 4 h |grad||v| is allowed."""
    T, d, f = 40, 64, 96
    D = _data(T, d, f, seed=8)
    g = Guarded()
    y, ab, s = _run(act, D, T, d, f, False, g)
    grads = _bwd(act, D, T, d, f, False, g, ab, s)
    N = {k: h64(v) for k, v in D.items()}

    def loss(x, wg, w2):
        return float((B.ffn_forward(act, x, wg, w2)[0] * N["dy"]).sum())

    args = [N["x"], N["w_gu"], N["w2"]]
    rng = np.random.default_rng(0)
    for i, grad in enumerate(grads):
        v = rng.normal(size=args[i].shape)
        hi = [a + 1e-5 * v if j == i else a for j, a in enumerate(args)]
        lo = [a - 1e-5 * v if j == i else a for j, a in enumerate(args)]
        quot = (loss(*hi) - loss(*lo)) / 2e-5
        G = h64(grad)
        assert abs(quot - (G * v).sum()) <= 4 * H * np.linalg.norm(
            G) * np.linalg.norm(v)
        # and along the gradient itself, where nothing cancels
        gn = G / np.linalg.norm(G)
        hi = [a + 1e-5 * gn if j == i else a for j, a in enumerate(args)]
        lo = [a - 1e-5 * gn if j == i else a for j, a in enumerate(args)]
        quot = (loss(*hi) - loss(*lo)) / 2e-5
        assert abs(quot - np.linalg.norm(G)) <= 4 * H * np.linalg.norm(G)


@gpu
@pytest.mark.parametrize("T", [7, 150, 1500])
def test_ffn_in_a_graph_and_on_another_stream(T):
    d, f = 264, 392
    D = _data(T, d, f, seed=T)
    g = Guarded()
    out = dict(y=g.new(T, d), ab=g.new(T, 2 * f), s=g.new(T, f),
               dx=g.new(T, d), dwg=g.new(2 * f, d), dw2=g.new(d, f))
    ws = _ws(moe.MOE_ENTRY_FFN_FWD, T, d, f, g)
    wsb = _ws(moe.MOE_ENTRY_FFN_BWD, T, d, f, g)

    def step(stream=None):
        o = out
        moe.moe_ffn_fwd(0, D["x"], D["w_gu"], D["w2"], D["y_add"], o["ab"],
                        o["s"], o["y"], ws, stream=stream)
        moe.moe_ffn_bwd(0, D["dy"], D["x"], D["w_gu"], D["w2"], o["ab"],
                        o["s"], D["dx_add"], o["dx"], o["dwg"], o["dw2"],
                        wsb, stream=stream)

    step()
    torch.cuda.synchronize()
    ref = {n: t.clone() for n, t in out.items()}
    side = torch.cuda.Stream()
    for t in out.values():
        t.zero_()
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    assert all(torch.equal(out[n], ref[n]) for n in ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in out.values():
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], ref[n]) for n in ref)
    g.check()


def _ref_rows(act, D, ab, s, sl):
    """Float64 backward pieces of the rows sl, on the GPU."""
    f = D["w2"].shape[1]
    a, u = ab[sl, :f].double(), ab[sl, f:].double()
    if act == "silu":
        g = torch.sigmoid(a)
        h, slope = a * g, g * (1 + a * (1 - g))
    else:
        c = (2 / np.pi) ** 0.5
        th = torch.tanh(c * (a + 0.044715 * a ** 3))
        h = 0.5 * a * (1 + th)
        slope = 0.5 * (1 + th) + 0.5 * a * (1 - th * th) * c * (
            1 + 3 * 0.044715 * a * a)
    ds = D["dy"][sl].double() @ D["w2"].double()
    return torch.cat((ds * u * slope, ds * h), dim=1), h * u


def _close(name, got, ref):
    """Mean-square and worst error in units of h and of the mean square: a
    chain of roundings <= h in random order, as above; the worst of up to
    2^30 nearly Gaussian errors stays within 8 of their standard
    deviations, which is below 1.6 h of the output's."""
    err = got.double() - ref
    rms = float(ref.square().mean().sqrt())
    q = float(err.square().mean().sqrt()) / rms / H
    w = float((err.abs() - H * ref.abs()).max()) / rms / H
    print(f"{name}: rms {q:.2f} h, worst {w:.2f} h")
    assert q <= 1.6 and w <= 8 * 1.6, name


# products at which the 256-wide tiles are the estimated best: rows and
# columns ending inside a tile, a last round that is half empty
@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,d,f", [(4090, 4088, 1032), (2050, 4096, 4088),
                                   (8192, 2048, 4096), (4100, 4096, 6136)])
def test_ffn_large_products(T, d, f, act):
    g = Guarded()
    D = _data(T, d, f, seed=T)
    y, ab, s = _run(act, D, T, d, f, True, g)
    y2, _, _ = _run(act, D, T, d, f, True, g, save=False)
    assert torch.equal(y, y2)
    x, wg, w2 = (D[k].double() for k in ("x", "w_gu", "w2"))
    rab = x @ wg.t()
    _close("ab", ab, rab)
    # S and y from the exact gate and up, dAB from the saved ones
    _, hu = _ref_rows(act, D, rab, s, slice(None))
    _close("s", s, hu)
    _close("y", y, hu @ w2.t() + D["y_add"].double())
    dab, _ = _ref_rows(act, D, ab, s, slice(None))
    dx, dwg, dw2 = _bwd(act, D, T, d, f, True, g, ab, s)
    # each gradient alone too: its product in a launch of its own
    alone = (g.new(T, d), g.new(2 * f, d), g.new(d, f))
    for i in range(3):
        o = [t if j == i else None for j, t in enumerate(alone)]
        moe.moe_ffn_bwd(_act(act), D["dy"], D["x"], D["w_gu"], D["w2"], ab,
                        s, D["dx_add"] if i == 0 else None, *o,
                        _ws(moe.MOE_ENTRY_FFN_BWD, T, d, f, g))
    for got in ((dx, dwg, dw2), alone):
        _close("dx", got[0], dab @ wg + D["dx_add"].double())
        _close("dw_gu", got[1], dab.t() @ x)
        _close("dw2", got[2], D["dy"].double().t() @ s.double())
    g.check()


@gpu
def test_ffn_past_32_bit_offsets():
    """dAB of 80000 x 28672 bf16 passes 4 GiB and 2^31 elements: the far rows
    are right and the weight gradients sum all of them."""
    T, d, f = 80000, 64, 14336
    g = Guarded()
    D = _data(T, d, f, seed=6)
    y, ab, s = _run("silu", D, T, d, f, False, g)
    dx, dwg, dw2 = _bwd("silu", D, T, d, f, False, g, ab, s)
    wg, w2 = D["w_gu"].double(), D["w2"].double()
    rwg, rw2 = torch.zeros_like(wg), torch.zeros_like(w2)
    for r0 in range(0, T, 8000):
        sl = slice(r0, r0 + 8000)
        x = D["x"][sl].double()
        dab, _ = _ref_rows("silu", D, ab, s, sl)
        rwg += dab.t() @ x
        rw2 += D["dy"][sl].double().t() @ s[sl].double()
        if r0 in (0, 72000):
            rab = x @ wg.t()
            _close("ab", ab[sl], rab)
            hu = rab[:, :f] * torch.sigmoid(rab[:, :f]) * rab[:, f:]
            _close("y", y[sl], hu @ w2.t())
            _close("dx", dx[sl], dab @ wg)
    _close("dw_gu", dwg, rwg)
    _close("dw2", dw2, rw2)
    g.check()


# the 128 x 64 tiles: fc1 with one group a tile; y over a split reduction;
# [dA dU]; dx; dw2; y and [dA dU] with two groups
TALL = [(137, 264, 3720), (65, 1160, 3208), (2420, 264, 520),
        (2420, 520, 136), (65, 4232, 392), (326, 3720, 4232)]


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,d,f", TALL)
def test_ffn_tall_tiles(T, d, f, act):
    test_ffn_parity(T, d, f, act)
