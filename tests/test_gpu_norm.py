"""GPU parity of moe_norm_fwd / moe_norm_bwd (through the C-ABI) against the
float64 oracle, element by element, within bounds derived from the kernel's
arithmetic (u = 2^-24, A = mean |x| of the row, chains of at most 48
additions a row sum: 16 in a lane, 6 exchanges, 16 waves and a product):
  * mean: |err| <= 48 u A; a centred value: that + u |xc|;
  * rstd: the variance is a sum of squares of centred values (48 u, plus the
    square of the mean's error, plus 2 u a term), halved by the root: 64 u
    with the root's and the division's rounding; so
    dxh := 48 u A rstd + 66 u |xh| bounds the error of xh;
  * y: |gamma| dxh + 2 u (|y| + |beta|) + 2^-8 |y| (one bf16 rounding);
  * dx: with c0 = mean(g xh), c1 = mean(g): their errors are
    e0 = mean(|g| dxh) + 50 u mean|g xh| and e1 = 50 u mean|g|, and dx is off
    by rstd (e1 + |xh| e0 + |c0| dxh + 70 u (|g| + |c1| + |xh c0|)) plus
    2 u |dres| and one rounding to its type;
  * dgamma, dbeta: a column's sum is at most T + 64 additions in any order:
    (T + 64) u sum|dy xh| + sum |dy| dxh, and (T + 64) u sum|dy|.
"""

import numpy as np
import pytest
import torch

from mixture_experts_expert_top_amd import inputs as I
from oracle import block_ref as B

gpu = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5

if torch.cuda.is_available():
    from mixture_experts_expert_top_amd import moe

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}

# T, d: every width class (16 lanes, one wave of one or two chunks, 4, 8 and
# 16 waves) at its edges, rows fewer and more than the grid holds
SIZES = [(1, 8), (19, 128), (5, 136), (1, 512), (6, 520), (37, 1024),
         (3, 1032), (130, 2048), (2, 2056), (1, 4096), (2100, 4096),
         (3, 4104), (5, 8192), (2, 8200), (3, 16384), (9001, 64),
         (17001, 16), (5000, 264), (257, 16000)]


def h64(t):
    return t.double().cpu().numpy()


def _data(T, d, xt, seed, shift=0.3):
    dev = torch.device("cuda:0")
    mk = lambda shape, k, s=1.0, dt=F32: I.make_tensor(  # noqa: E731
        shape, seed=seed * 7 + k, scale=s, dtype=dt, device=dev)
    x = (mk((T, d), 0) + shift).to(xt)
    return (x, 1.0 + mk((d,), 1, 0.2), mk((d,), 2, 0.3),
            mk((T, d), 3, dt=BF), mk((T, d), 4, dt=xt))


def _check(name, got, ref, bound):
    err = np.abs(h64(got) - ref)
    assert np.isfinite(h64(got)).all(), name
    worst = float(np.max(err / np.maximum(bound, 1e-300)))
    print(f"{name}: max|err|/bound = {worst:.3f}")
    assert worst <= 1.0, name


def _guarded(shape, dt, dev):
    """A tensor inside a larger one filled with a pattern, and a check that
    the surroundings kept it."""
    n = int(np.prod(shape))
    pad = 64
    buf = torch.full((n + 2 * pad,), -77.0, dtype=dt, device=dev)
    t = buf[pad:pad + n].view(shape)

    def intact():
        assert (buf[:pad] == -77.0).all() and (buf[pad + n:] == -77.0).all()
    return t, intact


@gpu
@pytest.mark.parametrize("xt", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("T,d", SIZES)
def test_norm_parity(T, d, rms, xt):
    dev = torch.device("cuda:0")
    x, gamma, beta, dy, dres = _data(T, d, xt, seed=T + d)
    kind = moe.MOE_NORM_RMS if rms else moe.MOE_NORM_LAYER
    if rms:
        beta = None
    bufs = {}
    for n, shape, dt in (("y", (T, d), BF), ("mean", (T,), F32),
                         ("rstd", (T,), F32), ("dx", (T, d), xt),
                         ("dgamma", (d,), F32), ("dbeta", (d,), F32)):
        bufs[n] = _guarded(shape, dt, dev)
    y, mean, rstd, dx, dgamma, dbeta = (bufs[n][0] for n in bufs)
    ws = torch.empty(moe.moe_workspace_bytes(moe.MOE_ENTRY_NORM_BWD, 0, T, 1,
                                             1, d, 0), dtype=torch.uint8,
                     device=dev)
    moe.moe_norm_fwd(kind, x, gamma, beta, EPS, y, None if rms else mean,
                     rstd)
    moe.moe_norm_bwd(kind, dy, x, gamma, None if rms else mean, rstd, dres,
                     dx, dgamma, None if rms else dbeta, ws)
    torch.cuda.synchronize()
    for _, intact in bufs.values():
        intact()

    X, G, DY, DR = h64(x), h64(gamma), h64(dy), h64(dres)
    BE = 0.0 if rms else h64(beta)
    ry, rm, rr = B.norm_forward(X, G, None if rms else BE, EPS, rms)
    rdx, rdg, rdb = B.norm_backward(DY, X, G, EPS, rms, DR)
    A = np.abs(X).mean(axis=1, keepdims=True)
    r = rr[:, None]
    xh = (X - rm[:, None]) * r
    dxh = (0.0 if rms else 48 * U) * A * r + 66 * U * np.abs(xh)
    _check("y", y, ry, np.abs(G) * dxh + 2 * U * (np.abs(ry) + np.abs(BE)) +
           HALF[BF] * np.abs(ry))
    if not rms:
        _check("mean", mean, rm, 48 * U * A[:, 0])
    _check("rstd", rstd, rr, 66 * U * rr +
           (0.0 if rms else (48 * U * A[:, 0] * rr) ** 2 * rr))
    g = np.abs(DY * G)
    c0 = np.abs((DY * G * xh).mean(axis=1, keepdims=True))
    c1 = 0.0 if rms else np.abs((DY * G).mean(axis=1, keepdims=True))
    e0 = ((g * dxh).mean(axis=1, keepdims=True) +
          50 * U * (g * np.abs(xh)).mean(axis=1, keepdims=True))
    e1 = 0.0 if rms else 50 * U * g.mean(axis=1, keepdims=True)
    bound = r * (e1 + np.abs(xh) * e0 + c0 * dxh +
                 70 * U * (g + c1 + np.abs(xh) * c0))
    _check("dx", dx, rdx, bound + 2 * U * np.abs(DR) +
           HALF[xt] * (np.abs(rdx) + bound))
    _check("dgamma", dgamma, rdg, (T + 64) * U * np.abs(DY * xh).sum(axis=0) +
           (np.abs(DY) * dxh).sum(axis=0))
    if not rms:
        _check("dbeta", dbeta, rdb, (T + 64) * U * np.abs(DY).sum(axis=0))


@gpu
def test_norm_optional_outputs_and_alias():
    """Missing outputs and residual leave the others' bits as they are; dx may
    be dres itself; no workspace without weight gradients; equal calls give
    equal bits."""
    dev = torch.device("cuda:0")
    T, d = 77, 1040
    x, gamma, beta, dy, dres = _data(T, d, BF, seed=3)
    y, y2 = torch.empty(T, d, dtype=BF, device=dev), torch.empty(
        T, d, dtype=BF, device=dev)
    mean, rstd = torch.empty(T, device=dev), torch.empty(T, device=dev)
    L = moe.MOE_NORM_LAYER
    moe.moe_norm_fwd(L, x, gamma, beta, EPS, y, mean, rstd)
    moe.moe_norm_fwd(L, x, gamma, beta, EPS, y2)
    assert torch.equal(y, y2)
    ws = torch.empty(moe.moe_workspace_bytes(moe.MOE_ENTRY_NORM_BWD, 0, T, 1,
                                             1, d, 0), dtype=torch.uint8,
                     device=dev)
    new = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device=dev)  # noqa
    dx, dg, db = new(T, d, dt=BF), new(d), new(d)
    moe.moe_norm_bwd(L, dy, x, gamma, mean, rstd, dres, dx, dg, db, ws)
    alias, dg2, db2 = dres.clone(), new(d), new(d)
    moe.moe_norm_bwd(L, dy, x, gamma, mean, rstd, alias, alias, dg2, None, ws)
    assert torch.equal(alias, dx) and torch.equal(dg2, dg)
    moe.moe_norm_bwd(L, dy, x, gamma, mean, rstd, dres, alias, None, db2, ws)
    assert torch.equal(db2, db)
    alias.zero_()
    moe.moe_norm_bwd(L, dy, x, gamma, mean, rstd, dres, alias, None, None,
                     None)
    assert torch.equal(alias, dx)
    # without a residual: the difference to a zero residual is nothing
    moe.moe_norm_bwd(L, dy, x, gamma, mean, rstd, None, alias, dg2, db2, ws)
    moe.moe_norm_bwd(L, dy, x, gamma, mean, rstd, torch.zeros_like(dres), dx,
                     dg, db, ws)
    assert torch.equal(alias, dx) and torch.equal(dg, dg2)
    assert torch.equal(db, db2)


@gpu
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_norm_far_mean_constant_and_nonfinite_rows(rms):
    """A row far from zero keeps its variance (centred sums), a constant row
    gives beta, and a NaN or infinite row stays in its own row."""
    dev = torch.device("cuda:0")
    T, d = 6, 4096
    x, gamma, beta, dy, _ = _data(T, d, F32, seed=9)
    if rms:
        beta = None
    x[1] = 1000.0 + x[1] * 0.01
    x[2] = 7.0
    x[4, 17] = float("nan")
    x[5, 3] = float("inf")
    y = torch.empty(T, d, dtype=BF, device=dev)
    mean, rstd = torch.empty(T, device=dev), torch.empty(T, device=dev)
    kind = moe.MOE_NORM_RMS if rms else moe.MOE_NORM_LAYER
    moe.moe_norm_fwd(kind, x, gamma, beta, EPS, y, None if rms else mean,
                     rstd)
    dx = torch.empty_like(x)
    moe.moe_norm_bwd(kind, dy, x, gamma, None if rms else mean, rstd, None,
                     dx, None, None, None)
    ok = slice(0, 4)
    X, G = h64(x)[ok], h64(gamma)
    BE = None if rms else h64(beta)
    ry, rm, rr = B.norm_forward(X, G, BE, EPS, rms)
    if not rms:
        # the mean of row 1 is off by at most 48 u 1000 = 2.9e-3, against a
        # standard deviation of 0.01; its square enters the variance
        e = (48 * U * np.abs(X).mean(axis=1)) * rr
        assert (np.abs(h64(rstd)[ok] - rr) <=
                rr * (66 * U + 0.5 * e * e + 2 * U * e)).all()
        assert torch.equal(y[2], beta.to(BF))
    assert np.isfinite(h64(y)[ok]).all() and np.isfinite(h64(dx)[ok]).all()
    assert torch.isnan(y[4]).all()
    assert torch.isnan(y[5]).any() and torch.isnan(dx[4]).all()


@gpu
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_norm_gradient_against_differences(rms):
    """<dx, v>, <dgamma, v> and <dbeta, v> against central differences of the
    float64 forward.  fp32 dx is within 2^-13 of its norm here (the bounds of
    the parity test summed over 64 x 8 columns), the quotient within 1e-6."""
    dev = torch.device("cuda:0")
    T, d = 5, 264
    x, gamma, beta, dy, _ = _data(T, d, F32, seed=21)
    if rms:
        beta = None
    kind = moe.MOE_NORM_RMS if rms else moe.MOE_NORM_LAYER
    y = torch.empty(T, d, dtype=BF, device=dev)
    mean, rstd = torch.empty(T, device=dev), torch.empty(T, device=dev)
    dx, dg, db = (torch.empty_like(x), torch.empty(d, device=dev),
                  torch.empty(d, device=dev))
    ws = torch.empty(moe.moe_workspace_bytes(moe.MOE_ENTRY_NORM_BWD, 0, T, 1,
                                             1, d, 0), dtype=torch.uint8,
                     device=dev)
    moe.moe_norm_fwd(kind, x, gamma, beta, EPS, y, None if rms else mean,
                     rstd)
    moe.moe_norm_bwd(kind, dy, x, gamma, None if rms else mean, rstd, None,
                     dx, dg, None if rms else db, ws)
    X, G, DY = h64(x), h64(gamma), h64(dy)
    BE = None if rms else h64(beta)

    def loss(x_, g_, b_):
        return float((B.norm_forward(x_, g_, b_, EPS, rms)[0] * DY).sum())

    rng = np.random.default_rng(4)
    h = 1e-5
    trial = [(X, h64(dx), lambda t: loss(t, G, BE)),
             (G, h64(dg), lambda t: loss(X, t, BE))]
    if not rms:
        trial.append((BE, h64(db), lambda t: loss(X, G, t)))
    for base, grad, fun in trial:
        v = rng.normal(size=base.shape)
        quot = (fun(base + h * v) - fun(base - h * v)) / (2 * h)
        tol = (2.0 ** -13 + 1e-6) * np.linalg.norm(grad) * np.linalg.norm(v)
        assert abs(quot - (grad * v).sum()) <= tol


@gpu
def test_norm_on_another_stream_and_in_a_graph():
    dev = torch.device("cuda:0")
    T, d = 300, 2048
    x, gamma, beta, dy, dres = _data(T, d, BF, seed=5)
    new = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device=dev)  # noqa
    out = dict(y=new(T, d, dt=BF), mean=new(T), rstd=new(T),
               dx=new(T, d, dt=BF), dg=new(d), db=new(d))
    ws = new(moe.moe_workspace_bytes(moe.MOE_ENTRY_NORM_BWD, 0, T, 1, 1, d,
                                     0), dt=torch.uint8)

    def step(stream=None):
        o = out
        moe.moe_norm_fwd(0, x, gamma, beta, EPS, o["y"], o["mean"],
                         o["rstd"], stream=stream)
        moe.moe_norm_bwd(0, dy, x, gamma, o["mean"], o["rstd"], dres,
                         o["dx"], o["dg"], o["db"], ws, stream=stream)

    step()
    torch.cuda.synchronize()
    ref = {n: t.clone() for n, t in out.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in out.values():
        t.zero_()
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    assert all(torch.equal(out[n], ref[n]) for n in ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for t in out.values():
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], ref[n]) for n in ref)


@gpu
def test_norm_past_32_bit_offsets():
    """600000 x 4096 passes 2^31 elements: the last rows equal those of a
    small call bit for bit (rows do not depend on one another), and the
    gradient of beta sums all rows."""
    dev = torch.device("cuda:0")
    T, d, n = 600000, 4096, 64
    x = torch.empty(T, d, dtype=BF, device=dev)
    for r in range(0, T, 50000):
        x[r:r + 50000].normal_()
    gamma, beta = _data(1, d, F32, 1)[1:3]
    new = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device=dev)  # noqa

    def call(xs):
        t = xs.shape[0]
        o = dict(y=new(t, d, dt=BF), mean=new(t), rstd=new(t))
        moe.moe_norm_fwd(0, xs, gamma, beta, EPS, o["y"], o["mean"],
                         o["rstd"])
        dx, db = new(t, d, dt=BF), new(d)
        ws = new(moe.moe_workspace_bytes(moe.MOE_ENTRY_NORM_BWD, 0, t, 1, 1,
                                         d, 0), dt=torch.uint8)
        moe.moe_norm_bwd(0, o["y"], xs, gamma, o["mean"], o["rstd"], None,
                         dx, None, db, ws)
        return o["y"], o["mean"], o["rstd"], dx, db

    big, small = call(x), call(x[-n:].clone())
    for a, b in zip(big[:4], small[:4]):
        assert torch.equal(a[-n:], b)
    ref = torch.zeros(d, dtype=torch.float64, device=dev)
    mag = torch.zeros_like(ref)
    for r in range(0, T, 50000):
        v = big[0][r:r + 50000].double()
        ref += v.sum(dim=0)
        mag += v.abs().sum(dim=0)
    # chains: the rows of a workgroup, then the partials of a wave, then 16
    chain = T / 512 + 512 / 16 + 16
    assert ((big[4].double() - ref).abs() <= chain * U * mag).all()
