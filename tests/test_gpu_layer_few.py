"""GPU parity of moe_layer_fwd (through the C-ABI) against the layer's
formulas in float64, element by element, within bounds derived from the
kernel's arithmetic, u = 2^-24:
  * a score is a sum of d products in 64 lanes: at most d / 64 + 8 + 7
    additions in a row, e_z = (d / 64 + 16) u sum |x w|;
  * a routing weight: its exponent is off by 2 e_z, expf and the division by
    4 u, the sum by (E + 16) u at most: w (2 e_z + (E + 24) u);
  * gate and up: each half of a wave's lanes adds 32 products for every 64 k.
    Where a wave goes through the whole sum it joins two halves, 32 ceil(d /
    64) + 1 additions in a row at most; where four waves take 256 k in turn,
    128 ceil(d / 1024) and 8 sums: with c the larger, e_a = c u sum |x G|;
  * S = w silu(a) v: silu has a slope below 1.1 and costs 8 u (exponential,
    reciprocal, products): e_S = |w| (|v| (1.1 e_a + 8 u |a|) + |silu(a)|
    e_v) + |S| (2 e_z + (E + 28) u), and it is held as two bf16 values, the
    second of which rounds what the first leaves: 2^-8 2^-8 |S|;
  * y: where a wave adds an expert's products whole, 32 ceil(f / 64) in a row
    and then two halves, S's two parts, n experts, and at most 64 parts of the
    reduction (16 in a row, then 2 sums); where 16 waves take 256 k of the n
    experts in turn, 128 ceil(n ceil(f / 256) / 16), then 32 sums, S's parts
    and up to 8 parts: with c' the larger, sum (e_S + c' u |S| (1 + 2^-7))
    |W2| + 2 u |y_add| + 2^-8 |y|, where 1 + 2^-7 is above |S's parts| / |S|.
"""

import math

import numpy as np
import pytest
import torch

from mixture_experts_expert_top_amd import inputs as I

gpu = pytest.mark.gpu
U = 2.0 ** -24
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8

if torch.cuda.is_available():
    from mixture_experts_expert_top_amd import moe


def decode(codes, scales):
    """float64 values of E4M3 codes with E8M0 scales along the last axis."""
    v = codes.view(torch.float8_e4m3fn).double()
    s = torch.exp2(scales.double() - 127.0)
    return (v.view(*s.shape, 32) * s[..., None]).view(v.shape)


class Case:
    """Inputs and buffers of one call."""

    def __init__(self, T, d, f, E, k, mx=False, bias=False, add=False,
                 seed=0, weights=None, w_scale=None):
        dev = torch.device("cuda:0")
        mk = lambda shape, i, s=1.0, dt=BF: I.make_tensor(  # noqa: E731
            shape, seed=seed * 11 + i, scale=s, dtype=dt, device=dev)
        self.T, self.d, self.f, self.E, self.k, self.mx = T, d, f, E, k, mx
        self.x = mk((T, d), 0)
        self.w_g = mk((E, d), 1, d ** -0.5)
        self.bias = mk((E,), 2, 0.2, F32) if bias else None
        self.y_add = mk((T, d), 3) if add else None
        self.logits = None
        s = 0.05 if w_scale is None else w_scale
        self.wb = [mk((E, 2 * f, d), 4, s), mk((E, d, f), 5, s)]
        self.w, self.s = list(self.wb), [None, None]
        if mx:
            for i, w in enumerate(self.wb):
                c = torch.empty(w.shape, dtype=U8, device=dev)
                n = w.shape[2] // 32
                sc = torch.empty(*w.shape[:2], n, dtype=U8, device=dev)
                moe.moe_mxfp8_quantize(w.view(-1, w.shape[2]), 0, None,
                                       c.view(-1, w.shape[2]),
                                       sc.view(-1, n))
                self.w[i], self.s[i] = c, sc
        self.prec = moe.MOE_MXFP8 if mx else moe.MOE_BF16
        n = moe.moe_workspace_bytes(moe.MOE_ENTRY_LAYER_FWD, self.prec, T, E,
                                    k, d, f)
        assert n > 0
        self.ws = torch.full((n,), 255, dtype=U8, device=dev)
        self.y = torch.full((T, d), float("nan"), dtype=BF, device=dev)
        self.idx = torch.full((T, k), -1, dtype=torch.int32, device=dev)
        self.p = torch.full((T, k), float("nan"), device=dev)

    def run(self, renorm=True, y=None, y_add="own", **kw):
        own_logits = self.logits is not None
        moe.moe_layer_fwd(
            self.prec, self.x, None if own_logits else self.w_g,
            None if own_logits else self.bias, self.logits, self.k, renorm,
            self.w[0], self.s[0], self.w[1], self.s[1],
            self.y_add if isinstance(y_add, str) else y_add, self.idx,
            self.p, self.y if y is None else y, self.ws, **kw)
        return self.y if y is None else y


def reference(c, renorm=True):
    """idx, weights, y, and the bounds of the weights and of y."""
    T, d, f, E, k = c.T, c.d, c.f, c.E, c.k
    x = c.x.double()
    if c.logits is not None:
        z, ez = c.logits.double(), torch.zeros(T, E, device=x.device)
    else:
        wg = c.w_g.double()
        z = x @ wg.t()
        ez = (d / 64 + 16) * U * (x.abs() @ wg.abs().t())
        if c.bias is not None:
            z = z + c.bias.double()
            ez = ez + U * z.abs()
    order = torch.sort(z, dim=1, descending=True, stable=True)[1]
    idx = order[:, :k]
    p = torch.softmax(z, 1)
    w = torch.gather(p, 1, idx)
    if renorm:
        w = torch.softmax(torch.gather(z, 1, idx), 1)
    rel = 2 * ez.max(dim=1, keepdim=True)[0] + (E + 24) * U
    # a choice is settled where the k-th and the next score differ by more
    # than both may be off
    s = torch.sort(z, dim=1, descending=True)[0]
    gap = (s[:, :-1] - s[:, 1:])[:, :k] if E > 1 else s[:, :0]
    settled = (gap > 2 * ez.max(dim=1, keepdim=True)[0]).all(dim=1) | (
        torch.full((T,), c.logits is not None, device=x.device))
    y = torch.zeros(T, d, dtype=torch.float64, device=x.device)
    b = torch.zeros_like(y)
    reached = torch.unique(idx).tolist()
    n = len(reached)
    ca = max(32 * math.ceil(d / 64) + 1, 128 * math.ceil(d / 1024) + 8)
    cy = max(32 * math.ceil(f / 64) + 2 + n + 18,
             128 * math.ceil(n * math.ceil(f / 256) / 16) + 32 + 1 + 8)
    for e in reached:
        tok, slot = torch.nonzero(idx == e, as_tuple=True)
        if c.mx:
            w1, w2 = (decode(c.w[i][e], c.s[i][e]) for i in (0, 1))
        else:
            w1, w2 = c.w[0][e].double(), c.w[1][e].double()
        ab = x[tok] @ w1.t()
        eab = ca * U * (x[tok].abs() @ w1.abs().t())
        a, v, ea, ev = ab[:, :f], ab[:, f:], eab[:, :f], eab[:, f:]
        sl = a * torch.sigmoid(a)
        pw = w[tok, slot][:, None]
        S = pw * sl * v
        eS = (pw * (v.abs() * (1.1 * ea + 8 * U * a.abs()) + sl.abs() * ev) +
              S.abs() * (rel[tok] + 4 * U) + 2.0 ** -16 * S.abs())
        y[tok] += S @ w2.t()
        b[tok] += (eS + cy * U * (1 + 2.0 ** -7) * S.abs()) @ w2.abs().t()
    if c.y_add is not None:
        y += c.y_add.double()
        b += 2 * U * c.y_add.double().abs()
    b += 2.0 ** -8 * (y.abs() + b)
    return idx, w, y, w * rel, b, settled


def check(c, renorm=True, y=None):
    idx, w, ref, ew, bound, settled = reference(c, renorm)
    got = c.y if y is None else y
    assert torch.isfinite(got).all()
    n = int(settled.sum())
    assert n >= 0.9 * c.T          # scores next to each other are rare
    assert torch.equal(c.idx[settled].long(), idx[settled])
    assert ((c.p.double() - w).abs() <= ew + 1e-300)[settled].all()
    off = ((got.double() - ref).abs() / bound.clamp(min=1e-300))[settled]
    assert float(off.max()) <= 1.0, float(off.max())


# tokens at the edges of the blocks of 8; widths below, at and past a chunk of
# 256, a wave round of 2048 and off them; experts as slots and as a grid
SIZES = [
    (1, 8, 8, 1, 1), (1, 64, 16, 4, 2), (3, 32, 64, 4, 2),
    (1, 2048, 1408, 64, 8), (2, 264, 72, 7, 7), (5, 2056, 264, 16, 4),
    (8, 256, 256, 9, 3), (9, 520, 136, 3, 2), (16, 1032, 680, 41, 3),
    (17, 136, 1000, 5, 1), (24, 512, 264, 64, 8), (32, 2304, 40, 2, 1),
    (33, 72, 2600, 6, 2), (61, 1032, 680, 41, 3), (64, 128, 128, 1, 1),
    (64, 96, 48, 130, 32), (7, 16, 24, 1024, 32), (64, 24, 16, 1024, 4),
    (1, 4104, 2056, 3, 2), (40, 4096, 24, 300, 2), (34, 1664, 160, 11, 6),
    (64, 512, 2048, 20, 8)]


@gpu
@pytest.mark.parametrize("T,d,f,E,k", SIZES)
@pytest.mark.parametrize("renorm", [True, False])
def test_bf16(T, d, f, E, k, renorm):
    c = Case(T, d, f, E, k, bias=T % 2 == 0, add=d % 16 == 0, seed=T + d)
    c.run(renorm)
    check(c, renorm)


@gpu
@pytest.mark.parametrize("T,d,f,E,k", [
    (1, 128, 128, 1, 1), (1, 2048, 1408, 64, 8), (3, 256, 384, 4, 2),
    (8, 640, 128, 9, 3), (24, 512, 256, 64, 8), (33, 128, 2688, 6, 2),
    (64, 2176, 384, 2, 1), (64, 384, 128, 130, 8), (16, 4096, 640, 8, 2)])
@pytest.mark.parametrize("renorm", [True, False])
def test_mxfp8(T, d, f, E, k, renorm):
    c = Case(T, d, f, E, k, mx=True, bias=T % 2 == 1, add=d % 256 == 0,
             seed=T + f)
    c.run(renorm)
    check(c, renorm)


@gpu
def test_mxfp8_scales_from_tiny_to_large():
    """Scale bytes over their range, and blocks of zeros."""
    c = Case(4, 256, 256, 3, 2, mx=True, seed=5)
    g = torch.Generator(device="cuda:0")
    g.manual_seed(3)
    for i in (0, 1):
        shift = torch.randint(-40, 8, c.s[i].shape, generator=g,
                              device="cuda:0")
        c.s[i] = (c.s[i].int() + shift).clamp(0, 254).to(U8)
        c.w[i].view(*c.s[i].shape, 32)[:, ::5, 1] = 0
        c.s[i][:, ::5, 1] = 0
    c.run()
    check(c)


@gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [8, 9, 20, 64])
def test_every_token_to_one_expert(T, mx):
    """An expert with all tokens and experts with none."""
    c = Case(T, 384, 256, 12, 2, mx=mx, add=True, seed=T)
    c.logits = I.make_tensor((T, 12), seed=7, dtype=F32, device="cuda:0")
    c.logits[:, 5] = 20.0
    c.logits[:, :3] = -30.0
    c.run()
    check(c)


@gpu
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (5, 64, 8), (64, 40, 32),
                                   (3, 1024, 32), (13, 1, 1)])
@pytest.mark.parametrize("renorm", [True, False])
def test_routing_as_moe_route(T, E, k, renorm):
    """Ties, signed zeros, infinities and NaN are chosen as moe_route does."""
    c = Case(T, 16, 8, E, k, seed=E)
    L = I.make_tensor((T, E), seed=1, dtype=F32, device="cuda:0")
    L = (L * 4).round() / 4                     # many ties
    L[0, ::3] = 0.0
    L[0, 1::3] = -0.0
    if T > 2:
        L[1, ::2] = float("-inf")
        L[2, E // 2] = float("nan")
        L[2, 0] = float("-inf")
    c.logits = L
    c.run(renorm)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda:0")
    w = torch.empty(T, k, device="cuda:0")
    moe.moe_route(L, k, renorm, idx, w)
    assert torch.equal(c.idx, idx)
    same = torch.isnan(w) == torch.isnan(c.p)
    assert same.all()
    ok = ~torch.isnan(w)
    assert ((c.p - w).abs()[ok] <= (2 * E + 8) * U * w[ok] + 1e-37).all()


@gpu
@pytest.mark.parametrize("T", [6, 40])
def test_bad_values_stay_with_their_tokens(T):
    """A token of NaN or infinities, and an expert of them, leave the other
    tokens' bits as they are."""
    c = Case(T, 520, 264, 6, 2, seed=3)
    c.logits = torch.full((T, 6), -9.0, device="cuda:0")
    t = torch.arange(T, device="cuda:0")
    c.logits[t, t % 5] = 2.0
    c.logits[t, (t + 1) % 5] = 1.0
    want = c.run().clone()
    c.x[2] = float("nan")
    c.x[4, 7] = float("inf")
    c.w[0][5].fill_(float("nan"))           # nobody's
    c.w[1][3, 9, :] = float("inf")
    got = c.run()
    bad = ((t == 2) | (t == 4))[:, None].expand(T, 520).clone()
    hit = ((t % 5 == 3) | ((t + 1) % 5 == 3))
    bad[hit, 9] = True
    assert torch.equal(got[~bad], want[~bad])
    assert torch.isnan(got[2]).all() and not torch.isfinite(got[hit, 9]).any()


@gpu
@pytest.mark.parametrize("mx", [False, True])
def test_sum_into_y_and_neighbours(mx):
    """y may be y_add; what lies around every output stays as it was."""
    T, d, f, E, k = 11, 384, 128, 10, 3
    c = Case(T, d, f, E, k, mx=mx, add=True, seed=2)
    want = c.run().clone()
    big = torch.full((T + 2, d), 7.0, dtype=BF, device="cuda:0")
    big[1:-1] = c.y_add
    c.run(y=big[1:-1], y_add=big[1:-1])
    assert torch.equal(big[1:-1], want)
    assert (big[0] == 7).all() and (big[-1] == 7).all()
    n = c.ws.numel()
    ws = torch.full((n + 512,), 9, dtype=U8, device="cuda:0")
    c.ws = ws[256:256 + n]
    c.run()
    assert torch.equal(c.y, want)
    assert (ws[:256] == 9).all() and (ws[256 + n:] == 9).all()


@gpu
@pytest.mark.parametrize("T", [2, 12])
def test_past_32_bit_offsets(T):
    """Weights past 4 GiB, the last and the first expert."""
    d, f, E, k = 4096, 14336, 20, 2
    c = Case(1, 8, 8, 1, 1)
    dev = torch.device("cuda:0")
    c.T, c.d, c.f, c.E, c.k = T, d, f, E, k
    c.x = I.make_tensor((T, d), seed=1, device=dev)
    w1 = torch.zeros(E, 2 * f, d, dtype=BF, device=dev)
    w2 = torch.zeros(E, d, f, dtype=BF, device=dev)
    for e in (0, 18, 19):
        w1[e] = I.make_tensor((2 * f, d), seed=e, scale=0.02, device=dev)
        w2[e] = I.make_tensor((d, f), seed=e + 50, scale=0.02, device=dev)
    c.w = [w1, w2]
    c.logits = torch.full((T, E), -5.0, device=dev)
    c.logits[0, 19], c.logits[0, 0] = 1.0, 0.5
    c.logits[1, 18], c.logits[1, 19] = 1.0, 0.5
    c.ws = torch.empty(moe.moe_workspace_bytes(
        moe.MOE_ENTRY_LAYER_FWD, c.prec, T, E, k, d, f), dtype=U8, device=dev)
    c.y = torch.empty(T, d, dtype=BF, device=dev)
    c.idx = torch.empty(T, k, dtype=torch.int32, device=dev)
    c.p = torch.empty(T, k, device=dev)
    c.run()
    check(c)


@gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 19])
def test_captured_and_replayed(T, mx):
    """Replays with new tokens in place, eager calls between them, are the
    eager call's bits; so are two streams at once with a workspace each."""
    c, e = (Case(T, 640, 384, 12, 3, mx=mx, bias=True, add=True, seed=4)
            for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    c.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        c.run()
    for i in range(4):
        x = I.make_tensor((T, 640), seed=90 + i, device="cuda:0")
        c.x.copy_(x)
        e.x.copy_(x)
        c.y.fill_(float("nan"))
        c.ws.fill_(i * 50)
        graph.replay()
        e.run()
        torch.cuda.synchronize()
        assert torch.equal(c.y, e.y) and torch.equal(c.idx, e.idx)
        assert torch.equal(c.p, e.p)
    streams = [torch.cuda.Stream() for _ in range(2)]
    want = e.y.clone()
    for s, q in zip(streams, (c, e)):
        q.y.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for s, q in zip(streams, (c, e)):
            q.run(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(c.y, want) and torch.equal(e.y, want)


@gpu
def test_binding_refuses():
    c = Case(2, 128, 128, 4, 2)
    for name, bad, exc in (
            ("x", c.x.float(), TypeError), ("x", c.x.t(), ValueError),
            ("y", c.y[:1], ValueError), ("idx", c.idx.long(), TypeError),
            ("w_g", c.w_g[:3], ValueError), ("p", c.p.cpu(), ValueError),
            ("ws", c.ws[:16], moe.MoeError), ("ws", None, moe.MoeError),
            ("w_g", None, moe.MoeError), ("y", c.x, moe.MoeError),
            ("y_add", c.x[:1], ValueError), ("k", 3, ValueError)):
        keep = getattr(c, name)
        setattr(c, name, bad)
        with pytest.raises(exc):
            c.run()
        setattr(c, name, keep)
    c.s = [torch.zeros(4, 256, 4, dtype=U8, device="cuda:0"), None]
    with pytest.raises((moe.MoeError, ValueError)):
        c.run()
    big = Case(1, 16, 8, 2, 1)
    big.x = torch.zeros(65, 16, dtype=BF, device="cuda:0")
    big.y = torch.zeros_like(big.x)
    big.idx = torch.zeros(65, 1, dtype=torch.int32, device="cuda:0")
    big.p = torch.zeros(65, 1, device="cuda:0")
    with pytest.raises(moe.MoeError, match="64"):
        big.run()


@gpu
@pytest.mark.parametrize("T,E,k", [(1, 64, 8), (4, 65, 3), (8, 200, 32),
                                   (7, 256, 9), (8, 257, 5), (9, 256, 8),
                                   (2, 130, 32), (8, 5, 5)])
@pytest.mark.parametrize("renorm", [True, False])
def test_routing_inside_the_first_product_and_apart(T, E, k, renorm):
    """Both sides of what is chosen inside a kernel, ties and special values
    included, are moe_route's choices."""
    c = Case(T, 16, 16, E, k, seed=E)
    L = (I.make_tensor((T, E), seed=2, dtype=F32, device="cuda:0") * 2).round()
    L[0, E // 2] = float("nan")
    L[T - 1, :] = 1.5
    L[T // 2, ::2] = float("-inf")
    L[T // 2, 1::4] = -0.0
    c.logits = L
    c.run(renorm)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda:0")
    w = torch.empty(T, k, device="cuda:0")
    moe.moe_route(L, k, renorm, idx, w)
    assert torch.equal(c.idx, idx)
    ok = ~torch.isnan(w)
    assert torch.equal(ok, ~torch.isnan(c.p))
    assert ((c.p - w).abs()[ok] <= (2 * E + 8) * U * w[ok] + 1e-37).all()


@gpu
@pytest.mark.parametrize("mx", [False, True])
def test_an_expert_past_32_members_and_small_ones(mx):
    """Parts of y whose experts hold 0 to 64 of the tokens."""
    T, E = 64, 20
    c = Case(T, 640, 1152, E, 3, mx=mx, add=True, seed=9)
    L = I.make_tensor((T, E), seed=3, dtype=F32, device="cuda:0")
    L[:, 7] = 9.0
    L[:40, 3] = 8.0
    L[:, 11:] -= 4.0
    c.logits = L
    c.run()
    check(c)


@gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [2, 3, 4, 7, 20])
def test_bad_weights_stay_with_their_expert(T, mx):
    """A NaN, an infinity or (MXFP8) a NaN scale reaches the tokens of its
    expert, in the columns that it belongs to, and no others."""
    c = Case(T, 256, 384, 4, 1, mx=mx, seed=8)
    c.logits = torch.full((T, 4), -9.0, device="cuda:0")
    t = torch.arange(T, device="cuda:0")
    c.logits[t, t % 3] = 2.0
    want = c.run().clone()
    if mx:
        c.w[0][3].fill_(127)               # nobody's
        c.w[1][0, 9, 77] = 127             # a NaN of E4M3
        c.s[1][1, 30, 5] = 255             # a NaN of E8M0
    else:
        c.w[0][3].fill_(float("nan"))
        c.w[1][0, 9, 77] = float("nan")
        c.w[1][1, 30, 5] = float("inf")
    got = c.run()
    bad = torch.zeros(T, 256, dtype=torch.bool, device="cuda:0")
    bad[t % 3 == 0, 9] = True
    bad[t % 3 == 1, 30] = True
    assert torch.equal(got[~bad], want[~bad])
    assert not torch.isfinite(got[bad]).any()
