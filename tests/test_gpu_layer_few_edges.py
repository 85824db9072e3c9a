"""moe_layer_fwd where test_gpu_layer_few.py's sizes do not reach, held to its
bounds."""

import pytest
import torch

import test_gpu_layer_few as L
from mixture_experts_expert_top_amd import inputs as I

gpu = pytest.mark.gpu
BF, U8 = torch.bfloat16, torch.uint8

if torch.cuda.is_available():
    from mixture_experts_expert_top_amd import moe


def to_one_expert_each(c, hot=3):
    """Logits that give token t the expert t % hot."""
    c.logits = torch.full((c.T, c.E), -9.0, device="cuda:0")
    t = torch.arange(c.T, device="cuda:0")
    c.logits[t, t % hot] = 2.0
    return t


@gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 2, 4, 7, 20, 64])
@pytest.mark.parametrize("f", [128, 384, 640, 896])
def test_a_nan_scale_stays_in_its_row(T, mx, f):
    """A NaN in the first blocks of a row of w2 (MXFP8: a NaN scale) is no
    part of the row before it, wherever f ends in a load."""
    c = L.Case(T, 256, f, 4, 1, mx=mx, seed=8)
    t = to_one_expert_each(c)
    want = c.run().clone()
    rows = (1, 8, 16, 30, 128, 255)
    for i, r in enumerate(rows):
        if mx:
            c.s[1][0, r, i % 4] = 255
        else:
            c.w[1][0, r, 32 * (i % 4)] = float("nan")
    got = c.run()
    bad = torch.zeros(T, 256, dtype=torch.bool, device="cuda:0")
    for r in rows:
        bad[t % 3 == 0, r] = True
    assert torch.equal(got[~bad], want[~bad])
    assert not torch.isfinite(got[bad]).any()


@gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,first", [(1, 0), (1, 1), (1, 3), (4, 0), (7, 0),
                                     (20, 0), (64, 0)])
def test_values_of_s_past_the_end_of_bf16(T, first, mx):
    """One value of S a token, times rows of w2 of +-2^-100 and 0: an infinite
    one gives infinities (and NaN at 0), as a single product would; one between
    bf16's largest value and fp32's gives 2^28 (1 - 2^-10); S itself is off by
    12 u and held to 2^-16, y rounds to 2^-8."""
    dev = torch.device("cuda:0")
    c = L.Case(T, 128, 128, 2, 1, mx=mx, seed=1)
    c.logits = torch.tensor([[1.0, -1.0]], device=dev).repeat(T, 1)
    a = [2.0 ** 70, 2.0 ** 64 * (1 + 2.0 ** -5), 2.0, 2.0 ** 64]
    u = [2.0 ** 70, 2.0 ** 64 * (1 - 2.0 ** -5), 3.0, -2.0 ** 80]
    kind = [(t + first) % 4 for t in range(T)]
    c.x.zero_()
    for t, i in enumerate(kind):
        c.x[t, 0], c.x[t, 1] = a[i], u[i]
    for w in c.w:
        w.zero_()
    one, minus = (0x38, 0xB8) if mx else (1.0, -1.0)
    c.w[0][0, 0, 0] = one               # gate reads x[0], up x[1]
    c.w[0][0, 128, 1] = one
    if mx:
        c.s[0].fill_(127)
        c.s[1].fill_(27)
    else:
        one, minus = 2.0 ** -100, -2.0 ** -100
    c.w[1][0, ::2, 0], c.w[1][0, 1::2, 0] = one, minus
    c.w[1][0, 7, 0] = 0
    y = c.run().double()
    sign = torch.ones(128, dtype=torch.float64, device=dev)
    sign[1::2] = -1
    sign[7] = 0
    live = sign != 0
    for t, i in enumerate(kind):
        if i in (0, 3):
            want = sign * (1 if i == 0 else -1) * float("inf")
            assert torch.equal(y[t][live], want[live]), i
            assert torch.isnan(y[t, 7])
        else:
            S = (torch.tensor(a[i], dtype=torch.float64).sigmoid() * a[i] *
                 u[i])
            want = sign * float(S) * 2.0 ** -100
            tol = (2.0 ** -8 + 2.0 ** -15) * want.abs()
            assert ((y[t] - want).abs() <= tol).all(), i


@gpu
@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("mx,T,d,f,E,k", [
    (False, 1, 1024, 1024, 64, 8),      # 2 parts, 128 tiles
    (False, 1, 520, 1096, 40, 8),       # 2 parts, odd widths
    (False, 2, 264, 2056, 16, 8),       # 4 parts, 33 tiles
    (False, 4, 256, 1000, 64, 8),       # 8 parts
    (False, 3, 16, 264, 300, 32),       # 8 parts of 2 tiles
    (True, 1, 1024, 1024, 64, 8), (True, 4, 256, 1152, 33, 8),
    (True, 2, 128, 640, 24, 12)])
def test_direct_second_product_in_parts(mx, T, d, f, E, k, same):
    """Up to 4 tokens, narrow y and many items of the reduction: the direct
    form leaves parts for the sum.  same: all tokens choose the same experts,
    fewer than the parts were counted for."""
    c = L.Case(T, d, f, E, k, mx=mx, bias=not same, add=T > 1, seed=T + d)
    if same:
        c.logits = I.make_tensor((1, E), seed=5, dtype=torch.float32,
                                 device="cuda:0").repeat(T, 1)
    S = (T * k * f * 4 + 255) // 256 * 256
    z = (T * E * 4 + 255) // 256 * 256
    parts = (c.ws.numel() - S - z) // (T * d * 4)
    assert parts >= 2                   # what the test is for
    c.run()
    L.check(c)
    if c.y_add is not None:             # the sum may go into y itself
        want = c.y.clone()
        y = c.y_add.clone()
        c.run(y=y, y_add=y)
        assert torch.equal(y, want)


@gpu
@pytest.mark.parametrize("T,mx", [(1, False), (2, False), (12, False),
                                  (1, True), (2, True), (12, True)])
def test_second_product_past_32_bit_offsets(T, mx):
    """w2 past 4 GiB (w_gu past 8), the first and the last expert; one or two
    of them are few enough values for the direct second product, 12 tokens
    take the batch form."""
    dev = torch.device("cuda:0")
    d = f = 4096
    E = 330 if mx else 160
    c = L.Case(1, 128, 128, 1, 1, mx=mx)
    c.T, c.d, c.f, c.E, c.k = T, d, f, E, 1
    c.x = I.make_tensor((T, d), seed=1, device=dev)
    c.y_add = None
    for i, (rows, cols) in enumerate(((2 * f, d), (d, f))):
        w = torch.zeros(E, rows, cols, dtype=U8 if mx else BF, device=dev)
        assert w.numel() * w.element_size() > 1 << 32
        s = torch.zeros(E, rows, cols // 32, dtype=U8, device=dev)
        for e in (0, E - 2, E - 1):
            v = I.make_tensor((rows, cols), seed=e + 7 * i, scale=0.02,
                              device=dev)
            if mx:
                moe.moe_mxfp8_quantize(v, 0, None, w[e], s[e])
            else:
                w[e] = v
        c.w[i], c.s[i] = w, s if mx else None
    c.logits = torch.full((T, E), -5.0, device=dev)
    hot = torch.tensor([E - 1, 0, E - 2], device=dev)
    t = torch.arange(T, device=dev)
    c.logits[t, hot[t % 3]] = 1.0
    c.ws = torch.empty(moe.moe_workspace_bytes(
        moe.MOE_ENTRY_LAYER_FWD, c.prec, T, E, 1, d, f), dtype=U8, device=dev)
    c.y = torch.empty(T, d, dtype=BF, device=dev)
    c.idx = torch.empty(T, 1, dtype=torch.int32, device=dev)
    c.p = torch.empty(T, 1, device=dev)
    c.run()
    L.check(c)
