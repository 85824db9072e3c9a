"""Argument checks of the norm and dropout entries that need no GPU: fake
device pointers are safe because every call here is refused before a launch;
the binding refuses tensors that are not on a GPU."""

import pytest
import torch

from mixture_experts_expert_top_amd import moe

L = moe.lib
OK, INVALID, UNSUP, WS = 0, 1, 2, 3
NAN = float("nan")


def at(i):
    """The i-th fake device address, 1 GiB apart."""
    return (i + 1) << 30


def _fwd(kind=0, x=at(0), fp32=0, gamma=at(1), beta=None, eps=1e-5, T=4,
         d=64, y=at(2), mean=at(3), rstd=at(4)):
    return L.moe_norm_fwd(kind, x, fp32, gamma, beta, eps, T, d, y, mean,
                          rstd, None)


@pytest.mark.parametrize("kw,want", [
    (dict(kind=2), INVALID), (dict(kind=-1), INVALID), (dict(T=0), INVALID),
    (dict(T=-3), INVALID), (dict(d=0), INVALID), (dict(d=12), INVALID),
    (dict(d=16392), UNSUP), (dict(T=1 << 40), UNSUP),
    (dict(eps=-1e-5), INVALID), (dict(eps=NAN), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID),
    (dict(gamma=None), INVALID), (dict(y=None), INVALID),
    (dict(x=at(0) + 8), INVALID), (dict(mean=at(3) + 4), INVALID),
    (dict(kind=1, beta=at(5)), INVALID), (dict(y=at(0)), INVALID),
    (dict(y=at(0) + 496), INVALID), (dict(rstd=at(3)), INVALID),
    (dict(fp32=1, y=at(0) + 1008), INVALID), (dict(rstd=at(1)), INVALID)])
def test_norm_fwd_refusals(kw, want):
    assert _fwd(**kw) == want
    assert L.moe_last_error()


def _bwd(kind=0, dy=at(0), x=at(1), fp32=0, gamma=at(2), mean=at(3),
         rstd=at(4), dres=at(5), T=4, d=64, dx=at(6), dgamma=at(7),
         dbeta=at(8), ws=at(9), nbytes=None):
    if nbytes is None:
        nbytes = L.moe_workspace_bytes(moe.MOE_ENTRY_NORM_BWD, 0, max(T, 1),
                                       1, 1, d, 0)
    return L.moe_norm_bwd(kind, dy, x, fp32, gamma, mean, rstd, dres, T, d,
                          dx, dgamma, dbeta, ws, nbytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), INVALID), (dict(d=20), INVALID), (dict(d=16392), UNSUP),
    (dict(mean=None), INVALID), (dict(kind=1), INVALID),
    (dict(kind=1, mean=None), INVALID), (dict(rstd=None), INVALID),
    (dict(dy=None), INVALID), (dict(dx=None), INVALID),
    (dict(nbytes=1), WS), (dict(ws=None), INVALID),
    (dict(ws=at(9) + 4), INVALID), (dict(dx=at(1)), INVALID),
    (dict(dx=at(0)), INVALID), (dict(dx=at(5) + 16), INVALID),
    (dict(dgamma=at(2)), INVALID), (dict(dbeta=at(7)), INVALID),
    (dict(ws=at(1)), INVALID), (dict(ws=at(6)), INVALID)])
def test_norm_bwd_refusals(kw, want):
    assert _bwd(**kw) == want
    assert L.moe_last_error()


def test_norm_workspace_sizes():
    ws = lambda T, d: L.moe_workspace_bytes(  # noqa: E731
        moe.MOE_ENTRY_NORM_BWD, 0, T, 1, 1, d, 0)
    assert ws(1, 8) == 2 * 8 * 4
    assert ws(1, 16384) == 2 * 16384 * 4
    assert ws(0, 8) == 0 and ws(4, 0) == 0 and ws(4, 16392) == 0
    # bounded however many rows there are
    assert ws(1 << 20, 4096) == ws(1 << 30, 4096)


def _drop(x=at(0), xf=0, res=at(1), of=0, n=64, p=0.1, rng=at(2), delta=0,
          out=at(3)):
    return L.moe_dropout(x, xf, res, of, n, p, rng, delta, out, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), INVALID), (dict(n=-1), INVALID), (dict(n=1 << 41), UNSUP),
    (dict(p=-0.1), INVALID), (dict(p=1.1), INVALID), (dict(p=NAN), INVALID),
    (dict(x=None), INVALID), (dict(rng=None), INVALID),
    (dict(out=None), INVALID), (dict(x=at(0) + 2), INVALID),
    (dict(out=at(0) + 16), INVALID), (dict(out=at(1) - 16), INVALID),
    (dict(rng=at(3) + 112), INVALID),
    (dict(out=at(0), of=1), INVALID), (dict(out=at(0), xf=1), INVALID), (dict(out=at(2)), INVALID)])
def test_dropout_refusals(kw, want):
    assert _drop(**kw) == want
    assert L.moe_last_error()


def test_binding_refuses_cpu_tensors_and_wrong_types():
    T, d = 4, 64
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    f32 = lambda *s: torch.zeros(*s)  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_norm_fwd(0, bf(T, d), f32(d), f32(d), 1e-5, bf(T, d))
    with pytest.raises(TypeError):
        moe.moe_norm_fwd(0, bf(T, d).half(), f32(d), None, 1e-5, bf(T, d))
    with pytest.raises(TypeError):
        moe.moe_norm_fwd(0, bf(T, d), bf(d), None, 1e-5, bf(T, d))
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_norm_fwd(0, bf(d, T).t(), f32(d), None, 1e-5, bf(T, d))
    with pytest.raises(ValueError, match="shape"):
        moe.moe_norm_bwd(0, bf(T, d), bf(T, d), f32(d), f32(T), f32(T), None,
                         bf(T + 1, d), None, None, None)
    rng = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_dropout(bf(T, d), None, 0.1, rng, 0, bf(T, d))
    with pytest.raises(TypeError):
        moe.moe_dropout(bf(T, d), f32(T, d), 0.1, rng, 0, bf(T, d))
    with pytest.raises(TypeError):
        moe.moe_dropout(bf(T, d), None, 0.1, rng.float(), 0, bf(T, d))


def _ffn(act=0, x=at(0), w_gu=at(1), w2=at(2), y_add=None, T=4, d=64, f=128,
         ab=at(3), s=at(4), y=at(5), ws=at(6), nbytes=None):
    if nbytes is None:
        nbytes = max(L.moe_workspace_bytes(moe.MOE_ENTRY_FFN_FWD, 0,
                                           max(T, 1), 1, 1, d, f), 1 << 20)
    return L.moe_ffn_fwd(act, x, w_gu, w2, y_add, T, d, f, ab, s, y, ws,
                         nbytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(act=2), INVALID), (dict(T=0), INVALID), (dict(d=12), INVALID),
    (dict(f=12), INVALID), (dict(f=0), INVALID), (dict(T=1 << 30), UNSUP),
    (dict(d=1 << 16, f=1 << 14), UNSUP), (dict(d=(1 << 21) + 8), UNSUP),
    (dict(d=8, f=(1 << 21) + 8), UNSUP), (dict(d=1 << 40, f=1 << 40), UNSUP),
    (dict(x=None), INVALID), (dict(w_gu=None), INVALID),
    (dict(w2=None), INVALID), (dict(y=None), INVALID),
    (dict(y=at(5) + 8), INVALID), (dict(ws=None), INVALID),
    (dict(nbytes=16), WS), (dict(y=at(0)), INVALID),
    (dict(y_add=at(5) + 16), INVALID), (dict(ab=at(1) + 64), INVALID),
    (dict(s=at(3) + 512), INVALID), (dict(ws=at(4)), INVALID)])
def test_ffn_fwd_refusals(kw, want):
    assert _ffn(**kw) == want
    assert L.moe_last_error()


def _ffn_b(act=0, dy=at(0), x=at(1), w_gu=at(2), w2=at(3), ab=at(4), s=at(5),
           dx_add=None, T=4, d=64, f=128, dx=at(6), dw_gu=at(7), dw2=at(8),
           ws=at(9), nbytes=None):
    if nbytes is None:
        nbytes = L.moe_workspace_bytes(moe.MOE_ENTRY_FFN_BWD, 0, max(T, 1),
                                       1, 1, d, f)
    return L.moe_ffn_bwd(act, dy, x, w_gu, w2, ab, s, dx_add, T, d, f, dx,
                         dw_gu, dw2, ws, nbytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(act=-1), INVALID), (dict(T=0), INVALID), (dict(d=20), INVALID),
    (dict(f=4), INVALID), (dict(dy=None), INVALID),
    (dict(dx=None, dw_gu=None, dw2=None), INVALID),
    (dict(s=None), INVALID), (dict(x=None), INVALID),
    (dict(dx=None, dx_add=at(10)), INVALID), (dict(ab=None), INVALID),
    (dict(nbytes=16), WS), (dict(dx=at(0)), INVALID),
    (dict(dx_add=at(6) + 32), INVALID), (dict(dw2=at(3)), INVALID),
    (dict(dw_gu=at(8)), INVALID), (dict(ws=at(5)), INVALID)])
def test_ffn_bwd_refusals(kw, want):
    assert _ffn_b(**kw) == want
    assert L.moe_last_error()


def test_ffn_workspace_sizes():
    for e in (moe.MOE_ENTRY_FFN_FWD, moe.MOE_ENTRY_FFN_BWD):
        ws = lambda T, d, f: L.moe_workspace_bytes(  # noqa: E731
            e, 0, T, 1, 1, d, f)
        rows = 2 if e == moe.MOE_ENTRY_FFN_FWD else 4
        assert ws(1, 64, 128) >= rows * 128
        assert ws(8192, 4096, 14336) >= rows * 8192 * 14336
        assert ws(0, 64, 64) == 0 and ws(4, 12, 64) == 0
        assert ws(4, 64, 12) == 0 and ws(4, 1 << 16, 1 << 14) == 0
        assert ws(1 << 30, 64, 64) == 0


def test_ffn_binding_refuses_cpu_tensors_and_wrong_shapes():
    T, d, f = 4, 64, 128
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_ffn_fwd(0, bf(T, d), bf(2 * f, d), bf(d, f), None, None,
                        None, bf(T, d), ws)
    with pytest.raises(ValueError, match="shape"):
        moe.moe_ffn_fwd(0, bf(T, d), bf(f, d), bf(d, f), None, None, None,
                        bf(T, d), ws)
    with pytest.raises(TypeError):
        moe.moe_ffn_bwd(0, bf(T, d), bf(T, d), bf(2 * f, d), bf(d, f),
                        bf(T, 2 * f).float(), bf(T, f), None, bf(T, d), None,
                        None, ws)
