"""Host-side checks of moe_layer_fwd: what it refuses before anything is
launched (fake device addresses), and its workspace."""

import pytest

from mixture_experts_expert_top_amd import moe

L = moe.lib
INVALID, UNSUP, WS = 1, 2, 3
BASE = 1 << 32
GOOD = dict(prec=0, x=BASE, w_g=BASE + (1 << 20), bias=None, logits=None, T=4,
            d=256, f=128, E=8, k=2, renorm=1, w_gu=BASE + (2 << 20),
            w_gu_s=None, w2=BASE + (6 << 20), w2_s=None, y_add=None,
            idx=BASE + (9 << 20), w=BASE + (10 << 20), y=BASE + (11 << 20),
            ws=BASE + (12 << 20), nbytes=1 << 20)


def call(**kw):
    a = {**GOOD, **kw}
    st = L.moe_layer_fwd(*[a[n] for n in GOOD], None)
    return st, L.moe_last_error()


@pytest.mark.parametrize("kw,want,word", [
    (dict(prec=2), UNSUP, b"MXFP8"), (dict(prec=7), INVALID, b"precision"),
    (dict(x=None), INVALID, b"x"), (dict(x=BASE + 8), INVALID, b"x"),
    (dict(w_g=None), INVALID, b"either"),
    (dict(logits=BASE + (13 << 20)), INVALID, b"either"),
    (dict(w_g=None, logits=BASE + (13 << 20), bias=BASE + (14 << 20)),
     INVALID, b"bias"),
    (dict(w_g=BASE + 4), INVALID, b"w_g"),
    (dict(bias=BASE + 4), INVALID, b"bias"),
    (dict(w_gu=None), INVALID, b"w_gu"), (dict(w2=None), INVALID, b"w2"),
    (dict(w2=BASE + 2), INVALID, b"w2"),
    (dict(w_gu_s=BASE + (13 << 20)), INVALID, b"scales"),
    (dict(prec=1), INVALID, b"scales"),
    (dict(prec=1, w_gu_s=BASE + (13 << 20)), INVALID, b"w2_scales"),
    (dict(idx=None), INVALID, b"topk_idx"), (dict(w=None), INVALID, b"topk_w"),
    (dict(y=None), INVALID, b"y"), (dict(y=BASE + 12), INVALID, b"y"),
    (dict(y_add=BASE + 12), INVALID, b"y_add"),
    (dict(T=0), INVALID, b"T"), (dict(T=65), UNSUP, b"64"),
    (dict(E=0), INVALID, b"E"), (dict(E=1025), INVALID, b"E"),
    (dict(k=0), INVALID, b"k"), (dict(k=9), INVALID, b"k"),
    (dict(E=64, k=33), UNSUP, b"k"),
    (dict(d=0), INVALID, b"d"), (dict(d=12), INVALID, b"d"),
    (dict(f=4), INVALID, b"f"), (dict(f=129), INVALID, b"f"),
    (dict(d=1 << 16, f=1 << 15), UNSUP, b"4 GiB"),
    (dict(d=1 << 21, f=8), UNSUP, b"2^20"),
    (dict(prec=1, w_gu_s=BASE + (13 << 20), w2_s=BASE + (14 << 20), d=160),
     INVALID, b"128"),
    (dict(ws=None), INVALID, b"workspace"),
    (dict(ws=BASE + (12 << 20) + 8), INVALID, b"workspace"),
    (dict(nbytes=100), WS, b"workspace"),
    (dict(y=BASE), INVALID, b"overlaps"),
    (dict(y=BASE + (9 << 20)), INVALID, b"overlaps"),
    (dict(y_add=BASE + (11 << 20) + 16), INVALID, b"overlaps"),
    (dict(ws=BASE + (2 << 20) + 1024), INVALID, b"overlaps"),
    (dict(idx=BASE + (6 << 20)), INVALID, b"overlaps"),
    (dict(w=BASE + (9 << 20) + 16), INVALID, b"overlaps"),
    (dict(ws=BASE + (11 << 20) + 1024), INVALID, b"overlaps")])
def test_refuses(kw, want, word):
    st, msg = call(**kw)
    assert st == want, msg
    assert word in msg, msg


def test_workspace():
    """S, in bf16 for every slot; 0 for what no call takes."""
    W = lambda **kw: moe.moe_workspace_bytes(*{**dict(  # noqa: E731
        entry=moe.MOE_ENTRY_LAYER_FWD, prec=0, T=4, E=8, k=2, d=256, f=128),
        **kw}.values())
    assert W() >= 4 * 2 * 128 * 2
    assert W(T=64) >= 64 * 2 * 128 * 2
    for kw in (dict(T=65), dict(T=0), dict(k=9), dict(E=0), dict(E=2000),
               dict(E=64, k=33), dict(d=0), dict(f=0), dict(prec=9),
               dict(d=(1 << 20) + 8), dict(f=1 << 40)):
        assert W(**kw) == 0, kw


@pytest.mark.parametrize("kw", [
    dict(prec=2), dict(d=12), dict(f=12), dict(d=4), dict(f=4),
    dict(prec=1, d=160), dict(prec=1, f=160), dict(prec=1, d=64),
    dict(d=1 << 16, f=1 << 15), dict(prec=1, d=1 << 15, f=1 << 16),
    dict(T=64, E=64, k=32, d=8, f=1 << 19), dict(T=64, E=64, k=32, d=8,
                                                 f=1 << 20)])
def test_no_workspace_for_what_the_call_refuses(kw):
    """moe_workspace_bytes gives 0 where moe_layer_fwd refuses the same
    precision and sizes whatever workspace it is given."""
    a = {**dict(prec=0, T=4, E=8, k=2, d=256, f=128), **kw}
    n = moe.moe_workspace_bytes(moe.MOE_ENTRY_LAYER_FWD, a["prec"], a["T"],
                                a["E"], a["k"], a["d"], a["f"])
    assert n == 0
    # tensors far apart, so that nothing but the sizes can be at fault
    far = {n: (i + 1) << 44 for i, n in enumerate(
        ("x", "w_g", "w_gu", "w2", "idx", "w", "y", "ws"))}
    if a["prec"] != 0:
        far.update(w_gu_s=20 << 44, w2_s=21 << 44)
    st, msg = call(**{**far, **a}, nbytes=1 << 62)
    assert st in (INVALID, UNSUP), msg
    assert b"workspace" not in msg and b"overlap" not in msg


@pytest.mark.parametrize("kw", [
    dict(), dict(prec=1), dict(d=8, f=8, T=1, E=1, k=1),
    dict(T=64, E=64, k=32, d=8, f=524280), dict(d=32768, f=32760),
    dict(prec=1, d=32768, f=32640)])
def test_workspace_up_to_the_limits(kw):
    """Sizes next to the refused ones have a workspace, and pass the call's
    checks as far as the workspace's own."""
    a = {**dict(prec=0, T=4, E=8, k=2, d=256, f=128), **kw}
    n = moe.moe_workspace_bytes(moe.MOE_ENTRY_LAYER_FWD, a["prec"], a["T"],
                                a["E"], a["k"], a["d"], a["f"])
    assert n > 0
    far = {n: (i + 1) << 44 for i, n in enumerate(
        ("x", "w_g", "w_gu", "w2", "idx", "w", "y", "ws"))}
    if a["prec"] != 0:
        far.update(w_gu_s=20 << 44, w2_s=21 << 44)
    st, msg = call(**{**far, **a}, nbytes=n - 1)
    assert st == WS, msg


@pytest.mark.parametrize("kw", [
    dict(prec=2), dict(d=12), dict(prec=1, f=160), dict(T=65), dict(T=0),
    dict(k=9), dict(d=1 << 16, f=1 << 15)])
def test_moe_decode_refuses_when_it_is_made(kw):
    """Before any buffer is, with the sizes in the message."""
    from mixture_experts_expert_top_amd.layer import MoEDecode
    a = {**dict(T=4, d=256, f=128, E=8, k=2, prec=0), **kw}
    with pytest.raises(ValueError, match=f"d={a['d']}.*prec={a['prec']}"):
        MoEDecode(**a)


def test_quantize_runs_on_its_weights_device(monkeypatch):
    """The quantizer launches on the current device's stream, so that device
    is made the weight's; a weight in host memory is refused."""
    import contextlib

    import torch

    from mixture_experts_expert_top_amd.layer import MoEDecode
    made, current = [], []

    @contextlib.contextmanager
    def device(d):
        current.append(d)
        yield
        current.pop()
    monkeypatch.setattr(moe, "moe_mxfp8_quantize",
                        lambda *a, **k: made.append(list(current)))
    w = torch.zeros(3, 32, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        MoEDecode.quantize(w)
    assert not made
    monkeypatch.setattr(torch.cuda, "device", device)
    codes, scales = MoEDecode.quantize(w)
    assert made == [[w.device]] * 3
    assert codes.shape == w.shape and scales.shape == (3, 32, 4)
