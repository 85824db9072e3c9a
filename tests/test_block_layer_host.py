"""MoEBlock's own argument checks, without a GPU: the block and its path hold
CPU tensors and the library's calls are replaced by a list of their names, so
what is tested is what the block lets through to them."""

import contextlib

import pytest
import torch

from mixture_experts_expert_top_amd import layer, moe

BF, F32 = torch.bfloat16, torch.float32
T, D, F, E, FS = 16, 64, 64, 4, 64
LAUNCHES = [n for n in moe.EXPORTED if hasattr(moe, n) and n not in (
    "moe_workspace_bytes", "moe_dp_tiles", "moe_row_planes",
    "moe_mxfp8_padded_rows")]


@pytest.fixture
def calls(monkeypatch):
    """Names of the library calls made, in order."""
    made = []
    for name in LAUNCHES:
        monkeypatch.setattr(moe, name,
                            lambda *a, _n=name, **k: made.append(_n))
    monkeypatch.setattr(torch.cuda, "device",
                        lambda d: contextlib.nullcontext())
    return made


def _block(k=2, f_shared=FS, stream_fp32=False):
    path = layer.MoEPath(T, D, F, E, k, device="cpu")
    return layer.MoEBlock(path, f_shared=f_shared, stream_fp32=stream_fp32)


def _weights(blk):
    fs = blk.f_shared
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt)  # noqa: E731
    return dict(gamma=z(D, dt=F32), w_gu=z(E, 2 * F, D), w2=z(E, D, F),
                sw_gu=z(2 * fs, D) if fs else None,
                sw2=z(D, fs) if fs else None)


def _fwd(blk, x, **kw):
    return blk.forward(x, w_g=torch.zeros(E, D, dtype=BF),
                       **{**_weights(blk), **kw})


def _bwd(blk, dy, **kw):
    return blk.backward(dy, **{**_weights(blk), **kw})


def _rows(blk):
    return torch.zeros(T, D, dtype=blk.stream_dtype)


@pytest.mark.parametrize("what", ["dz", "path.dx", "path.dout_perm"])
def test_dy_in_a_buffer_that_backward_replaces_is_refused(calls, what):
    """dy is read twice: by the dropout, and at the end as the residual's
    gradient.  What lies in between may not replace it."""
    blk = _block(k=1)
    _fwd(blk, _rows(blk))
    _bwd(blk, _rows(blk))
    dy = blk.dz if what == "dz" else getattr(blk.path, what[5:])
    assert dy.shape == (T, D) and dy.dtype == blk.stream_dtype
    _fwd(blk, _rows(blk))
    calls.clear()
    with pytest.raises(ValueError, match="dy overlaps"):
        _bwd(blk, dy)
    assert calls == []


@pytest.mark.parametrize("what", ["dz", "path.dx", "dx"])
def test_x_in_a_buffer_that_backward_replaces_is_refused(calls, what):
    """The forward's x is read again by the norm's gradient."""
    blk = _block()
    _fwd(blk, _rows(blk))
    _bwd(blk, _rows(blk))
    x = blk.path.dx if what == "path.dx" else getattr(blk, what)
    _fwd(blk, x)
    calls.clear()
    with pytest.raises(ValueError, match="x overlaps"):
        _bwd(blk, _rows(blk))
    assert calls == []


@pytest.mark.parametrize("what", ["path.y", "path.x_perm", "s", "n"])
def test_x_in_a_buffer_that_forward_replaces_is_refused(calls, what):
    """x is read by the norm and, at the end, as the residual."""
    blk = _block(k=1)
    x = getattr(blk.path, what[5:]) if "." in what else getattr(blk, what)
    assert x.shape == (T, D)
    with pytest.raises(ValueError, match="x overlaps"):
        _fwd(blk, x)
    assert calls == []


def test_dy_in_the_blocks_results_is_taken(calls):
    """dx may be the dres of the norm's gradient, and nothing of the backward
    writes y: stacked uses of one block pass either."""
    blk = _block()
    _fwd(blk, _rows(blk))
    _bwd(blk, blk.y)
    dx = _bwd(blk, _rows(blk))
    assert _bwd(blk, dx) is dx
    # an fp32 stream's gradient has no buffer of its type between
    blk = _block(stream_fp32=True, f_shared=0)
    _fwd(blk, _rows(blk))
    assert _bwd(blk, _rows(blk)) is blk.dx


@pytest.mark.parametrize("at", ["moe_permute", "moe_ffn_fwd", "moe_dropout"])
def test_no_backward_after_a_forward_that_failed(calls, monkeypatch, at):
    """A forward that ends half way has replaced n and the norm's statistics:
    the backward of the forward before it is gone too."""
    blk = _block()
    _fwd(blk, _rows(blk))

    def fail(*a, **k):
        raise moe.MoeError(at, 1, "MOE_ERR_INVALID_ARG", "refused")

    with monkeypatch.context() as m:
        m.setattr(moe, at, fail)
        with pytest.raises(moe.MoeError):
            _fwd(blk, _rows(blk))
    with pytest.raises(ValueError, match="backward needs a forward"):
        _bwd(blk, _rows(blk))
    _fwd(blk, _rows(blk))
    _bwd(blk, _rows(blk))


def test_a_refused_forward_leaves_the_one_before(calls):
    blk = _block()
    _fwd(blk, _rows(blk))
    for kw in (dict(p=0.5), dict(sw2=None)):
        with pytest.raises(ValueError):
            _fwd(blk, _rows(blk), **kw)
    with pytest.raises(ValueError):
        _fwd(blk, blk.path.y)
    _bwd(blk, _rows(blk))


def test_no_backward_after_the_path_ran_for_another(calls):
    """The path keeps one forward: two blocks around one path, or a call of
    the path itself, replace what the first block's backward would read."""
    blk = _block()
    other = layer.MoEBlock(blk.path)
    _fwd(blk, _rows(blk))
    _fwd(other, _rows(blk))
    calls.clear()
    with pytest.raises(ValueError, match="another forward"):
        _bwd(blk, _rows(blk))
    assert calls == []
    _bwd(other, _rows(blk))
    w = _weights(blk)
    x = torch.zeros(T, D, dtype=BF)
    for use in (lambda: blk.path.forward(x, w["w_gu"], w["w2"], w_g=x[:E]),
                lambda: blk.path.route(x, x[:E])):
        _fwd(blk, _rows(blk))
        use()
        with pytest.raises(ValueError, match="another forward"):
            _bwd(blk, _rows(blk))
    _fwd(blk, _rows(blk))
    _bwd(blk, _rows(blk))
    _bwd(blk, _rows(blk))


def test_calls_run_on_the_paths_device(calls, monkeypatch):
    """The path's calls take the current device's stream, the others their
    tensors' device: both are the path's device while the block runs."""
    on = []

    @contextlib.contextmanager
    def device(d):
        on.append(d)
        yield
        on.pop()

    where = {}
    for name in LAUNCHES:
        monkeypatch.setattr(moe, name, lambda *a, _n=name, **k:
                            where.setdefault(_n, list(on)))
    monkeypatch.setattr(torch.cuda, "device", device)
    blk = _block()
    _fwd(blk, _rows(blk))
    _bwd(blk, _rows(blk))
    assert {"moe_norm_fwd", "moe_permute", "moe_grouped_mlp_bwd",
            "moe_ffn_bwd", "moe_norm_bwd"} <= set(where)
    assert all(w == [torch.device("cpu")] for w in where.values()), where
    assert on == []


@pytest.mark.parametrize("missing", ["sw_gu", "sw2"])
def test_backward_needs_the_feed_forward_weights(calls, missing):
    """Refused before the path's backward has run, as in the forward."""
    blk = _block()
    _fwd(blk, _rows(blk))
    calls.clear()
    with pytest.raises(ValueError, match="sw_gu and sw2"):
        _bwd(blk, _rows(blk), **{missing: None})
    assert calls == []
