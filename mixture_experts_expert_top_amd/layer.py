"""One MoE expert-MLP layer driven through the C-ABI.

``MoEPath`` owns the device buffers of one problem size (allocated once
with torch, reused every step) and issues the library calls in order:

  forward : moe_router_logits -> moe_route -> moe_permute
            -> moe_grouped_mlp_fwd -> moe_unpermute
  backward: moe_permute_rows (dY) -> moe_grouped_mlp_bwd
            -> moe_router_backward (when the forward computed the router
               scores: dlogits with the balancing term, dW_g, db)
            -> moe_unpermute (dX, with the router's share added before its
               one rounding)

With a ``timers`` object (see ``StageTimers``) the GEMMs are issued
through the per-GEMM stage entry points instead of the fused ones, with
HIP events recorded around each stage on the stream it runs on.

``MoEPathMX`` is the same layer with MXFP8 GEMM operands: x is quantized
along d before the permutation, the weights along their rows once per step
(forward) and along their columns inside the backward, S and dAB inside the
GEMM epilogues that produce them (both along their GEMM axis and along each
expert's tokens, the latter for the weight gradients), and dO and Xp along
each expert's tokens in the backward.  No bf16 copy of S or dAB is kept.
With ``act_fp4`` the GEMMs stay MXFP8 but x is quantized to MXFP4 along d
(the dispatched payload, half the bytes), the gate_up GEMM widens it to
E4M3 on its way to LDS, and the backward converts that payload to MXFP4
blocks along each expert's tokens for the dW_gu GEMM (widened the same way)
instead of re-permuting bf16 x.

``MoEBlock`` is the residual block around either of them: the norm in
front, optionally a dense gated feed-forward block that every token passes
beside its routed experts, and the residual sum with dropout behind.

``MoEDecode`` is the layer for the few tokens of generation, one call without
a dispatch plan or a backward, in a block as the other two are; ``AdamW`` is
the step that uses the gradients that they leave.

No arithmetic happens here: every step runs in the library's kernels.
"""

import contextlib
import functools

import torch

from . import moe
from .moe import (MOE_ACT_SILU, MOE_BF16, MOE_ENTRY_FFN_BWD,
                  MOE_ENTRY_FFN_FWD, MOE_ENTRY_GRAD_NORM, MOE_ENTRY_LAYER_FWD,
                  MOE_ENTRY_MLP_BWD, MOE_ENTRY_MLP_FWD, MOE_ENTRY_NORM_BWD,
                  MOE_ENTRY_PERMUTE, MOE_ENTRY_ROUTER_BWD, MOE_MOMENTS_FP32,
                  MOE_MOMENTS_FP8, MOE_MXFP4, MOE_MXFP8, MOE_NORM_LAYER,
                  MOE_NORM_RMS)


class StageTimers:
    """Pairs of HIP events recorded around named stages on the current
    stream; ``mean_ms()`` gives each stage's average duration."""

    def __init__(self):
        self.events = {}

    @contextlib.contextmanager
    def around(self, name):
        a = torch.cuda.Event(enable_timing=True)
        b = torch.cuda.Event(enable_timing=True)
        a.record()
        yield
        b.record()
        self.events.setdefault(name, []).append((a, b))

    def mean_ms(self):
        return {n: sum(a.elapsed_time(b) for a, b in ev) / len(ev)
                for n, ev in self.events.items()}

    def counts(self):
        return {n: len(ev) for n, ev in self.events.items()}


def _around(timers, name):
    return timers.around(name) if timers is not None else \
        contextlib.nullcontext()


class MoEPath:
    def __init__(self, T, d, f, E, k, renorm=True, prec=MOE_BF16,
                 device="cuda", y_fp32=False, aux_coef=0.01):
        if prec != MOE_BF16:
            raise NotImplementedError("use MoEPathMX for the MXFP8 path")
        self.T, self.d, self.f, self.E, self.k = T, d, f, E, k
        self.renorm = renorm
        self.aux_coef = aux_coef
        self._router = None
        self._forwards = 0      # tells whose forward the buffers hold
        self.prec = prec
        Tk = T * k
        dev = torch.device(device)
        i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
        z = lambda *s, dt: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        self.logits = z(T, E, dt=f32)
        self.topk_idx = z(T, k, dt=i32)
        self.topk_w = z(T, k, dt=f32)
        self.counts = z(E, dt=i32)
        self.offsets = z(E + 1, dt=i32)
        self.pos = z(T, k, dt=i32)
        self.src = z(Tk, dt=i32)
        self.w_perm = z(Tk, dt=f32)
        self.x_perm = z(Tk, d, dt=bf)
        self.ab = z(Tk, 2 * f, dt=bf)
        self.s = z(Tk, f, dt=bf)
        self.o = z(moe.row_planes(f), Tk, d, dt=f32)
        self.y = z(T, d, dt=f32 if y_fp32 else bf)
        ws_p = moe.moe_workspace_bytes(MOE_ENTRY_PERMUTE, prec, T, E, k, d, f)
        self.ws_permute = z(max(ws_p, 16), dt=torch.uint8)
        self._bwd_ready = False

    def _alloc_bwd(self):
        T, d, f, E, k = self.T, self.d, self.f, self.E, self.k
        Tk = T * k
        dev = self.x_perm.device
        bf = torch.bfloat16
        self.dout_perm = torch.empty(Tk, d, dtype=bf, device=dev)
        self.dx_perm = torch.empty(moe.row_planes(f), Tk, d,
                                   dtype=torch.float32, device=dev)
        self.dw_gu = torch.empty(E, 2 * f, d, dtype=bf, device=dev)
        self.dw2 = torch.empty(E, d, f, dtype=bf, device=dev)
        self.dp = torch.empty(T, k, dtype=torch.float32, device=dev)
        self.dx = torch.empty(T, d, dtype=bf, device=dev)
        self.dab = torch.empty(Tk, 2 * f, dtype=bf, device=dev)
        self.dp_part = torch.empty(Tk, moe.moe_dp_tiles(f),
                                   dtype=torch.float32, device=dev)
        ws_b = moe.moe_workspace_bytes(MOE_ENTRY_MLP_BWD, self.prec, T, E, k,
                                       d, f)
        self.ws_bwd = torch.empty(max(ws_b, 16), dtype=torch.uint8,
                                  device=dev)
        # router backward
        self.dlogits = torch.empty(T, E, dtype=torch.float32, device=dev)
        self.dw_g = torch.empty(E, d, dtype=torch.float32, device=dev)
        self.db = torch.empty(E, dtype=torch.float32, device=dev)
        self.aux_loss = torch.empty(1, dtype=torch.float32, device=dev)
        ws_r = moe.moe_workspace_bytes(MOE_ENTRY_ROUTER_BWD, MOE_BF16, T, E,
                                       k, d, f)
        self.ws_router = torch.empty(max(ws_r, 16), dtype=torch.uint8,
                                     device=dev)
        self._bwd_ready = True

    def gradients(self, w_gu, w2, w_g=None, bias=None):
        """(weight, gradient[, weight decay]) of the weights that a backward
        with them leaves gradients for, as ``AdamW`` takes them."""
        if not self._bwd_ready:
            self._alloc_bwd()
        out = [(w_gu, self.dw_gu), (w2, self.dw2)]
        if w_g is not None:
            out.append((w_g, self.dw_g))
        if bias is not None:
            out.append((bias, self.db, 0.0))
        return out

    # ------------------------------------------------------------------
    def route(self, x=None, w_g=None, bias=None, logits=None, timers=None):
        self._forwards += 1
        if logits is None:
            with _around(timers, "router_logits"):
                moe.moe_router_logits(x, w_g, bias, self.logits)
            logits = self.logits
            self._router = (x, w_g, bias)
        else:
            self._router = None
        self._logits_used = logits
        with _around(timers, "route"):
            moe.moe_route(logits, self.k, self.renorm, self.topk_idx,
                          self.topk_w)

    def forward(self, x, w_gu, w2, w_g=None, bias=None, logits=None,
                timers=None):
        self.route(x, w_g, bias, logits, timers)
        with _around(timers, "permute"):
            moe.moe_permute(self.prec, self.topk_idx, self.topk_w, self.E, x,
                            None, self.counts, self.offsets, self.pos,
                            self.src, self.w_perm, self.x_perm, None,
                            self.ws_permute)
        if timers is None:
            moe.moe_grouped_mlp_fwd(self.prec, self.x_perm, None,
                                    self.offsets, w_gu, None, w2, None,
                                    self.w_perm, self.ab, self.s, self.o)
        else:
            with timers.around("gate_up_swiglu_fwd"):
                moe.moe_gate_up_swiglu_fwd(self.x_perm, self.offsets, w_gu,
                                           self.w_perm, self.ab, self.s)
            with timers.around("down_fwd"):
                moe.moe_down_fwd(self.s, self.offsets, w2, self.o)
        with _around(timers, "unpermute_y"):
            moe.moe_unpermute(self.o, self.pos, None, self.y)
        return self.y

    def backward(self, dy, w_gu, w2, timers=None):
        if not self._bwd_ready:
            self._alloc_bwd()
        with _around(timers, "permute_dy"):
            moe.moe_permute_rows(self.prec, self.pos, dy, None,
                                 self.dout_perm, None)
        if timers is None:
            moe.moe_grouped_mlp_bwd(self.prec, self.dout_perm, self.x_perm,
                                    self.offsets, self.pos, w_gu, w2, self.ab,
                                    self.s, self.w_perm, self.dx_perm,
                                    self.dw_gu, self.dw2, self.dp,
                                    self.ws_bwd)
        else:
            # the same kernels in the same order as moe_grouped_mlp_bwd
            with timers.around("down_swiglu_bwd"):
                moe.moe_down_swiglu_bwd(self.dout_perm, self.offsets, w2,
                                        self.ab, self.w_perm, self.dab,
                                        self.dp_part)
            with timers.around("dp_reduce"):
                moe.moe_dp_reduce(self.dp_part, self.pos, self.dp)
            with timers.around("wgrad_down"):
                moe.moe_grouped_wgrad(self.dout_perm, self.s, self.offsets,
                                      self.dw2)
            with timers.around("gate_up_dgrad"):
                moe.moe_gate_up_dgrad(self.dab, self.offsets, w_gu,
                                      self.dx_perm)
            with timers.around("wgrad_gate_up"):
                moe.moe_grouped_wgrad(self.dab, self.x_perm, self.offsets,
                                      self.dw_gu)
        self._finish_dx(timers)
        return self.dx, self.dw_gu, self.dw2, self.dp

    def _finish_dx(self, timers):
        """Combine dX; with a router, its backward runs first (score
        gradients, dW_g, db, the balancing loss) and the combine adds the
        router's share of dX before the one rounding."""
        if self._router is None:
            with _around(timers, "unpermute_dx"):
                moe.moe_unpermute(self.dx_perm, self.pos, None, self.dx)
            return
        x, w_g, bias = self._router
        with _around(timers, "router_backward"):
            moe.moe_router_backward(
                self._logits_used, self.topk_idx, self.topk_w, self.dp,
                self.counts, self.aux_coef, self.renorm, x, w_g,
                self.dlogits, self.dw_g, self.db if bias is not None else None,
                None, None, self.aux_loss, self.ws_router)
        with _around(timers, "unpermute_dx"):
            moe.moe_unpermute(self.dx_perm, self.pos, None, self.dx,
                              dlogits=self.dlogits, w_g=w_g)


class StepGraph:
    """A step (e.g. one forward and backward of a path) captured once as a
    HIP graph and replayed.  Every buffer and workspace belongs to the path
    and no entry point allocates, clears with a memset, synchronizes or
    reads back to the host, so the captured launches are the whole step.
    The step runs eagerly twice first: once to allocate what the path
    allocates lazily, once on the capture's side stream."""

    def __init__(self, step):
        step()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            step()
        torch.cuda.synchronize()

    def replay(self):
        self.graph.replay()


class MoEPathMX(MoEPath):
    """The layer with MXFP8 GEMM operands (see the module docstring)."""

    def __init__(self, T, d, f, E, k, renorm=True, device="cuda",
                 y_fp32=False, aux_coef=0.01, act_fp4=False, training=True):
        super().__init__(T, d, f, E, k, renorm=renorm, prec=MOE_BF16,
                         device=device, y_fp32=y_fp32, aux_coef=aux_coef)
        # training: the forward quantizes each weight for both of its GEMMs
        # from one read (moe_mxfp8_quantize_weight) and the backward uses
        # those column-wise codes; otherwise only the forward's codes are
        # made and the backward quantizes the weights it is given
        self.training = training
        self.act_fp4 = act_fp4
        self.prec = MOE_MXFP4 if act_fp4 else MOE_MXFP8
        Tk = T * k
        dev = self.x_perm.device
        u8 = torch.uint8
        z = lambda *s: torch.empty(*s, dtype=u8, device=dev)  # noqa: E731
        dx = d // 2 if act_fp4 else d          # payload bytes a row
        self.xq, self.xs = z(T, dx), z(T, d // 32)
        self.xpq, self.xps = z(Tk, dx), z(Tk, d // 32)
        self.wguq, self.wgus = z(E, 2 * f, d), z(E, 2 * f, d // 32)
        self.w2q, self.w2s = z(E, d, f), z(E, d, f // 32)
        self.sq, self.ss = z(Tk, f), z(Tk, f // 32)
        # S along each expert's tokens, written by the gate_up epilogue and
        # read by the dW2 GEMM of the backward
        tp = moe.moe_mxfp8_padded_rows(Tk, E)
        self.tk_pad = tp
        self.st, self.sts = z(f, tp), z(f, tp // 32)
        self.s = None
        if training:
            self.w2tq, self.w2ts = z(f, E * d), z(f, E * d // 32)
            self.wgutq, self.wguts = z(d, E * 2 * f), z(d, E * 2 * f // 32)
        ws_f = moe.moe_workspace_bytes(MOE_ENTRY_MLP_FWD, MOE_MXFP8, T, E, k,
                                       d, f)
        self.ws_fwd = z(max(ws_f, 16))

    def _alloc_bwd(self):
        super()._alloc_bwd()
        T, d, f, E, k = self.T, self.d, self.f, self.E, self.k
        Tk = T * k
        dev = self.x_perm.device
        u8 = torch.uint8
        z = lambda *s: torch.empty(*s, dtype=u8, device=dev)  # noqa: E731
        tp = self.tk_pad
        self.doq, self.dos = z(Tk, d), z(Tk, d // 32)
        if not self.training:
            self.w2tq, self.w2ts = z(f, E * d), z(f, E * d // 32)
            self.wgutq, self.wguts = z(d, E * 2 * f), z(d, E * 2 * f // 32)
        self.dab = None
        self.dabq, self.dabs = z(Tk, 2 * f), z(Tk, 2 * f // 32)
        self.dot, self.dots = z(d, tp), z(d, tp // 32)
        self.dabt, self.dabts = z(2 * f, tp), z(2 * f, tp // 32)
        self.xpt = z(d, tp // 2 if self.act_fp4 else tp)
        self.xpts = z(d, tp // 32)
        ws_b = moe.moe_workspace_bytes(MOE_ENTRY_MLP_BWD, MOE_MXFP8, T, E, k,
                                       d, f)
        self.ws_bwd = z(max(ws_b, 16))

    def quantize_weights(self, w_gu, w2, timers=None):
        """MX codes of the weights (once per optimizer step): along their
        rows for the forward GEMMs and, when training, along their columns
        for the data-gradient GEMMs, from the same read."""
        E, d, f = self.E, self.d, self.f
        with _around(timers, "quant_weights"):
            if self.training:
                moe.moe_mxfp8_quantize_weight(
                    w_gu.view(E * 2 * f, d), self.wguq.view(E * 2 * f, d),
                    self.wgus.view(E * 2 * f, d // 32), self.wgutq,
                    self.wguts)
                moe.moe_mxfp8_quantize_weight(
                    w2.view(E * d, f), self.w2q.view(E * d, f),
                    self.w2s.view(E * d, f // 32), self.w2tq, self.w2ts)
            else:
                moe.moe_mxfp8_quantize(w_gu.view(E * 2 * f, d), 0, None,
                                       self.wguq.view(E * 2 * f, d),
                                       self.wgus.view(E * 2 * f, d // 32))
                moe.moe_mxfp8_quantize(w2.view(E * d, f), 0, None,
                                       self.w2q.view(E * d, f),
                                       self.w2s.view(E * d, f // 32))

    def forward(self, x, w_gu, w2, w_g=None, bias=None, logits=None,
                timers=None):
        self.route(x, w_g, bias, logits, timers)
        with _around(timers, "quant_x"):
            if self.act_fp4:
                moe.moe_mxfp4_quantize(x, 0, None, self.xq, self.xs)
            else:
                moe.moe_mxfp8_quantize(x, 0, None, self.xq, self.xs)
        with _around(timers, "permute"):
            moe.moe_permute(self.prec, self.topk_idx, self.topk_w, self.E,
                            self.xq, self.xs, self.counts, self.offsets,
                            self.pos, self.src, self.w_perm, self.xpq,
                            self.xps, self.ws_permute)
        self.quantize_weights(w_gu, w2, timers)
        if timers is None:
            moe.moe_grouped_mlp_fwd(self.prec, self.xpq, self.xps,
                                    self.offsets, self.wguq, self.wgus,
                                    self.w2q, self.w2s, self.w_perm, self.ab,
                                    None, self.o, self.ws_fwd,
                                    s_tok=self.st, s_tok_scales=self.sts)
        else:
            with timers.around("gate_up_swiglu_fwd"):
                moe.moe_mx_gate_up_swiglu_fwd(
                    self.xpq, self.xps, self.offsets, self.wguq, self.wgus,
                    self.w_perm, self.ab, None, self.sq, self.ss,
                    s_tok=self.st, s_tok_scales=self.sts,
                    x_fp4=self.act_fp4)
            with timers.around("down_fwd"):
                moe.moe_mx_down_fwd(self.sq, self.ss, self.offsets, self.w2q,
                                    self.w2s, self.o)
        with _around(timers, "unpermute_y"):
            moe.moe_unpermute(self.o, self.pos, None, self.y)
        self._x = x
        return self.y

    def backward(self, dy, w_gu, w2, timers=None):
        if not self._bwd_ready:
            self._alloc_bwd()
        E, d, f = self.E, self.d, self.f
        with _around(timers, "permute_dy"):
            moe.moe_permute_rows(MOE_BF16, self.pos, dy, None,
                                 self.dout_perm, None)
        if not self.act_fp4:
            # the MXFP4 variant reads the forward's payload instead
            with _around(timers, "permute_x"):
                moe.moe_permute_rows(MOE_BF16, self.pos, self._x, None,
                                     self.x_perm, None)
        xp, xps = ((self.xpq, self.xps) if self.act_fp4
                   else (self.x_perm, None))
        if timers is None:
            # when training, the forward's column-wise weight codes go in
            # ready-made
            cols = ({"w_gu_col": (self.wgutq, self.wguts),
                     "w2_col": (self.w2tq, self.w2ts)} if self.training
                    else {})
            moe.moe_grouped_mlp_bwd(self.prec, self.dout_perm, xp,
                                    self.offsets, self.pos, w_gu, w2, self.ab,
                                    None, self.w_perm, self.dx_perm,
                                    self.dw_gu, self.dw2, self.dp,
                                    self.ws_bwd, s_tok=self.st,
                                    s_tok_scales=self.sts,
                                    x_perm_scales=xps, **cols)
        else:
            # the kernels of moe_grouped_mlp_bwd in its order (when
            # training, the column-wise weight codes from the forward's
            # quantize_weights, as the fused call is given them)
            tp = self.tk_pad
            with timers.around("quant_bwd_operands"):
                moe.moe_mxfp8_quantize(self.dout_perm, 0, None, self.doq,
                                       self.dos)
                if not self.training:
                    moe.moe_mxfp8_quantize(w2.view(E * d, f), 1, None,
                                           self.w2tq, self.w2ts, E * d)
                    moe.moe_mxfp8_quantize(w_gu.view(E * 2 * f, d), 1, None,
                                           self.wgutq, self.wguts, E * 2 * f)
            with timers.around("down_swiglu_bwd"):
                moe.moe_mx_down_swiglu_bwd(
                    self.doq, self.dos, self.offsets, self.w2tq, self.w2ts,
                    self.ab, self.w_perm, None, self.dabq, self.dabs,
                    self.dp_part, dab_tok=self.dabt,
                    dab_tok_scales=self.dabts)
            with timers.around("dp_reduce"):
                moe.moe_dp_reduce(self.dp_part, self.pos, self.dp)
            with timers.around("gate_up_dgrad"):
                moe.moe_mx_gate_up_dgrad(self.dabq, self.dabs, self.offsets,
                                         self.wgutq, self.wguts, self.dx_perm)
            with timers.around("quant_tokens"):
                moe.moe_mxfp8_quantize(self.dout_perm, 1, self.offsets,
                                       self.dot, self.dots, tp)
                if self.act_fp4:
                    moe.moe_mxfp4_quantize(self.xpq, 1, self.offsets,
                                           self.xpt, self.xpts, tp,
                                           src_scales=self.xps)
                else:
                    moe.moe_mxfp8_quantize(self.x_perm, 1, self.offsets,
                                           self.xpt, self.xpts, tp)
            Tk = self.T * self.k
            with timers.around("wgrad_down"):
                moe.moe_mx_grouped_wgrad(self.dot, self.dots, self.st,
                                         self.sts, self.offsets, Tk, self.dw2)
            with timers.around("wgrad_gate_up"):
                moe.moe_mx_grouped_wgrad(self.dabt, self.dabts, self.xpt,
                                         self.xpts, self.offsets, Tk,
                                         self.dw_gu, b_fp4=self.act_fp4)
        self._finish_dx(timers)
        return self.dx, self.dw_gu, self.dw2, self.dp


class MoEDecode:
    """The layer for a fixed number of tokens, up to
    ``moe.MOE_LAYER_MAX_TOKENS``, forward only: one library call that reads
    the weights of the experts it reaches once (w2 twice for an expert of
    more than 32 tokens).  With prec MOE_MXFP8 w_gu and w2 are pairs of codes
    and scales, as ``quantize`` makes them of the bf16 weights once."""

    def __init__(self, T, d, f, E, k, renorm=True, prec=MOE_BF16,
                 device="cuda"):
        n = moe.moe_workspace_bytes(MOE_ENTRY_LAYER_FWD, prec, T, E, k, d, f)
        if n == 0:
            raise ValueError(
                f"MoEDecode takes 1 to {moe.MOE_LAYER_MAX_TOKENS} tokens, "
                "k <= 32 of up to 1024 experts, prec MOE_BF16 (d and f "
                "multiples of 8) or MOE_MXFP8 (of 128) and an expert's weight "
                f"below 4 GiB; got T={T}, d={d}, f={f}, E={E}, k={k}, "
                f"prec={prec}")
        self.T, self.d, self.f, self.E, self.k = T, d, f, E, k
        self.renorm, self.prec = renorm, prec
        dev = torch.device(device)
        self.topk_idx = torch.empty(T, k, dtype=torch.int32, device=dev)
        self.topk_w = torch.empty(T, k, dtype=torch.float32, device=dev)
        self.y = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
        self.ws = torch.empty(n, dtype=torch.uint8, device=dev)
        self._forwards = 0

    @staticmethod
    def quantize(w):
        """MXFP8 codes and scales of a bf16 weight [E, rows, cols] along its
        last axis."""
        E, rows, cols = w.shape
        z = lambda n: torch.empty(E, rows, n, dtype=torch.uint8,  # noqa: E731
                                  device=w.device)
        codes, scales = z(cols), z(cols // 32)
        with torch.cuda.device(w.device):
            for e in range(E):
                moe.moe_mxfp8_quantize(w[e], 0, None, codes[e], scales[e])
        return codes, scales

    def forward(self, x, w_gu, w2, w_g=None, bias=None, logits=None,
                timers=None, y_add=None):
        """y = y_add + the layer's output for x."""
        self._forwards += 1
        gu, gu_s = (w_gu, None) if self.prec == MOE_BF16 else w_gu
        dn, dn_s = (w2, None) if self.prec == MOE_BF16 else w2
        given = logits is not None
        with _around(timers, "layer_fwd"):
            moe.moe_layer_fwd(self.prec, x, None if given else w_g,
                              None if given else bias, logits, self.k,
                              self.renorm, gu, gu_s, dn, dn_s, y_add,
                              self.topk_idx, self.topk_w, self.y, self.ws)
        return self.y

    def _alloc_bwd(self):
        raise NotImplementedError("MoEDecode has no backward: use MoEPath or "
                                  "MoEPathMX")

    _bwd_ready = False


class AdamW:
    """AdamW over the weights of paths and blocks, one library call a step.

    params: (weight, gradient) or (weight, gradient, weight_decay), as the
    ``gradients`` methods of paths and blocks give them; the gradients' buffers
    are read anew at every step.  moments: MOE_MOMENTS_FP32 or
    MOE_MOMENTS_FP8 (8 bits and a scale for 256 values).  master: keep an fp32
    copy of each bf16 weight, from which it is updated.  max_norm: clip the
    gradients to that norm over all of them, and leave a step out whose norm
    is not finite.  lr, the number of steps made and the norm live on the
    device, so that ``step`` can be captured; ``lr.fill_`` changes the rate of
    captured steps too.  ``state_dict`` and ``load_state_dict`` store and load
    what a run that goes on needs beside the weights: the number of steps, the
    rate, the moments with their scales and the fp32 copies.
    """

    _KEPT = ("master", "m", "v", "m_scale", "v_scale")

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.95), eps=1e-8,
                 weight_decay=0.1, moments=MOE_MOMENTS_FP32, master=True,
                 max_norm=None):
        if max_norm is not None and not 0 < max_norm <= 3.4e38:
            raise ValueError("AdamW: max_norm must be finite and above 0")
        if moments not in (MOE_MOMENTS_FP32, MOE_MOMENTS_FP8):
            raise ValueError(f"AdamW: unknown form of the moments {moments}")
        if not all(0 <= b < 1 for b in betas):
            raise ValueError("AdamW: betas must be in [0, 1)")
        least = 1e-12 if moments == MOE_MOMENTS_FP8 else 1e-20
        if not least <= eps <= 1:
            raise ValueError(f"AdamW: eps must be in [{least}, 1]")
        self.betas, self.eps, self.max_norm = betas, eps, max_norm
        rows = []
        for w, g, *wd in params:
            row = {"p": w, "g": g, "weight_decay": wd[0] if wd else
                   weight_decay}
            if master and w.dtype == torch.bfloat16:
                row["master"] = w.detach().float()
            if moments == MOE_MOMENTS_FP32:
                for n in ("m", "v"):
                    row[n] = torch.zeros_like(w, dtype=torch.float32)
            else:
                blocks = -(-w.numel() // moe.MOE_ADAMW_BLOCK)
                for n in ("m", "v"):
                    row[n] = torch.zeros_like(w, dtype=torch.uint8).view(
                        torch.float8_e4m3fn)
                    row[n + "_scale"] = torch.zeros(
                        blocks, dtype=torch.float32, device=w.device)
            rows.append(row)
        self.table = moe.adamw_table(rows)
        self.grads = moe.grad_table([r["g"] for r in rows])
        self.rows = rows
        dev = rows[0]["p"].device
        self.lr = torch.full((1,), lr, dtype=torch.float32, device=dev)
        self.steps = torch.zeros(1, dtype=torch.int64, device=dev)
        self.norm = torch.zeros(1, dtype=torch.float32, device=dev)
        n = moe.moe_workspace_bytes(MOE_ENTRY_GRAD_NORM, MOE_BF16, 1, 1, 1, 8,
                                    8)
        self.ws = torch.empty(n, dtype=torch.uint8, device=dev)

    def step(self, timers=None):
        with torch.cuda.device(self.norm.device):
            norm = None
            if self.max_norm is not None:
                norm = self.norm
                with _around(timers, "grad_norm"):
                    moe.moe_grad_norm(self.grads, norm, self.ws)
                self.steps.add_(torch.isfinite(norm))
            else:
                self.steps.add_(1)
            with _around(timers, "adamw"):
                moe.moe_adamw(self.table, self.steps, self.lr, *self.betas,
                              self.eps, norm, self.max_norm or 1.0)


    def state_dict(self):
        """The optimizer's own tensors (not copies of them), those of a weight
        in a dict each, in the order of the weights."""
        return {"steps": self.steps, "lr": self.lr,
                "weights": [{n: r[n] for n in self._KEPT if n in r}
                            for r in self.rows]}

    def load_state_dict(self, state):
        """Copies a state_dict of the same weights, moments and copies into
        this optimizer's tensors, which stay where they are (so captured steps
        go on with them); anything else is refused before the first copy."""
        mine = self.state_dict()
        if len(state["weights"]) != len(mine["weights"]):
            raise ValueError(f"state of {len(state['weights'])} weights, not "
                             f"of {len(mine['weights'])}")
        pairs = [("steps", self.steps, state["steps"]),
                 ("lr", self.lr, state["lr"])]
        for i, (a, b) in enumerate(zip(mine["weights"], state["weights"])):
            if a.keys() != b.keys():
                raise ValueError(f"weight {i}: state of {sorted(b)}, not of "
                                 f"{sorted(a)}")
            pairs += [(f"weight {i}: {n}", a[n], b[n]) for n in a]
        for name, a, b in pairs:
            if a.shape != b.shape or a.dtype != b.dtype:
                raise ValueError(f"{name}: {b.dtype} {tuple(b.shape)}, not "
                                 f"{a.dtype} {tuple(a.shape)}")
        for _, a, b in pairs:
            a.copy_(b)


def _extent(t):
    """First byte of a contiguous tensor and the byte past its last."""
    lo = t.data_ptr()
    return lo, lo + t.numel() * t.element_size()


def _buffers(owner, label, but=()):
    """(name, first byte, end) of the tensors that owner allocated for its
    calls; names with an underscore hold a caller's."""
    return [(f"{label} {n}", *_extent(t)) for n, t in vars(owner).items()
            if isinstance(t, torch.Tensor) and n[0] != "_" and n not in but]


def _refuse_overlap(name, t, buffers):
    lo, hi = _extent(t)
    for n, b, e in buffers:
        if lo < e and b < hi:
            raise ValueError(f"{name} overlaps {n}, which the block replaces "
                             f"before it has read {name} for the last time")


def _on_its_device(call):
    """Runs a block's call with its path's device as the current one: the
    path's entries launch on the current device's stream, those around it on
    their tensors', and the two have to be one stream."""
    @functools.wraps(call)
    def run(self, *args, **kw):
        with torch.cuda.device(self.path.y.device):
            return call(self, *args, **kw)
    return run


class MoEBlock:
    """Pre-norm residual block around an expert layer (a ``MoEPath``,
    ``MoEPathMX`` or, forward only, ``MoEDecode`` with bf16 output):

      n = norm(x);  z = experts(n) [+ ffn(n)];  y = x + dropout(z)

    f_shared > 0 adds the dense feed-forward block (the "shared expert") of
    that width.  x, y and their gradients are the residual stream, bf16 or
    (stream_fp32) fp32.  The buffers belong to the block and the path; y, dx
    and the gradients are overwritten by the next call, and a backward is
    that of the path's last forward.  x and dy are read twice, first and
    last, so neither may lie in a buffer of the block or the path, but for
    the block's own results: a forward takes its y (and then has no
    backward), a backward its y or its dx as dy.

    forward:  moe_norm_fwd -> the path's calls -> moe_ffn_fwd (into the
              path's y) -> moe_dropout
    backward: moe_dropout -> the path's calls -> moe_ffn_bwd (into the
              path's dx) -> moe_norm_bwd (adding the residual's dy)
    """

    def __init__(self, path, norm=MOE_NORM_RMS, eps=1e-5, f_shared=0,
                 act=MOE_ACT_SILU, stream_fp32=False):
        if path.y.dtype != torch.bfloat16:
            raise ValueError("MoEBlock needs a path with bf16 output")
        self.path, self.norm, self.eps = path, norm, eps
        self.f_shared, self.act = f_shared, act
        T, d = path.T, path.d
        dev = path.y.device
        self.stream_dtype = torch.float32 if stream_fp32 else torch.bfloat16
        f32, bf = torch.float32, torch.bfloat16
        z = lambda *s, dt=bf: torch.empty(*s, dtype=dt, device=dev)  # noqa
        self.n = z(T, d)
        self.y = z(T, d, dt=self.stream_dtype)
        self.mean = z(T, dt=f32) if norm == MOE_NORM_LAYER else None
        self.rstd = z(T, dt=f32)
        # a generator state for calls without dropout, which draw nothing
        self._no_rng = torch.zeros(2, dtype=torch.int64, device=dev)
        if f_shared:
            self.ab, self.s = z(T, 2 * f_shared), z(T, f_shared)
            self.ws_ffn = self._ws(MOE_ENTRY_FFN_FWD, f_shared)
        # what a forward replaces; dx is a backward's alone
        self._fwd_bufs = (_buffers(path, "the path's", ("dx",)) +
                          _buffers(self, "the block's", ("y",)))
        self._x = None
        self._bwd_ready = False

    def _ws(self, entry, f):
        n = moe.moe_workspace_bytes(entry, MOE_BF16, self.path.T, 1, 1,
                                    self.path.d, f)
        return torch.empty(max(n, 16), dtype=torch.uint8,
                           device=self.path.y.device)

    def _alloc_bwd(self):
        T, d, f = self.path.T, self.path.d, self.f_shared
        dev = self.path.y.device
        f32, bf = torch.float32, torch.bfloat16
        z = lambda *s, dt=bf: torch.empty(*s, dtype=dt, device=dev)  # noqa
        self.dz = z(T, d)
        self.dx = z(T, d, dt=self.stream_dtype)
        self.dgamma = z(d, dt=f32)
        self.dbeta = z(d, dt=f32) if self.norm == MOE_NORM_LAYER else None
        self.ws_norm = self._ws(MOE_ENTRY_NORM_BWD, 0)
        if f:
            self.dsw_gu, self.dsw2 = z(2 * f, d), z(d, f)
            self.ws_ffn_bwd = self._ws(MOE_ENTRY_FFN_BWD, f)
        if not self.path._bwd_ready:
            self.path._alloc_bwd()
        # what stands between a backward's two reads of dy, and of x
        self._bwd_bufs = (_buffers(self.path, "the path's", ("y",)) +
                          _buffers(self, "the block's", ("y", "dx")))
        self._dx_buf = [("the block's dx", *_extent(self.dx))]
        self._bwd_ready = True

    def gradients(self, gamma, w_gu, w2, beta=None, w_g=None, bias=None,
                  sw_gu=None, sw2=None):
        """(weight, gradient[, weight decay]) of the block's and the path's
        weights, as ``AdamW`` takes them; the norm's have no weight decay."""
        if self.f_shared and (sw_gu is None or sw2 is None):
            raise ValueError("f_shared > 0 needs sw_gu and sw2")
        if beta is not None and self.norm != MOE_NORM_LAYER:
            raise ValueError("beta goes with layer norm")
        if not self._bwd_ready:
            self._alloc_bwd()
        out = [(gamma, self.dgamma, 0.0)]
        if beta is not None:
            out.append((beta, self.dbeta, 0.0))
        out += self.path.gradients(w_gu, w2, w_g, bias)
        if self.f_shared:
            out += [(sw_gu, self.dsw_gu), (sw2, self.dsw2)]
        return out

    @_on_its_device
    def forward(self, x, gamma, w_gu, w2, beta=None, w_g=None, bias=None,
                logits=None, sw_gu=None, sw2=None, p=0.0, rng=None, delta=0,
                timers=None):
        """y = x + dropout(experts(norm(x)) + ffn(norm(x))).  sw_gu, sw2 are
        the feed-forward block's weights; rng (int64 {seed, offset} on the
        device) and delta choose the dropout mask, as in moe_dropout, and
        are needed when p > 0; backward uses the same p, rng and delta, so
        rng is advanced only between a backward and the next forward."""
        if p > 0 and rng is None:
            raise ValueError("dropout (p > 0) needs rng")
        if self.f_shared and (sw_gu is None or sw2 is None):
            raise ValueError("f_shared > 0 needs sw_gu and sw2")
        _refuse_overlap("x", x, self._fwd_bufs)
        self._x = None      # until every call below has been made
        with _around(timers, "norm_fwd"):
            moe.moe_norm_fwd(self.norm, x, gamma, beta, self.eps, self.n,
                             self.mean, self.rstd)
        z = self.path.forward(self.n, w_gu, w2, w_g=w_g, bias=bias,
                              logits=logits, timers=timers)
        if self.f_shared:
            with _around(timers, "ffn_fwd"):
                moe.moe_ffn_fwd(self.act, self.n, sw_gu, sw2, z, self.ab,
                                self.s, z, self.ws_ffn)
        self._drop = (p, self._no_rng if rng is None else rng, delta)
        with _around(timers, "dropout_fwd"):
            moe.moe_dropout(z, x, *self._drop, self.y)
        # x may be the last call's y, which this call's y has replaced
        if x.data_ptr() != self.y.data_ptr():
            self._x = x
        self._path_forward = self.path._forwards
        return self.y

    @_on_its_device
    def backward(self, dy, gamma, w_gu, w2, sw_gu=None, sw2=None,
                 timers=None):
        """dx; the weights' gradients are left in dgamma, dbeta, dsw_gu and
        dsw2, and in the path (dw_gu, dw2, and the router's).  It reads the
        forward's x again, so that must be as it was and not the block's own
        y."""
        if self._x is None:
            raise ValueError("backward needs a forward that has ended and "
                             "whose x was not this block's y")
        if self.f_shared and (sw_gu is None or sw2 is None):
            raise ValueError("f_shared > 0 needs sw_gu and sw2")
        if self.path._forwards != self._path_forward:
            raise ValueError("the path has run another forward since this "
                             "block's")
        if not self._bwd_ready:
            self._alloc_bwd()
        _refuse_overlap("dy", dy, self._bwd_bufs)
        _refuse_overlap("x", self._x, self._bwd_bufs + self._dx_buf)
        with _around(timers, "dropout_bwd"):
            moe.moe_dropout(dy, None, *self._drop, self.dz)
        dn = self.path.backward(self.dz, w_gu, w2, timers=timers)[0]
        if self.f_shared:
            with _around(timers, "ffn_bwd"):
                moe.moe_ffn_bwd(self.act, self.dz, self.n, sw_gu, sw2,
                                self.ab, self.s, dn, dn, self.dsw_gu,
                                self.dsw2, self.ws_ffn_bwd)
        with _around(timers, "norm_bwd"):
            moe.moe_norm_bwd(self.norm, dn, self._x, gamma, self.mean,
                             self.rstd, dy, self.dx, self.dgamma, self.dbeta,
                             self.ws_norm)
        return self.dx
