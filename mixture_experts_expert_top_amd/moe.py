"""Python binding of libmoe.so (see include/moe.h for the semantics).

Argument marshalling only: each function checks that the torch tensors have
the dtype, device and contiguity the C-ABI expects, passes their device
pointers and the current HIP stream, and raises MoeError on a non-zero
status.  All compute happens in the library's kernels.  Importing this
module fails loudly when libmoe.so has not been built.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_BF16 = 0
MOE_MXFP8 = 1
MOE_MXFP4 = 2
MOE_ENTRY_PERMUTE = 0
MOE_ENTRY_MLP_FWD = 1
MOE_ENTRY_MLP_BWD = 2
MOE_ENTRY_ROUTER_BWD = 3
MOE_ENTRY_NORM_BWD = 4
MOE_ENTRY_FFN_FWD = 5
MOE_ENTRY_FFN_BWD = 6
MOE_ENTRY_GRAD_NORM = 7
MOE_ENTRY_LAYER_FWD = 8
MOE_LAYER_MAX_TOKENS = 64
MOE_MOMENTS_FP32 = 0
MOE_MOMENTS_FP8 = 1
MOE_ADAMW_BLOCK = 256
MOE_NORM_LAYER = 0
MOE_NORM_RMS = 1
MOE_ACT_SILU = 0
MOE_ACT_GELU_TANH = 1

EXPORTED = [
    "moe_status_str", "moe_last_error", "moe_version", "moe_router_logits",
    "moe_route", "moe_permute", "moe_permute_rows", "moe_grouped_mlp_fwd",
    "moe_grouped_mlp_bwd", "moe_unpermute", "moe_mxfp8_quantize",
    "moe_mxfp8_quantize_weight",
    "moe_mxfp8_padded_rows", "moe_workspace_bytes", "moe_dp_tiles",
    "moe_gate_up_swiglu_fwd", "moe_down_fwd", "moe_down_swiglu_bwd",
    "moe_gate_up_dgrad", "moe_grouped_wgrad", "moe_dp_reduce",
    "moe_row_planes", "moe_mx_gate_up_swiglu_fwd", "moe_mx_down_fwd",
    "moe_mx_down_swiglu_bwd", "moe_mx_gate_up_dgrad", "moe_mx_grouped_wgrad",
    "moe_router_backward", "moe_mxfp4_quantize", "moe_permute_noalloc",
    "moe_norm_fwd", "moe_norm_bwd", "moe_dropout", "moe_ffn_fwd",
    "moe_ffn_bwd", "moe_grad_norm", "moe_adamw", "moe_layer_fwd",
]
# fixed per-GPU scratch of moe_permute_noalloc (MOE_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 2 << 20


class MoeError(RuntimeError):
    def __init__(self, name, status, status_str, message):
        super().__init__(f"{name} failed: {status_str}: {message}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m mixture_experts_expert_top_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                       ctypes.c_size_t)
    sig = {
        "moe_status_str": (ctypes.c_char_p, [I32]),
        "moe_last_error": (ctypes.c_char_p, []),
        "moe_version": (ctypes.c_char_p, []),
        "moe_router_logits": (I32, [P, P, P, I64, I64, I32, P, P]),
        "moe_route": (I32, [P, I64, I32, I32, I32, P, P, P]),
        "moe_permute": (I32, [I32, P, P, I64, I32, I32, P, P, I64, P, P, P,
                              P, P, P, P, P, SZ, P]),
        "moe_permute_noalloc": (I32, [I32, P, P, I64, I32, I32, P, P, I64,
                                      P, P, P, P, P, P, P, P]),
        "moe_permute_rows": (I32, [I32, P, I64, I32, P, P, I64, P, P, P]),
        "moe_grouped_mlp_fwd": (I32, [I32, P, P, P, I32, I64, I64, I64, P, P,
                                      P, P, P, P, P, P, P, P, I64, P, SZ,
                                      P]),
        "moe_grouped_mlp_bwd": (I32, [I32, P, P, P, P, P, I64, I32, I32,
                                      I64, I64, P, P, P, P, P, P, I64, P, P,
                                      P, P, P, P, P, P, P, P, SZ, P]),
        "moe_unpermute": (I32, [P, I32, I32, P, P, I64, I32, I64, I32, P,
                                P, P, I32, P]),
        "moe_row_planes": (I32, [I64]),
        "moe_mxfp8_quantize": (I32, [P, I64, I64, I32, P, I32, P, P, I64, P]),
        "moe_mxfp8_quantize_weight": (I32, [P, I64, I64, P, P, P, P, P]),
        "moe_mxfp8_padded_rows": (I64, [I64, I32]),
        "moe_mxfp4_quantize": (I32, [P, I32, P, I64, I64, I32, P, I32, P, P,
                                     I64, P]),
        "moe_workspace_bytes": (SZ, [I32, I32, I64, I32, I32, I64, I64]),
        "moe_dp_tiles": (I32, [I64]),
        "moe_gate_up_swiglu_fwd": (I32, [P, P, I32, I64, I64, I64, P, P, P,
                                         P, P]),
        "moe_down_fwd": (I32, [P, P, I32, I64, I64, I64, P, P, P]),
        "moe_down_swiglu_bwd": (I32, [P, P, I32, I64, I64, I64, P, P, P, P,
                                      P, P]),
        "moe_gate_up_dgrad": (I32, [P, P, I32, I64, I64, I64, P, P, P]),
        "moe_grouped_wgrad": (I32, [P, I64, P, I64, P, I32, I64, I64, I64, P,
                                    P]),
        "moe_dp_reduce": (I32, [P, I32, P, I64, I32, P, P]),
        "moe_mx_gate_up_swiglu_fwd": (I32, [P, P, I32, P, I32, I64, I64, I64,
                                            P, P, P, P, P, P, P, P, P, I64,
                                            P]),
        "moe_mx_down_fwd": (I32, [P, P, P, I32, I64, I64, I64, P, P, P, P]),
        "moe_mx_down_swiglu_bwd": (I32, [P, P, P, I32, I64, I64, I64, P, P,
                                         P, P, P, P, P, P, P, I64, P, P]),
        "moe_mx_gate_up_dgrad": (I32, [P, P, P, I32, I64, I64, I64, P, P, P,
                                       P]),
        "moe_mx_grouped_wgrad": (I32, [P, P, P, P, I32, I64, P, I32, I64,
                                       I64, I64, P, P]),
        "moe_router_backward": (I32, [P, P, P, P, P, ctypes.c_float, I64,
                                      I32, I32, I32, P, P, I64, P, P, P, P,
                                      P, P, P, SZ, P]),
        "moe_norm_fwd": (I32, [I32, P, I32, P, P, ctypes.c_float, I64, I64,
                               P, P, P, P]),
        "moe_norm_bwd": (I32, [I32, P, P, I32, P, P, P, P, I64, I64, P, P, P,
                               P, SZ, P]),
        "moe_dropout": (I32, [P, I32, P, I32, I64, ctypes.c_double, P,
                              ctypes.c_uint64, P, P]),
        "moe_ffn_fwd": (I32, [I32, P, P, P, P, I64, I64, I64, P, P, P, P, SZ,
                              P]),
        "moe_ffn_bwd": (I32, [I32, P, P, P, P, P, P, P, I64, I64, I64, P, P,
                              P, P, SZ, P]),
        "moe_layer_fwd": (I32, [I32, P, P, P, P, I64, I64, I64, I32, I32, I32,
                                P, P, P, P, P, P, P, P, P, SZ, P]),
        "moe_grad_norm": (I32, [P, I32, P, P, SZ, P]),
        "moe_adamw": (I32, [I32, P, I32, P, P, ctypes.c_double,
                            ctypes.c_double, ctypes.c_double, P,
                            ctypes.c_double, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def _p(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(name, status):
    if status != 0:
        raise MoeError(name, status, lib.moe_status_str(status).decode(),
                       lib.moe_last_error().decode())


def _want(t, name, dtype, shape=None, allow_none=False):
    if t is None:
        if allow_none:
            return
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, "
                         f"got {tuple(t.shape)}")


def version():
    return lib.moe_version().decode()




def row_planes(f):
    """Partial-sum planes of out_perm / dx_perm for intermediate width f."""
    return int(lib.moe_row_planes(int(f)))


def moe_workspace_bytes(entry, prec, T, E, k, d, f):
    return int(lib.moe_workspace_bytes(entry, prec, T, E, k, d, f))


def moe_router_logits(x, w_g, bias, logits, stream=None):
    T, d = x.shape
    E = w_g.shape[0]
    _want(x, "x", torch.bfloat16)
    _want(w_g, "w_g", torch.bfloat16, (E, d))
    _want(bias, "bias", torch.float32, (E,), allow_none=True)
    _want(logits, "logits", torch.float32, (T, E))
    _check("moe_router_logits", lib.moe_router_logits(
        _p(x), _p(w_g), _p(bias), T, d, E, _p(logits), _stream(stream)))


def moe_route(logits, k, renorm, topk_idx, topk_w, stream=None):
    T, E = logits.shape
    _want(logits, "logits", torch.float32)
    _want(topk_idx, "topk_idx", torch.int32, (T, k))
    _want(topk_w, "topk_w", torch.float32, (T, k))
    _check("moe_route", lib.moe_route(_p(logits), T, E, k, int(renorm),
                                      _p(topk_idx), _p(topk_w),
                                      _stream(stream)))


def moe_router_backward(logits, topk_idx, topk_w, dp, counts, aux_coef,
                        renorm, x, w_g, dlogits, dw_g, db, dx_in, dx_out,
                        aux_loss, workspace, stream=None):
    T, E = logits.shape
    k = topk_idx.shape[1]
    d = (x if x is not None else w_g).shape[1] if (
        x is not None or w_g is not None) else 0
    _want(logits, "logits", torch.float32)
    _want(topk_idx, "topk_idx", torch.int32, (T, k))
    _want(topk_w, "topk_w", torch.float32, (T, k))
    _want(dp, "dp", torch.float32, (T, k))
    _want(counts, "counts", torch.int32, (E,), allow_none=True)
    _want(x, "x", torch.bfloat16, (T, d), allow_none=True)
    _want(w_g, "w_g", torch.bfloat16, (E, d), allow_none=True)
    _want(dlogits, "dlogits", torch.float32, (T, E))
    _want(dw_g, "dw_g", torch.float32, (E, d), allow_none=True)
    _want(db, "db", torch.float32, (E,), allow_none=True)
    _want(dx_in, "dx_in", torch.float32, (T, d), allow_none=True)
    _want(dx_out, "dx_out", torch.bfloat16, (T, d), allow_none=True)
    _want(aux_loss, "aux_loss", torch.float32, (1,), allow_none=True)
    nbytes = workspace.numel() * workspace.element_size() if workspace \
        is not None else 0
    _check("moe_router_backward", lib.moe_router_backward(
        _p(logits), _p(topk_idx), _p(topk_w), _p(dp), _p(counts),
        float(aux_coef), T, E, k, int(renorm), _p(x), _p(w_g), d,
        _p(dlogits), _p(dw_g), _p(db), _p(dx_in), _p(dx_out), _p(aux_loss),
        _p(workspace), nbytes, _stream(stream)))


def _permute_args(prec, topk_idx, topk_w, E, x, x_scales, counts, offsets,
                  pos, src, w_perm, x_perm, x_perm_scales):
    T, k = topk_idx.shape
    xdt, per = _act(prec, x, "x")
    w = x.shape[1]
    d = w * per
    _want(topk_idx, "topk_idx", torch.int32)
    _want(topk_w, "topk_w", torch.float32, (T, k), allow_none=True)
    _want(x, "x", xdt, (T, w))
    _want(x_perm, "x_perm", xdt, (T * k, w))
    if prec != MOE_BF16:
        _want(x_scales, "x_scales", torch.uint8, (T, d // 32))
        _want(x_perm_scales, "x_perm_scales", torch.uint8, (T * k, d // 32))
    for n, t, shp in (("counts", counts, (E,)), ("offsets", offsets, (E + 1,)),
                      ("pos", pos, (T, k)), ("src", src, (T * k,))):
        _want(t, n, torch.int32, shp)
    _want(w_perm, "w_perm", torch.float32, (T * k,), allow_none=True)
    return (prec, _p(topk_idx), _p(topk_w), T, E, k, _p(x), _p(x_scales), d,
            _p(counts), _p(offsets), _p(pos), _p(src), _p(w_perm), _p(x_perm),
            _p(x_perm_scales))


def moe_permute(prec, topk_idx, topk_w, E, x, x_scales, counts, offsets, pos,
                src, w_perm, x_perm, x_perm_scales, workspace, stream=None):
    args = _permute_args(prec, topk_idx, topk_w, E, x, x_scales, counts,
                         offsets, pos, src, w_perm, x_perm, x_perm_scales)
    nbytes = workspace.numel() * workspace.element_size() if workspace \
        is not None else 0
    _check("moe_permute", lib.moe_permute(*args, _p(workspace), nbytes,
                                          _stream(stream)))


def moe_permute_noalloc(prec, topk_idx, topk_w, E, x, x_scales, counts,
                        offsets, pos, src, w_perm, x_perm, x_perm_scales,
                        stream=None):
    args = _permute_args(prec, topk_idx, topk_w, E, x, x_scales, counts,
                         offsets, pos, src, w_perm, x_perm, x_perm_scales)
    _check("moe_permute_noalloc", lib.moe_permute_noalloc(*args,
                                                          _stream(stream)))


def moe_permute_rows(prec, pos, x, x_scales, x_perm, x_perm_scales,
                     stream=None):
    T, k = pos.shape
    xdt, per = _act(prec, x, "x")
    w = x.shape[1]
    d = w * per
    _want(pos, "pos", torch.int32)
    _want(x, "x", xdt, (T, w))
    _want(x_perm, "x_perm", xdt, (T * k, w))
    _check("moe_permute_rows", lib.moe_permute_rows(
        prec, _p(pos), T, k, _p(x), _p(x_scales), d, _p(x_perm),
        _p(x_perm_scales), _stream(stream)))


def _act(prec, x, what):
    """(dtype, values per stored element) of an activation tensor: bf16,
    E4M3 codes, or E2M1 codes two a byte."""
    if prec == MOE_BF16:
        return torch.bfloat16, 1
    return torch.uint8, (2 if prec == MOE_MXFP4 else 1)


def _tok_out(name, codes, scales, cols):
    """(ldt, codes, scales) of an optional token-axis MX tensor
    ([cols][ldt] codes, [cols][ldt/32] scales)."""
    if codes is None and scales is None:
        return 0
    ldt = codes.shape[1]
    _want(codes, name, torch.uint8, (cols, ldt))
    _want(scales, name + "_scales", torch.uint8, (cols, ldt // 32))
    return ldt


def moe_grouped_mlp_fwd(prec, x_perm, x_perm_scales, offsets, w_gu,
                        w_gu_scales, w2, w2_scales, w_perm, ab_saved, s_saved,
                        out_perm, workspace=None, stream=None, s_tok=None,
                        s_tok_scales=None):
    Tk = x_perm.shape[0]
    E, two_f, d = w_gu.shape
    f = two_f // 2
    _want(offsets, "offsets", torch.int32, (E + 1,))
    xdt, per = _act(prec, x_perm, "x_perm")
    _want(x_perm, "x_perm", xdt, (Tk, d // per))
    if prec == MOE_BF16:
        _want(x_perm, "x_perm", torch.bfloat16)
        _want(w_gu, "w_gu", torch.bfloat16, (E, 2 * f, d))
        _want(w2, "w2", torch.bfloat16, (E, d, f))
    _want(w_perm, "w_perm", torch.float32, (Tk,), allow_none=True)
    _want(ab_saved, "ab_saved", torch.bfloat16, (Tk, 2 * f))
    _want(s_saved, "s_saved", torch.bfloat16, (Tk, f), allow_none=True)
    _want(out_perm, "out_perm", torch.float32, (row_planes(f), Tk, d))
    ldt = _tok_out("s_tok", s_tok, s_tok_scales, f)
    nbytes = workspace.numel() * workspace.element_size() if workspace \
        is not None else 0
    _check("moe_grouped_mlp_fwd", lib.moe_grouped_mlp_fwd(
        prec, _p(x_perm), _p(x_perm_scales), _p(offsets), E, Tk, d, f,
        _p(w_gu), _p(w_gu_scales), _p(w2), _p(w2_scales), _p(w_perm),
        _p(ab_saved), _p(s_saved), _p(out_perm), _p(s_tok), _p(s_tok_scales),
        ldt, _p(workspace), nbytes, _stream(stream)))


def moe_grouped_mlp_bwd(prec, dout_perm, x_perm, offsets, pos, w_gu, w2,
                        ab_saved, s_saved, w_perm, dx_perm, dw_gu, dw2, dp,
                        workspace, stream=None, s_tok=None, s_tok_scales=None,
                        x_perm_scales=None, w_gu_col=None, w2_col=None):
    """x_perm: bf16 rows (bf16 and MXFP8), or for MXFP4 the forward's
    payload, E2M1 codes [T*k, d/2] with x_perm_scales [T*k, d/32].
    w_gu_col / w2_col (MX): (codes, scales) of the weights along their
    columns as moe_mxfp8_quantize_weight makes them, codes [d, E*2f] /
    [f, E*d], scales [d, E*2f/32] / [f, E*d/32]; None to quantize inside
    the call."""
    Tk, d = dout_perm.shape
    T, k = pos.shape
    E, two_f, _ = w_gu.shape
    f = two_f // 2
    if prec == MOE_MXFP4:
        _want(x_perm, "x_perm", torch.uint8, (Tk, d // 2))
        _want(x_perm_scales, "x_perm_scales", torch.uint8, (Tk, d // 32))
    else:
        _want(x_perm, "x_perm", torch.bfloat16, (Tk, d))
    for n, t, shp in (("dout_perm", dout_perm, (Tk, d)),
                      ("w_gu", w_gu, (E, 2 * f, d)), ("w2", w2, (E, d, f)),
                      ("ab_saved", ab_saved, (Tk, 2 * f)),
                      ("dw_gu", dw_gu, (E, 2 * f, d)), ("dw2", dw2, (E, d, f))):
        _want(t, n, torch.bfloat16, shp)
    _want(s_saved, "s_saved", torch.bfloat16, (Tk, f), allow_none=True)
    ldt = _tok_out("s_tok", s_tok, s_tok_scales, f)
    _want(dx_perm, "dx_perm", torch.float32, (row_planes(f), Tk, d))
    _want(offsets, "offsets", torch.int32, (E + 1,))
    _want(pos, "pos", torch.int32)
    _want(w_perm, "w_perm", torch.float32, (Tk,), allow_none=True)
    _want(dp, "dp", torch.float32, (T, k))
    cols = {}
    for n, pair, rows, width in (("w_gu_col", w_gu_col, d, E * 2 * f),
                                 ("w2_col", w2_col, f, E * d)):
        if pair is None:
            cols[n] = (None, None)
            continue
        codes, scales = pair
        _want(codes, n + " codes", torch.uint8, (rows, width))
        _want(scales, n + " scales", torch.uint8, (rows, width // 32))
        cols[n] = (codes, scales)
    nbytes = workspace.numel() * workspace.element_size() if workspace \
        is not None else 0
    _check("moe_grouped_mlp_bwd", lib.moe_grouped_mlp_bwd(
        prec, _p(dout_perm), _p(x_perm), _p(x_perm_scales), _p(offsets),
        _p(pos), T, k, E, d, f,
        _p(w_gu), _p(w2), _p(ab_saved), _p(s_saved), _p(s_tok),
        _p(s_tok_scales), ldt, _p(cols["w_gu_col"][0]),
        _p(cols["w_gu_col"][1]), _p(cols["w2_col"][0]),
        _p(cols["w2_col"][1]), _p(w_perm), _p(dx_perm), _p(dw_gu), _p(dw2),
        _p(dp), _p(workspace), nbytes, _stream(stream)))


def moe_unpermute(o_perm, pos, w, y, stream=None, dlogits=None, w_g=None):
    """o_perm: bf16 [T*k, d] rows, or fp32 [T*k, d] / [planes, T*k, d].
    dlogits (fp32 [T, E]) with w_g (bf16 [E, d]): add the router's share
    of the input gradient before the rounding."""
    T, k = pos.shape
    d = o_perm.shape[-1]
    if o_perm.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("o_perm must be bfloat16 or float32")
    planes = o_perm.shape[0] if o_perm.dim() == 3 else 1
    _want(o_perm, "o_perm", o_perm.dtype,
          (planes, T * k, d) if o_perm.dim() == 3 else (T * k, d))
    _want(pos, "pos", torch.int32)
    _want(w, "w", torch.float32, (T, k), allow_none=True)
    if y.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("y must be bfloat16 or float32")
    _want(y, "y", y.dtype, (T, d))
    E = 0
    if dlogits is not None:
        E = dlogits.shape[1]
        _want(dlogits, "dlogits", torch.float32, (T, E))
        _want(w_g, "w_g", torch.bfloat16, (E, d))
    _check("moe_unpermute", lib.moe_unpermute(
        _p(o_perm), 1 if o_perm.dtype == torch.float32 else 0, planes,
        _p(pos), _p(w), T, k, d,
        1 if y.dtype == torch.float32 else 0, _p(y), _p(dlogits),
        _p(w_g) if dlogits is not None else None, E, _stream(stream)))


def moe_mxfp8_padded_rows(rows, nseg):
    return int(lib.moe_mxfp8_padded_rows(rows, nseg))


def moe_mxfp8_quantize(src, axis, seg_offsets, codes, scales, rows_pad=0,
                       stream=None):
    rows, cols = src.shape
    _want(src, "src", torch.bfloat16)
    _want(codes, "codes", torch.uint8)
    _want(scales, "scales", torch.uint8)
    nseg = 1 if seg_offsets is None else seg_offsets.numel() - 1
    if seg_offsets is not None:
        _want(seg_offsets, "seg_offsets", torch.int32)
    _check("moe_mxfp8_quantize", lib.moe_mxfp8_quantize(
        _p(src), rows, cols, axis, _p(seg_offsets), nseg, _p(codes),
        _p(scales), rows_pad, _stream(stream)))


def moe_mxfp8_quantize_weight(src, row_codes, row_scales, col_codes,
                              col_scales, stream=None):
    """Both MX layouts of a bf16 [rows, cols] weight from one read:
    row_codes [rows, cols] / row_scales [rows, cols/32] (axis 0) and
    col_codes [cols, rows] / col_scales [cols, rows/32] (axis 1, one
    segment)."""
    rows, cols = src.shape
    _want(src, "src", torch.bfloat16)
    _want(row_codes, "row_codes", torch.uint8, (rows, cols))
    _want(row_scales, "row_scales", torch.uint8, (rows, cols // 32))
    _want(col_codes, "col_codes", torch.uint8, (cols, rows))
    _want(col_scales, "col_scales", torch.uint8, (cols, rows // 32))
    _check("moe_mxfp8_quantize_weight", lib.moe_mxfp8_quantize_weight(
        _p(src), rows, cols, _p(row_codes), _p(row_scales), _p(col_codes),
        _p(col_scales), _stream(stream)))


def moe_mxfp4_quantize(src, axis, seg_offsets, codes, scales, rows_pad=0,
                       src_scales=None, cols=None, stream=None):
    """src: bf16 [rows, cols], or (with src_scales) MXFP4 rows as uint8
    codes [rows, cols/2] with scales [rows, cols/32].  Codes are two a
    byte: axis 0 gives [rows, cols/2], axis 1 [cols, rows_pad/2]."""
    rows = src.shape[0]
    if src_scales is None:
        _want(src, "src", torch.bfloat16)
        cols = src.shape[1]
        fmt = 0
    else:
        cols = 2 * src.shape[1]
        _want(src, "src", torch.uint8)
        _want(src_scales, "src_scales", torch.uint8, (rows, cols // 32))
        fmt = 1
    _want(codes, "codes", torch.uint8)
    _want(scales, "scales", torch.uint8)
    nseg = 1 if seg_offsets is None else seg_offsets.numel() - 1
    if seg_offsets is not None:
        _want(seg_offsets, "seg_offsets", torch.int32)
    _check("moe_mxfp4_quantize", lib.moe_mxfp4_quantize(
        _p(src), fmt, _p(src_scales), rows, cols, axis, _p(seg_offsets),
        nseg, _p(codes), _p(scales), rows_pad, _stream(stream)))


# ---------------------------------------------------------------- stages

def moe_dp_tiles(f):
    return int(lib.moe_dp_tiles(f))


def _mlp_dims(x_perm, w_gu):
    Tk, d = x_perm.shape
    E, two_f, _ = w_gu.shape
    return Tk, d, E, two_f // 2


def moe_gate_up_swiglu_fwd(x_perm, offsets, w_gu, w_perm, ab_saved, s_saved,
                           stream=None):
    Tk, d, E, f = _mlp_dims(x_perm, w_gu)
    _want(x_perm, "x_perm", torch.bfloat16)
    _want(w_gu, "w_gu", torch.bfloat16, (E, 2 * f, d))
    _want(offsets, "offsets", torch.int32, (E + 1,))
    _want(w_perm, "w_perm", torch.float32, (Tk,), allow_none=True)
    _want(ab_saved, "ab_saved", torch.bfloat16, (Tk, 2 * f))
    _want(s_saved, "s_saved", torch.bfloat16, (Tk, f))
    _check("moe_gate_up_swiglu_fwd", lib.moe_gate_up_swiglu_fwd(
        _p(x_perm), _p(offsets), E, Tk, d, f, _p(w_gu), _p(w_perm),
        _p(ab_saved), _p(s_saved), _stream(stream)))


def moe_down_fwd(s_saved, offsets, w2, out_perm, stream=None):
    Tk, f = s_saved.shape
    E, d, _ = w2.shape
    _want(s_saved, "s_saved", torch.bfloat16)
    _want(w2, "w2", torch.bfloat16, (E, d, f))
    _want(offsets, "offsets", torch.int32, (E + 1,))
    _want(out_perm, "out_perm", torch.float32, (row_planes(f), Tk, d))
    _check("moe_down_fwd", lib.moe_down_fwd(
        _p(s_saved), _p(offsets), E, Tk, d, f, _p(w2), _p(out_perm),
        _stream(stream)))


def moe_down_swiglu_bwd(dout_perm, offsets, w2, ab_saved, w_perm, dab,
                        dp_part, stream=None):
    Tk, d = dout_perm.shape
    E, _, f = w2.shape
    _want(dout_perm, "dout_perm", torch.bfloat16)
    _want(w2, "w2", torch.bfloat16, (E, d, f))
    _want(offsets, "offsets", torch.int32, (E + 1,))
    _want(ab_saved, "ab_saved", torch.bfloat16, (Tk, 2 * f))
    _want(w_perm, "w_perm", torch.float32, (Tk,), allow_none=True)
    _want(dab, "dab", torch.bfloat16, (Tk, 2 * f))
    _want(dp_part, "dp_part", torch.float32, (Tk, moe_dp_tiles(f)))
    _check("moe_down_swiglu_bwd", lib.moe_down_swiglu_bwd(
        _p(dout_perm), _p(offsets), E, Tk, d, f, _p(w2), _p(ab_saved),
        _p(w_perm), _p(dab), _p(dp_part), _stream(stream)))


def moe_gate_up_dgrad(dab, offsets, w_gu, dx_perm, stream=None):
    Tk, two_f = dab.shape
    E, _, d = w_gu.shape
    f = two_f // 2
    _want(dab, "dab", torch.bfloat16)
    _want(w_gu, "w_gu", torch.bfloat16, (E, 2 * f, d))
    _want(offsets, "offsets", torch.int32, (E + 1,))
    _want(dx_perm, "dx_perm", torch.float32, (row_planes(f), Tk, d))
    _check("moe_gate_up_dgrad", lib.moe_gate_up_dgrad(
        _p(dab), _p(offsets), E, Tk, d, f, _p(w_gu), _p(dx_perm),
        _stream(stream)))


def moe_grouped_wgrad(a, b, offsets, c, stream=None):
    Tk, M = a.shape
    _, N = b.shape
    E = offsets.numel() - 1
    _want(a, "a", torch.bfloat16)
    _want(b, "b", torch.bfloat16, (Tk, N))
    _want(offsets, "offsets", torch.int32)
    _want(c, "c", torch.bfloat16, (E, M, N))
    _check("moe_grouped_wgrad", lib.moe_grouped_wgrad(
        _p(a), M, _p(b), N, _p(offsets), E, Tk, M, N, _p(c),
        _stream(stream)))


def moe_dp_reduce(dp_part, pos, dp, stream=None):
    T, k = pos.shape
    _want(dp_part, "dp_part", torch.float32)
    _want(pos, "pos", torch.int32)
    _want(dp, "dp", torch.float32, (T, k))
    _check("moe_dp_reduce", lib.moe_dp_reduce(
        _p(dp_part), dp_part.shape[1], _p(pos), T, k, _p(dp),
        _stream(stream)))


# ------------------------------------------------------------- MX stages
# Codes are uint8 tensors, scales uint8 tensors with one byte per 32 codes
# along the reduction axis (layouts in include/moe.h).

def moe_mx_gate_up_swiglu_fwd(xq, xs, offsets, wq, ws, w_perm, ab_saved,
                              s_saved, sq, ss, s_tok=None, s_tok_scales=None,
                              stream=None, x_fp4=False):
    """xq: E4M3 codes [T*k, d], or (x_fp4) E2M1 codes [T*k, d/2]."""
    Tk = xq.shape[0]
    E, two_f, d = wq.shape
    f = two_f // 2
    _want(xq, "xq", torch.uint8, (Tk, d // 2 if x_fp4 else d))
    _want(xs, "xs", torch.uint8, (Tk, d // 32))
    _want(wq, "wq", torch.uint8, (E, 2 * f, d))
    _want(ws, "ws", torch.uint8, (E, 2 * f, d // 32))
    _want(offsets, "offsets", torch.int32, (E + 1,))
    _want(w_perm, "w_perm", torch.float32, (Tk,), allow_none=True)
    _want(ab_saved, "ab_saved", torch.bfloat16, (Tk, 2 * f))
    _want(s_saved, "s_saved", torch.bfloat16, (Tk, f), allow_none=True)
    _want(sq, "sq", torch.uint8, (Tk, f))
    _want(ss, "ss", torch.uint8, (Tk, f // 32))
    ldt = _tok_out("s_tok", s_tok, s_tok_scales, f)
    _check("moe_mx_gate_up_swiglu_fwd", lib.moe_mx_gate_up_swiglu_fwd(
        _p(xq), _p(xs), int(bool(x_fp4)), _p(offsets), E, Tk, d, f, _p(wq),
        _p(ws),
        _p(w_perm), _p(ab_saved), _p(s_saved), _p(sq), _p(ss), _p(s_tok),
        _p(s_tok_scales), ldt, _stream(stream)))


def moe_mx_down_fwd(sq, ss, offsets, wq, ws, out_perm, stream=None):
    Tk, f = sq.shape
    E, d, _ = wq.shape
    _want(sq, "sq", torch.uint8)
    _want(ss, "ss", torch.uint8, (Tk, f // 32))
    _want(wq, "wq", torch.uint8, (E, d, f))
    _want(ws, "ws", torch.uint8, (E, d, f // 32))
    _want(offsets, "offsets", torch.int32, (E + 1,))
    _want(out_perm, "out_perm", torch.float32, (row_planes(f), Tk, d))
    _check("moe_mx_down_fwd", lib.moe_mx_down_fwd(
        _p(sq), _p(ss), _p(offsets), E, Tk, d, f, _p(wq), _p(ws),
        _p(out_perm), _stream(stream)))


def moe_mx_down_swiglu_bwd(doq, dos, offsets, w2tq, w2ts, ab_saved, w_perm,
                           dab, dabq, dabs, dp_part, dab_tok=None,
                           dab_tok_scales=None, stream=None):
    Tk, d = doq.shape
    f, Ed = w2tq.shape
    E = offsets.numel() - 1
    _want(doq, "doq", torch.uint8)
    _want(dos, "dos", torch.uint8, (Tk, d // 32))
    _want(w2tq, "w2tq", torch.uint8, (f, E * d))
    _want(w2ts, "w2ts", torch.uint8, (f, E * d // 32))
    _want(offsets, "offsets", torch.int32)
    _want(ab_saved, "ab_saved", torch.bfloat16, (Tk, 2 * f))
    _want(w_perm, "w_perm", torch.float32, (Tk,), allow_none=True)
    _want(dab, "dab", torch.bfloat16, (Tk, 2 * f), allow_none=True)
    _want(dabq, "dabq", torch.uint8, (Tk, 2 * f))
    _want(dabs, "dabs", torch.uint8, (Tk, 2 * f // 32))
    _want(dp_part, "dp_part", torch.float32, (Tk, moe_dp_tiles(f)))
    ldt = _tok_out("dab_tok", dab_tok, dab_tok_scales, 2 * f)
    _check("moe_mx_down_swiglu_bwd", lib.moe_mx_down_swiglu_bwd(
        _p(doq), _p(dos), _p(offsets), E, Tk, d, f, _p(w2tq), _p(w2ts),
        _p(ab_saved), _p(w_perm), _p(dab), _p(dabq), _p(dabs), _p(dab_tok),
        _p(dab_tok_scales), ldt, _p(dp_part), _stream(stream)))


def moe_mx_gate_up_dgrad(dabq, dabs, offsets, wgutq, wguts, dx_perm,
                         stream=None):
    Tk, two_f = dabq.shape
    f = two_f // 2
    d = wgutq.shape[0]
    E = offsets.numel() - 1
    _want(dabq, "dabq", torch.uint8)
    _want(dabs, "dabs", torch.uint8, (Tk, two_f // 32))
    _want(wgutq, "wgutq", torch.uint8, (d, E * two_f))
    _want(wguts, "wguts", torch.uint8, (d, E * two_f // 32))
    _want(offsets, "offsets", torch.int32)
    _want(dx_perm, "dx_perm", torch.float32, (row_planes(f), Tk, d))
    _check("moe_mx_gate_up_dgrad", lib.moe_mx_gate_up_dgrad(
        _p(dabq), _p(dabs), _p(offsets), E, Tk, d, f, _p(wgutq), _p(wguts),
        _p(dx_perm), _stream(stream)))


def moe_mx_grouped_wgrad(aq, as_, bq, bs, offsets, Tk, c, stream=None,
                         b_fp4=False):
    """aq [M, ldt] E4M3 codes; bq [N, ldt] E4M3, or (b_fp4) E2M1 codes
    [N, ldt/2]."""
    M, ldt = aq.shape
    N = bq.shape[0]
    E = offsets.numel() - 1
    _want(aq, "aq", torch.uint8)
    _want(as_, "as", torch.uint8, (M, ldt // 32))
    _want(bq, "bq", torch.uint8, (N, ldt // 2 if b_fp4 else ldt))
    _want(bs, "bs", torch.uint8, (N, ldt // 32))
    _want(offsets, "offsets", torch.int32)
    _want(c, "c", torch.bfloat16, (E, M, N))
    _check("moe_mx_grouped_wgrad", lib.moe_mx_grouped_wgrad(
        _p(aq), _p(as_), _p(bq), _p(bs), int(bool(b_fp4)), ldt,
        _p(offsets), E, Tk, M, N, _p(c), _stream(stream)))


# ------------------------------------------------- around the expert layer
# The entries below take their device from their tensors: all must lie on
# one GPU, and the call runs on that GPU's current stream (or on `stream`,
# which must be one of that GPU's) whichever device is current.

_BF16, _F32 = torch.bfloat16, torch.float32
_F8, _U8, _I32 = torch.float8_e4m3fn, torch.uint8, torch.int32


def _checked(name, specs):
    """The device index and the pointers of the tensors of `specs`, a list of
    (name, tensor or None, dtype, shape or None); one pass over them, since
    the smallest calls cost little more than this."""
    dev = None
    mixed = False
    ptrs = []
    for tname, t, dtype, shape in specs:
        if t is None:
            ptrs.append(None)
            continue
        if t.dtype is not dtype or not t.is_contiguous() or (
                shape is not None and t.shape != shape):
            _want(t, f"{name}: {tname}", dtype, shape)
        i = t.get_device()
        if dev is None:
            dev = i
        elif i != dev:
            mixed = True
        ptrs.append(t.data_ptr())
    if mixed:
        raise ValueError(f"{name}: tensors on different devices: " + ", ".join(
            f"{n} {t.device}" for n, t, _, _ in specs if t is not None))
    if dev is None or dev < 0:
        raise ValueError(f"{name}: tensors must be on a GPU")
    return dev, ptrs


# The handle of a device's current stream without building a Stream object,
# and the current device's index, where torch offers them directly (1.4 us
# less of a 7 us call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice",
                          torch.cuda.current_device)


def _enqueue(name, stream, dev, fn, *args):
    """fn(*args, stream) on device `dev`; raises MoeError."""
    if stream is None:
        handle = _raw_stream(dev)
    else:
        if stream.device.index != dev:
            raise ValueError(f"{name}: tensors on cuda:{dev}, stream on "
                             f"{stream.device}")
        handle = stream.cuda_stream
    if dev == _current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status:
        _check(name, status)


def _stream_dtype(t, name):
    """The dtype of a residual-stream tensor: bf16 or fp32."""
    if t.dtype is not _BF16 and t.dtype is not _F32:
        raise TypeError(f"{name}: expected torch.bfloat16 or torch.float32, "
                        f"got {t.dtype}")
    return t.dtype


def _dtype(t):
    return None if t is None else t.dtype


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def moe_norm_fwd(kind, x, gamma, beta, eps, y, mean=None, rstd=None,
                 stream=None):
    """Layer norm or RMS norm of the rows of x (see include/moe.h); mean and
    rstd are written for moe_norm_bwd where given."""
    T, d = x.shape
    xt = _stream_dtype(x, "x")
    dev, p = _checked("moe_norm_fwd", (
        ("x", x, xt, None), ("gamma", gamma, _F32, (d,)),
        ("beta", beta, _F32, (d,)), ("y", y, _BF16, (T, d)),
        ("mean", mean, _F32, (T,)), ("rstd", rstd, _F32, (T,))))
    _enqueue("moe_norm_fwd", stream, dev, lib.moe_norm_fwd, kind, p[0],
             xt is _F32, p[1], p[2], eps, T, d, p[3], p[4], p[5])


def moe_norm_bwd(kind, dy, x, gamma, mean, rstd, dres, dx, dgamma, dbeta,
                 workspace, stream=None):
    """Gradient of moe_norm_fwd; dx = dres + the norm's (dres may be None,
    and dx may be dres)."""
    T, d = x.shape
    xt = _stream_dtype(x, "x")
    dev, p = _checked("moe_norm_bwd", (
        ("dy", dy, _BF16, (T, d)), ("x", x, xt, None),
        ("gamma", gamma, _F32, (d,)), ("mean", mean, _F32, (T,)),
        ("rstd", rstd, _F32, (T,)), ("dres", dres, xt, (T, d)),
        ("dx", dx, xt, (T, d)), ("dgamma", dgamma, _F32, (d,)),
        ("dbeta", dbeta, _F32, (d,)),
        ("workspace", workspace, _dtype(workspace), None)))
    _enqueue("moe_norm_bwd", stream, dev, lib.moe_norm_bwd, kind, p[0], p[1],
             xt is _F32, p[2], p[3], p[4], p[5], T, d, p[6], p[7], p[8],
             p[9], _nbytes(workspace))


def moe_dropout(x, res, p, rng, delta, out, stream=None):
    """out = res + dropout(x) (res may be None; out may be res, or x of its
    dtype; x and out may differ in dtype, res has out's).  rng is an int64
    tensor {seed, offset} on the device; the call on the upstream
    gradient with the same p, rng and delta is the backward pass."""
    xt, ot = _stream_dtype(x, "x"), _stream_dtype(out, "out")
    shape = x.shape
    dev, q = _checked("moe_dropout", (
        ("x", x, xt, None), ("res", res, ot, shape),
        ("rng", rng, torch.int64, (2,)), ("out", out, ot, shape)))
    _enqueue("moe_dropout", stream, dev, lib.moe_dropout, q[0], xt is _F32,
             q[1], ot is _F32, x.numel(), p, q[2], delta % (1 << 64), q[3])


def moe_ffn_fwd(act, x, w_gu, w2, y_add, ab_saved, s_saved, y, workspace,
                stream=None):
    """Dense gated feed-forward block, y = y_add + (act(gate) * up) . w2^T
    (y_add may be None, and y may be y_add); ab_saved and s_saved are written
    for moe_ffn_bwd where given."""
    T, d = x.shape
    f = w2.shape[1]
    dev, p = _checked("moe_ffn_fwd", (
        ("x", x, _BF16, None), ("w_gu", w_gu, _BF16, (2 * f, d)),
        ("w2", w2, _BF16, (d, f)), ("y_add", y_add, _BF16, (T, d)),
        ("ab_saved", ab_saved, _BF16, (T, 2 * f)),
        ("s_saved", s_saved, _BF16, (T, f)), ("y", y, _BF16, (T, d)),
        ("workspace", workspace, _dtype(workspace), None)))
    _enqueue("moe_ffn_fwd", stream, dev, lib.moe_ffn_fwd, act, p[0], p[1],
             p[2], p[3], T, d, f, p[4], p[5], p[6], p[7], _nbytes(workspace))


def moe_ffn_bwd(act, dy, x, w_gu, w2, ab_saved, s_saved, dx_add, dx, dw_gu,
                dw2, workspace, stream=None):
    """Gradient of moe_ffn_fwd; dx, dw_gu and dw2 may each be None, dx =
    dx_add + the block's (dx_add may be None, and dx may be dx_add)."""
    T, d = dy.shape
    f = w2.shape[1]
    dev, p = _checked("moe_ffn_bwd", (
        ("dy", dy, _BF16, None), ("x", x, _BF16, (T, d)),
        ("w_gu", w_gu, _BF16, (2 * f, d)), ("w2", w2, _BF16, (d, f)),
        ("ab_saved", ab_saved, _BF16, (T, 2 * f)),
        ("s_saved", s_saved, _BF16, (T, f)),
        ("dx_add", dx_add, _BF16, (T, d)), ("dx", dx, _BF16, (T, d)),
        ("dw_gu", dw_gu, _BF16, (2 * f, d)), ("dw2", dw2, _BF16, (d, f)),
        ("workspace", workspace, _dtype(workspace), None)))
    _enqueue("moe_ffn_bwd", stream, dev, lib.moe_ffn_bwd, act, p[0], p[1],
             p[2], p[3], p[4], p[5], p[6], T, d, f, p[7], p[8],
             p[9], p[10], _nbytes(workspace))


# --------------------------------------------------- few tokens (serving)

def moe_layer_fwd(prec, x, w_g, bias, logits, k, renorm, w_gu, w_gu_scales,
                  w2, w2_scales, y_add, topk_idx, topk_w, y, workspace,
                  stream=None):
    """The whole expert layer for up to MOE_LAYER_MAX_TOKENS tokens (see
    include/moe.h): the router's w_g (and bias) or its logits; weights bf16,
    or E4M3 codes with E8M0 scales (MOE_MXFP8); y = y_add + the layer's (y_add
    may be None, and y may be y_add)."""
    T, d = x.shape
    E, two_f, _ = w_gu.shape
    f = two_f // 2
    if prec == MOE_BF16:
        wt, sd, sf = _BF16, 0, 0
    else:
        wt, sd, sf = _U8, d // 32, f // 32
    dev, p = _checked("moe_layer_fwd", (
        ("x", x, _BF16, None), ("w_g", w_g, _BF16, (E, d)),
        ("bias", bias, _F32, (E,)), ("logits", logits, _F32, (T, E)),
        ("w_gu", w_gu, wt, (E, 2 * f, d)),
        ("w_gu_scales", w_gu_scales, _U8, (E, 2 * f, sd)),
        ("w2", w2, wt, (E, d, f)), ("w2_scales", w2_scales, _U8, (E, d, sf)),
        ("y_add", y_add, _BF16, (T, d)),
        ("topk_idx", topk_idx, _I32, (T, k)), ("topk_w", topk_w, _F32, (T, k)),
        ("y", y, _BF16, (T, d)),
        ("workspace", workspace, _dtype(workspace), None)))
    _enqueue("moe_layer_fwd", stream, dev, lib.moe_layer_fwd, prec, p[0], p[1],
             p[2], p[3], T, d, f, E, k, renorm, p[4], p[5], p[6], p[7], p[8],
             p[9], p[10], p[11], p[12], _nbytes(workspace))


# --------------------------------------------------------- optimizer step

class Grad(ctypes.Structure):
    """moe_grad of include/moe.h."""
    _fields_ = [("g", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("g_fp32", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class AdamwTensor(ctypes.Structure):
    """moe_adamw_tensor of include/moe.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("p", "master", "g", "m", "v", "m_scale", "v_scale")] + [
        ("n", ctypes.c_int64), ("weight_decay", ctypes.c_float),
        ("p_fp32", ctypes.c_int32), ("g_fp32", ctypes.c_int32),
        ("reserved", ctypes.c_int32)]


class _Table:
    """Descriptors of tensors that live as long as the table does, all on
    the GPU `dev`; built once and passed to every step."""

    def __init__(self, name, rows, struct, specs_of, fill):
        if not rows:
            raise ValueError(f"{name}: no tensors")
        self.entries = (struct * len(rows))()
        self.count = len(rows)
        self.tensors = []
        self.dev = None
        for i, row in enumerate(rows):
            specs = specs_of(row)
            dev, p = _checked(f"{name}: tensor {i}", specs)
            if self.dev is None:
                self.dev = dev
            elif dev != self.dev:
                raise ValueError(f"{name}: tensor {i} on cuda:{dev}, others "
                                 f"on cuda:{self.dev}")
            fill(self.entries[i], row, p)
            self.tensors.append([t for _, t, _, _ in specs if t is not None])
        self.ptr = ctypes.addressof(self.entries)


def grad_table(grads):
    """The table of moe_grad_norm: bf16 or fp32 tensors of any shape on one
    GPU, which have to stay where they are while the table is used (it holds
    a reference to each)."""
    def fill(e, g, p):
        e.g, e.n, e.g_fp32 = p[0], g.numel(), g.dtype is _F32
    return _Table("grad_table", grads, Grad,
                  lambda g: (("g", g, _stream_dtype(g, "g"), None),), fill)


class AdamwTable(_Table):
    moments = MOE_MOMENTS_FP32


def adamw_table(tensors):
    """The table of moe_adamw.  tensors: dicts of p (bf16 or fp32), g (bf16
    or fp32), m and v of one shape, master (fp32, for a bf16 p; optional) and
    weight_decay (0 if it is left out).  m and v are fp32, or all of them
    torch.float8_e4m3fn with m_scale and v_scale (fp32, one for each
    MOE_ADAMW_BLOCK values); a tensor that was never stepped has zeros in
    all of them.  The tensors have to stay where they are while the table is
    used (it holds a reference to each)."""
    known = {"p", "master", "g", "m", "v", "m_scale", "v_scale",
             "weight_decay"}
    fp8 = bool(tensors) and tensors[0]["m"].dtype is _F8

    def specs_of(t):
        if not known.issuperset(t):
            raise TypeError("adamw_table: unknown " +
                            ", ".join(sorted(set(t) - known)))
        p = t["p"]
        if p is None:
            raise ValueError("adamw_table: p is required")
        shape = p.shape
        for n in ("g", "m", "v"):
            _want(t[n], n, t[n].dtype if t[n] is not None else None)
        st = _F8 if fp8 else _F32
        blocks = (-(-p.numel() // MOE_ADAMW_BLOCK),)
        for n in ("m_scale", "v_scale"):
            if (t.get(n) is not None) != fp8:
                raise ValueError(f"adamw_table: {n} goes with moments in "
                                 "float8_e4m3fn")
        return (("p", p, _stream_dtype(p, "p"), None),
                ("master", t.get("master"), _F32, shape),
                ("g", t["g"], _stream_dtype(t["g"], "g"), shape),
                ("m", t["m"], st, shape), ("v", t["v"], st, shape),
                ("m_scale", t.get("m_scale"), _F32, blocks),
                ("v_scale", t.get("v_scale"), _F32, blocks))

    def fill(e, t, p):
        (e.p, e.master, e.g, e.m, e.v, e.m_scale, e.v_scale) = p
        e.n = t["p"].numel()
        e.weight_decay = float(t.get("weight_decay", 0.0))
        e.p_fp32 = t["p"].dtype is _F32
        e.g_fp32 = t["g"].dtype is _F32

    table = AdamwTable("adamw_table", tensors, AdamwTensor, specs_of, fill)
    table.moments = MOE_MOMENTS_FP8 if fp8 else MOE_MOMENTS_FP32
    return table


def _on_table(name, table, kind, specs):
    """Pointers of the tensors beside a table, which lie on its GPU."""
    if not isinstance(table, kind):
        raise TypeError(f"{name}: expected a table, got "
                        f"{type(table).__name__}")
    dev, p = _checked(name, specs)
    if dev != table.dev:
        raise ValueError(f"{name}: the table is on cuda:{table.dev}, other "
                         f"tensors on cuda:{dev}")
    return dev, p


def moe_grad_norm(table, norm, workspace, stream=None):
    """norm[0] = the 2-norm of all gradients of grad_table(...) together."""
    dev, p = _on_table("moe_grad_norm", table, _Table, (
        ("norm", norm, _F32, (1,)),
        ("workspace", workspace, _dtype(workspace), None)))
    if isinstance(table, AdamwTable):
        raise TypeError("moe_grad_norm: expected a grad_table")
    _enqueue("moe_grad_norm", stream, dev, lib.moe_grad_norm, table.ptr,
             table.count, p[0], p[1], _nbytes(workspace))


def moe_adamw(table, step, lr, beta1, beta2, eps, grad_norm=None,
              max_norm=1.0, stream=None):
    """One AdamW step over adamw_table(...), in place (see include/moe.h).
    step (int64 [1], the first step is 1), lr (fp32 [1]) and grad_norm (fp32
    [1] or None: no clipping) lie on the device and are read when the kernel
    runs."""
    dev, p = _on_table("moe_adamw", table, AdamwTable, (
        ("step", step, torch.int64, (1,)), ("lr", lr, _F32, (1,)),
        ("grad_norm", grad_norm, _F32, (1,))))
    _enqueue("moe_adamw", stream, dev, lib.moe_adamw, table.moments,
             table.ptr, table.count, p[0], p[1], beta1, beta2, eps, p[2],
             max_norm)
