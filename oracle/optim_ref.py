"""Numpy oracle of the optimizer step: the gradients' norm and AdamW in
float64, and the 8-bit moments in float32 with every operation rounded by
itself, as include/moe.h defines them."""

import math

import numpy as np

from . import mx_ref

BLOCK = 256
F = np.float32


def grad_norm(grads):
    """2-norm of all arrays taken together."""
    return math.sqrt(math.fsum(float((np.asarray(g, np.float64) ** 2).sum())
                               for g in grads))


def clip_factor(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6))


def moments(m, v, g, b1, b2):
    return b1 * m + (1.0 - b1) * g, b2 * v + (1.0 - b2) * g * g


def parameter(p, m, r, t, lr, b1, b2, eps, wd):
    """p after step t with the new moments m and r = sqrt(v)."""
    den = r / math.sqrt(1.0 - b2 ** t) + eps
    return p - lr * wd * p - lr / (1.0 - b1 ** t) * m / den


# -------------------------------------------------------------- 8 bits
class Moment(np.ndarray):
    """float32 values of a moment after a step, and (``codes``) the E4M3 codes
    that they had before it."""
    codes = None


def dither(t):
    """Units of 2^-20 of the distance between codes added at step t."""
    return ((t * 0x9E3779B1) & 0xFFFFFFFF) >> 12


def moments8(qm, sm, qr, sr, g, b1, b2):
    """New m and r = sqrt(v), float32 [n], from E4M3 codes, their scales and
    the float32 gradient."""
    n = g.size
    b1f, c1f, b2f, c2f = F(b1), F(1.0 - b1), F(b2), F(1.0 - b2)
    m = mx_ref.e4m3_decode(qm).astype(F) * np.repeat(sm, BLOCK)[:n]
    r = mx_ref.e4m3_decode(qr).astype(F) * np.repeat(sr, BLOCK)[:n]
    m = m * b1f + g * c1f
    v = r * r * b2f + g * g * c2f
    r = np.where(v >= F(2.0 ** -96), np.sqrt(v), F(0.0))
    m, r = m.view(Moment), r.view(Moment)
    m.codes, r.codes = np.array(qm), np.array(qr)
    return m, r


def _cut(y, t):
    """y after the dither of step t, cut to four significant bits."""
    bits = np.ascontiguousarray(y, F).view(np.uint32).astype(np.int64)
    return ((bits + dither(t)) & 0xFFF00000).astype(np.uint32).view(F)


def quantize8(x, t, second):
    """(codes, scales) of float32 x at step t; second: of r.  Values that
    moments8 gave know the codes that they had; others had none."""
    had = getattr(x, "codes", None)
    x = np.asarray(x)
    n = x.size
    blocks = -(-n // BLOCK)
    pad = np.zeros(blocks * BLOCK, F)
    pad[:n] = x
    b = pad.reshape(blocks, BLOCK)
    top = np.abs(b).max(axis=1)
    live = top >= F(1e-30)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.where(live, F(256.0) / top, F(0.0)).astype(F)
    y = b * inv[:, None]
    if second:
        y = np.where(b > 0, np.maximum(y, F(2.0 ** -9)), F(0.0)).astype(F)
    y = y.reshape(-1)[:n]
    codes = mx_ref.e4m3_encode(_cut(y, t).astype(np.float64))
    if had is not None:
        # below 2^-6 a value that would keep its code is cut to the code's
        # unit, 2^-9, which is that of four bits from 2^-6 to 2^-5
        held = (np.abs(y) < F(2.0 ** -6)) & (codes == had)
        low = np.copysign(F(2.0 ** -6), y)
        small = _cut(y + low, t) - low
        codes = np.where(held, mx_ref.e4m3_encode(small.astype(np.float64)),
                         codes)
    scales = np.where(live, top * F(2.0 ** -8), F(0.0)).astype(F)
    return codes, scales
