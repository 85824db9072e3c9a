"""Float64 numpy oracle of the operators around the expert layer: layer norm
and RMS norm, dropout from a counter-based generator, and the dense gated
feed-forward block, forward and backward, from their formulas."""

import numpy as np


# ------------------------------------------------------------------ norm
def norm_forward(x, gamma, beta, eps, rms):
    """y, mean, rstd of each row (mean is 0 for RMS norm)."""
    d = x.shape[1]
    mean = np.zeros(x.shape[0]) if rms else x.sum(axis=1) / d
    xc = x - mean[:, None]
    rstd = 1.0 / np.sqrt((xc * xc).sum(axis=1) / d + eps)
    y = xc * rstd[:, None] * gamma
    if beta is not None:
        y = y + beta
    return y, mean, rstd


def norm_backward(dy, x, gamma, eps, rms, dres=None):
    """dx, dgamma, dbeta."""
    _, mean, rstd = norm_forward(x, gamma, None, eps, rms)
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    t = g - xh * (g * xh).mean(axis=1, keepdims=True)
    if not rms:
        t = t - g.mean(axis=1, keepdims=True)
    dx = rstd[:, None] * t
    if dres is not None:
        dx = dx + dres
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


# --------------------------------------------------------------- dropout
def philox4x32(counter, key, rounds=10):
    """Philox4x32 (Salmon et al., SC'11).  counter: 4 arrays or ints, key: 2
    ints, 32-bit words.  Returns 4 uint64 arrays of 32-bit words."""
    m, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    c = [np.atleast_1d(np.asarray(v, dtype=np.uint64)) for v in counter]
    k = [int(v) for v in key]
    for _ in range(rounds):
        p0 = c[0] * np.uint64(0xD2511F53)
        p1 = c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> sh) ^ c[1] ^ np.uint64(k[0]), p1 & m,
             (p0 >> sh) ^ c[3] ^ np.uint64(k[1]), p0 & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF,
             (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_draws(n, seed, offset, first=0):
    """The 16-bit draws of elements first .. first + n - 1 (first a multiple
    of 8)."""
    seed, offset = int(seed) % (1 << 64), int(offset) % (1 << 64)
    blk = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    full = np.full_like(blk, 0)
    w = philox4x32([blk & np.uint64(0xFFFFFFFF), blk >> np.uint64(32),
                    full + np.uint64(offset & 0xFFFFFFFF),
                    full + np.uint64(offset >> 32)],
                   [seed & 0xFFFFFFFF, seed >> 32])
    out = np.empty((blk.size, 8), dtype=np.int64)
    for i in range(8):
        half = w[i // 2] >> np.uint64(16 * (i % 2))
        out[:, i] = half & np.uint64(0xFFFF)
    return out.reshape(-1)[:n]


def dropout(x, res, p, seed, offset):
    """res + dropout(x), flat order, and the kept mask."""
    thr = int(np.floor(p * 65536.0 + 0.5))
    keep = (dropout_draws(x.size, seed, offset) >= thr).reshape(x.shape)
    base = np.zeros_like(x) if res is None else res
    if thr == 65536:
        return base, keep
    kept = np.where(keep, x, 0.0) * (65536.0 / (65536 - thr))
    return base + kept, keep


# ------------------------------------------------------------------- ffn
def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def activation(act, a):
    """Value and slope; act "silu" or "gelu_tanh"."""
    if act == "silu":
        s = _sigmoid(a)
        return a * s, s * (1.0 + a * (1.0 - s))
    c = np.sqrt(2.0 / np.pi)
    th = np.tanh(c * (a + 0.044715 * a ** 3))
    return (0.5 * a * (1.0 + th),
            0.5 * (1.0 + th) + 0.5 * a * (1.0 - th * th) * c *
            (1.0 + 3 * 0.044715 * a * a))


def ffn_forward(act, x, w_gu, w2, y_add=None):
    """y and the saved gate, up and product."""
    f = w2.shape[1]
    a, u = x @ w_gu[:f].T, x @ w_gu[f:].T
    s = activation(act, a)[0] * u
    y = s @ w2.T
    if y_add is not None:
        y = y + y_add
    return y, a, u, s


def ffn_backward(act, dy, x, w_gu, w2, a, u, s, dx_add=None):
    """dx, dw_gu, dw2 from the saved a, u, s."""
    h, slope = activation(act, a)
    ds = dy @ w2
    dab = np.concatenate((ds * u * slope, ds * h), axis=1)
    dx = dab @ w_gu
    if dx_add is not None:
        dx = dx + dx_add
    return dx, dab.T @ x, dy.T @ s
