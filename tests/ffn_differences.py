"""Gradients of the dense feed-forward block against central differences of
the float64 forward, direction by direction.

Each gradient is taken over blocks of its rows and columns (all of it, its
first and last rows and columns, and for w_gu the gate's and the up
projection's rows), so that a missing piece shows.  In a block, the gradient
is compared along random directions v ~ N(0, 1) and along the formula's own
gradient, where nothing cancels.

Tolerance.  A result has passed at most four roundings to bf16 in a row (AB, S
or [dA dU], the sum), each of relative size at most h = 2^-8 and, uniform over
a step, of root mean square at most h / sqrt(3), on terms whose signs are
random: its error vector e has |e| <= 2 h / sqrt(3) |G| = 1.16 h |G| in the
mean square.  e is independent of v, so e . v is about normal with deviation
1.16 h |G|; 6 h |G| is 5.2 of them.  Along a unit vector |e . v| <= |e|, for
which 6 h |G| is ample.  |G| is that of the block.  The quotients themselves are exact to
1e-6 |G|."""

import numpy as np

from oracle import block_ref as B

H = 2.0 ** -8
STEP = 1e-5


def blocks(name, shape):
    """(what, mask) of the pieces of a gradient that are looked at alone."""
    rows, cols = shape
    r, c = np.arange(rows)[:, None], np.arange(cols)[None, :]
    cut = {"all": r >= 0, "first rows": r < rows // 4,
           "last rows": r >= rows - rows // 4}
    if name == "dw_gu":
        f = rows // 2
        cut.update({"gate": r < f, "up": r >= f,
                    "last gate rows": (r >= f - f // 4) & (r < f)})
    out = [(n, m & (c >= 0)) for n, m in cut.items()]
    out += [("first columns", (c < cols // 4) & (r >= 0)),
            ("last columns", (c >= cols - cols // 4) & (r >= 0))]
    return out


def worst(act, N, grads, directions=4):
    """The largest difference in units of the tolerance, and where.  N: x,
    w_gu, w2, dy in float64; grads: (dx, dw_gu, dw2) under test."""
    args = [N["x"], N["w_gu"], N["w2"]]

    def loss(a):
        return float((B.ffn_forward(act, *a)[0] * N["dy"]).sum())

    y, a, u, s = B.ffn_forward(act, *args)
    formula = B.ffn_backward(act, N["dy"], *args, a, u, s)
    rng = np.random.default_rng(0)
    top = (0.0, "")
    for i, name in enumerate(("dx", "dw_gu", "dw2")):
        for what, mask in blocks(name, args[i].shape):
            size = np.linalg.norm(formula[i] * mask)
            vs = [rng.normal(size=mask.shape) * mask
                  for _ in range(directions)]
            vs.append(formula[i] * mask / size)
            for v in vs:
                lo, hi = list(args), list(args)
                hi[i], lo[i] = args[i] + STEP * v, args[i] - STEP * v
                quot = (loss(hi) - loss(lo)) / (2 * STEP)
                off = abs(quot - float((grads[i] * v).sum())) / (6 * H * size)
                if not off <= top[0]:
                    top = (off, f"{name}, {what}")
    return top
