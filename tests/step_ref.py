"""Plain formulations, in 64 bits, of the operators in include/rope_step.h, for the
tests of the CUDA kernels.  numpy only, written lane by lane from the formulas."""
from __future__ import annotations

import numpy as np

from serving_ref import pair_lanes


def rotate(x, cos, sin, start, L, mode, back=False):
    """Lanes [start, start + L) turned (back: by the transposed rotation); and what
    each lane's terms add up to without their signs."""
    y, mag = x.copy(), np.abs(x)
    for i, j in pair_lanes(L, mode):
        a, b = x[..., start + i], x[..., start + j]
        ca, cb, sa, sb = cos[..., i], cos[..., j], sin[..., i], sin[..., j]
        if back:
            y[..., start + i], y[..., start + j] = a * ca + b * sb, b * cb - a * sa
            mag[..., start + i], mag[..., start + j] = abs(a * ca) + abs(b * sb), abs(b * cb) + abs(a * sa)
        else:
            y[..., start + i], y[..., start + j] = a * ca - b * sa, b * cb + a * sb
            mag[..., start + i], mag[..., start + j] = abs(a * ca) + abs(b * sa), abs(b * cb) + abs(a * sb)
    return y, mag


def norm_fwd(x, w, cos, sin, start, end, n0, n1, eps, mode):
    """(out, magnitudes of out's terms, rstd) of rows x (..., D)."""
    r = 1.0 / np.sqrt((x[..., n0:n1] ** 2).mean(-1) + eps)
    y = x.copy()
    y[..., n0:n1] = x[..., n0:n1] * r[..., None] * (1.0 if w is None else w)
    return (*rotate(y, cos, sin, start, end - start, mode), r)


def norm_bwd(g, x, w, r, cos, sin, start, end, n0, n1, mode):
    """(dx, magnitudes, dw, magnitudes) for g (..., D), the gradient of the result."""
    g, mag = rotate(g, cos, sin, start, end - start, mode, back=True)
    w = np.ones(n1 - n0) if w is None else w
    u = x[..., n0:n1] * r[..., None]
    gn, mn = g[..., n0:n1], mag[..., n0:n1]
    mean = (w * gn * u).sum(-1, keepdims=True) / (n1 - n0)
    most = (abs(w * u) * mn).sum(-1, keepdims=True) / (n1 - n0)
    dx, dmag = g.copy(), mag.copy()
    dx[..., n0:n1] = r[..., None] * (w * gn - u * mean)
    dmag[..., n0:n1] = r[..., None] * (abs(w) * mn + abs(u) * most)
    axes = tuple(range(g.ndim - 1))
    return dx, dmag, (gn * u).sum(axes), (mn * abs(u)).sum(axes)
