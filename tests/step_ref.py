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


def grow(kv_len, n, table, free, count, page, T):
    """One request after the other, as the header says; changes copies, returns them."""
    kv_len, table = kv_len.copy(), table.copy()
    have = top = max(0, min(int(count), len(free)))
    slots, positions = np.full(T, -1, np.int64), np.zeros(T, np.int64)
    start, granted, asked = [0], [], 0
    room = table.shape[1] * page
    for r in range(len(kv_len)):
        old, new = min(max(int(kv_len[r]), 0), room), max(int(n[r]), 0)
        ok = old + new <= room
        if ok:
            need = -(-(old + new) // page) - -(-old // page)
            asked += need
            ok = need == 0 or asked <= have
        if ok:
            for k in range(need):
                table[r, -(-old // page) + k] = free[have - 1 - (asked - need + k)]
            top -= need
        for i in range(new):
            t = start[-1] + i
            if t < T:
                positions[t] = old + i
                if ok:
                    slots[t] = int(table[r, (old + i) // page]) * page + (old + i) % page
        kv_len[r] = old + new if ok else old
        granted.append(int(ok))
        start.append(start[-1] + new)
    return kv_len, table, top, np.array(start), slots, positions, np.array(granted)


def trim(kv_len, keep, table, free, count, page):
    kv_len, table, free = kv_len.copy(), table.copy(), free.copy()
    count = max(0, min(int(count), len(free)))
    gone = []
    for r in range(len(kv_len)):
        old = min(max(int(kv_len[r]), 0), table.shape[1] * page)
        new = min(max(int(keep[r]), 0), old)
        for p in range(-(-new // page), -(-old // page)):
            gone.append(table[r, p])
            table[r, p] = -1
        kv_len[r] = new
    for k, page_number in enumerate(reversed(gone)):
        if count + k < len(free):
            free[count + k] = page_number
    return kv_len, table, free, min(count + len(gone), len(free))
