"""Plain formulations, in 64 bits, of the operators in include/rope_serving.h
(rotary positions with several axes, the paged cache, attention of drafted
tokens over it), for the tests of the CUDA kernels.  numpy only."""
from __future__ import annotations

import numpy as np

TOP = {"fp8": 448.0, "int8": 127.0}


def deal(sections, order):
    """(axis, index within the axis) of each pair."""
    if order == "blocked":
        return [(a, j) for a, n in enumerate(sections) for j in range(n)]
    got, used, a = [], [0] * len(sections), 0
    while len(got) < sum(sections):
        if used[a] < sections[a]:
            got.append((a, used[a]))
            used[a] += 1
        a = (a + 1) % len(sections)
    return got


def pair_lanes(L, mode):
    """The two lanes (slice-relative) of each pair."""
    return [(2 * k, 2 * k + 1) if mode == "interleave" else (k, k + L // 2) for k in range(L // 2)]


def angles(positions, sections, L, base, order, spectrum):
    """theta (B', S', L / 2) from int positions (axes, B', S')."""
    at = deal(sections, order)
    t = np.empty(positions.shape[1:] + (L // 2,))
    for k, (a, j) in enumerate(at):
        e = k / (L // 2) if spectrum == "shared" else j / sections[a]
        t[..., k] = positions[a].astype(np.float64) * float(base) ** -e
    return t


def axes_rope(x, positions, sections, start, end, base=10000.0, mode="interleave", order="blocked",
              spectrum="shared", backward=False):
    """x (B, S, N, D) float64 -> the rotated tensor, float64."""
    L = end - start
    t = angles(positions, sections, L, base, order, spectrum)[:, :, None, :]
    c, s = np.cos(t), np.sin(t) * (-1.0 if backward else 1.0)
    y = x.astype(np.float64).copy()
    for k, (m, n) in enumerate(pair_lanes(L, mode)):
        a, b = x[..., start + m].astype(np.float64), x[..., start + n].astype(np.float64)
        y[..., start + m] = a * c[..., k] - b * s[..., k]
        y[..., start + n] = b * c[..., k] + a * s[..., k]
    return y


def rotate_rows_fp32(k, cos, sin, start, end, mode):
    """k (T, H, D), cos and sin (T or 1, L), all float32: the rotation with one
    fp32 rounding per product and sum, as the kernels do it."""
    y = k.astype(np.float32).copy()
    c, s = cos.astype(np.float32)[:, None, :], sin.astype(np.float32)[:, None, :]
    for m, n in pair_lanes(end - start, mode):
        a, b = k[..., start + m].astype(np.float32), k[..., start + n].astype(np.float32)
        y[..., start + m] = a * c[..., m] - b * s[..., m]
        y[..., start + n] = b * c[..., n] + a * s[..., n]
    return y


def fp8_values():
    """The numbers of the 256 e4m3 codes (NaN for 0x7f and 0xff)."""
    v = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        x = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[b] = np.nan if (b & 127) == 127 else (-x if b >> 7 else x)
    return v


def to_fp8(x):
    """The nearest e4m3 code of each number in [-448, 448], ties to even."""
    pos = fp8_values()[:127]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    down, up = a - pos[lo], pos[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= 448.0, 126, code)
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantise_fp32(y, store):
    """(codes, scale) of float32 rows, with the kernels' fp32 steps."""
    top = np.float32(TOP[store])
    with np.errstate(invalid="ignore"):
        m = np.maximum(np.abs(y).max(-1), np.float32(2.0 ** -100)).astype(np.float32)
        finite = np.isfinite(y).all(-1)
        inv = (top / m).astype(np.float32)
        z = np.where(finite[..., None], (y * inv[..., None]).astype(np.float32), 0)
    codes = to_fp8(z.astype(np.float64)) if store == "fp8" else np.rint(z).astype(np.int8)
    scale = np.where(finite, (m / top).astype(np.float32), np.float32(np.nan))
    return codes, scale


def tree_attention(q, k_rows, v_rows, sees, scale):
    """One request and query head: q (n, Dk), k_rows (len, Dk), v_rows (len,
    Dv), sees (n, len) -> out, lse, and sum_j p_j |v_j| / sum_j p_j for error
    bounds, all float64.  What a token does not see is left out altogether."""
    n, dv = q.shape[0], v_rows.shape[1]
    out, lse, mag = np.zeros((n, dv)), np.full(n, -np.inf), np.zeros((n, dv))
    for i in range(n):
        at = np.nonzero(sees[i])[0]
        if at.size == 0:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            s = (k_rows[at] @ q[i]) * scale
            m = s.max()
            p = np.exp(s - m)
            out[i] = p @ v_rows[at] / p.sum()
            mag[i] = p @ np.abs(v_rows[at]) / p.sum()
            lse[i] = m + np.log(p.sum())
    return out, lse, mag


def tree_sees(n, length, prefix, words):
    """sees (n, length) from tree words (n, W) int64 (None: a chain)."""
    sees = np.zeros((n, length), bool)
    for i in range(n):
        for j in range(length):
            jj = j - prefix
            if jj < 0:
                sees[i, j] = True
            elif words is None:
                sees[i, j] = jj <= i
            elif jj < 64 * words.shape[1]:
                sees[i, j] = bool(int(words[i, jj // 64]) >> (jj % 64) & 1)
    return sees
