"""Gradients of gradients through the two in-place operators.

y = R x (a rotation), loss = sum(w y^3) / 3: its gradient is g = R^T (w y^2), and
that of sum(g d) is R^T (2 w y (R d)).  R and R^T are taken in 64 bits.  Each lane of
each of the three rotations is off by at most 1e-6 (|x_m| + |x_n|), the products by
3 2^-24 of themselves, all of numbers below 5: 2 w y (R d) is below 2 * 5^2 * 7.1 and
off by 7 times 1e-5 of that, its rotation by 1.42 times as much; 1e-2 is above."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from gpu_util import DEV
from place_partial_rope_gb300 import torch_op

pytestmark = pytest.mark.gpu
SHAPE, START, END = (2, 9, 3, 48), 8, 40
SECTIONS = (5, 6, 5)


def check(turn, rotate, rotate_back):
    rng = np.random.default_rng(4)
    x, w, d = (np.clip(rng.standard_normal(SHAPE), -3, 3) for _ in range(3))
    xt = torch.tensor(x, dtype=torch.float32, device=DEV, requires_grad=True)
    wt, dt = (torch.tensor(t, dtype=torch.float32, device=DEV) for t in (w, d))
    y = xt * 1.0
    turn(y)
    (g,) = torch.autograd.grad((wt * y ** 3).sum() / 3, xt, create_graph=True)
    (gg,) = torch.autograd.grad((g * dt).sum(), xt)
    x32, w32, d32 = (t.astype(np.float32).astype(np.float64) for t in (x, w, d))
    yy = rotate(x32)
    assert np.abs(g.detach().double().cpu().numpy() - rotate_back(w32 * yy ** 2)).max() <= 1e-2
    assert np.abs(gg.double().cpu().numpy() - rotate_back(2 * w32 * yy * rotate(d32))).max() <= 1e-2


@pytest.mark.parametrize("mode", ["interleave", "half"])
def test_axes(mode):
    pos = np.random.default_rng(2).integers(0, 600, size=(3,) + SHAPE[:2]).astype(np.int32)
    pd = torch.from_numpy(pos).to(DEV)

    def rotation(back):
        return lambda t: ref.axes_rope(t, pos, SECTIONS, START, END, mode=mode, backward=back)

    check(lambda y: torch_op.inplace_axes_rotary_mul(y, pd, SECTIONS, partial_slice=[START, END], rotary_mode=mode),
          rotation(False), rotation(True))


@pytest.mark.parametrize("mode", ["interleave", "half"])
def test_tables(mode):
    L = END - START
    half = np.random.default_rng(3).uniform(-3, 3, size=(1, SHAPE[1], 1, L // 2))
    angle = np.concatenate([half, half], -1) if mode == "half" else np.repeat(half, 2, -1)
    cos, sin = (torch.tensor(f(angle), dtype=torch.float32, device=DEV) for f in (np.cos, np.sin))

    def rotation(back):
        s = np.sin(half) * (-1 if back else 1)

        def go(t):
            y = t.copy()
            for k, (m, n) in enumerate(ref.pair_lanes(L, mode)):
                a, b = t[..., START + m], t[..., START + n]
                y[..., START + m] = a * np.cos(half)[..., k] - b * s[..., k]
                y[..., START + n] = b * np.cos(half)[..., k] + a * s[..., k]
            return y
        return go

    check(lambda y: torch_op.inplace_partial_rotary_mul(y, cos, sin, rotary_mode=mode, partial_slice=[START, END]),
          rotation(False), rotation(True))
