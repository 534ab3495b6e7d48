"""GPU parity of the positions call with several axes, and its gradient.

The kernel's cos and sin are within 8e-7 of the exact ones (for |position| <
2^24), so a lane differs from the 64-bit result by at most 1e-6 (|x_m| + |x_n|)
plus the final rounding: 2 ulp of fp32 (the products' and the sum's fp32
roundings are below the first term), or half an ulp of the 16-bit type, taken
as one."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from gpu_util import DEV, split, storage_ulp, to_dev
from oracle import widen
from place_partial_rope_gb300 import binding, synth, torch_op

pytestmark = pytest.mark.gpu


def run(direction, x, pos, sections, start, end, dtype, **kw):
    xd = to_dev(x, dtype)
    fn = (binding.rope_partial_inplace_fwd_axes if direction == "fwd"
          else binding.rope_partial_inplace_bwd_axes)
    fn(xd, pos if isinstance(pos, torch.Tensor) else torch.from_numpy(pos).to(DEV), sections, start, end, **kw)
    torch.cuda.synchronize()
    return synth.from_torch(xd)


def check(got, x, pos, sections, start, end, dtype, direction, what, **kw):
    xw = widen(x, dtype).astype(np.float64)
    want = ref.axes_rope(xw, pos, sections, start, end, backward=direction == "bwd", **kw)
    same = np.ones(x.shape[-1], bool)
    same[start:end] = False
    assert np.array_equal(got[..., same], x[..., same]), what  # bytes outside the slice
    g = widen(np.ascontiguousarray(got[..., start:end]), dtype).astype(np.float64)
    w = want[..., start:end]
    xm, xn = split(xw[..., start:end], kw.get("mode", "interleave"))
    mag = np.abs(xm) + np.abs(xn)
    mag = (np.concatenate([mag, mag], -1) if kw.get("mode") == "half" else np.repeat(mag, 2, -1))
    ulp = storage_ulp(np.ascontiguousarray(synth.to_storage(w.astype(np.float32), dtype)), dtype)
    tol = 1e-6 * mag + (2 if dtype == "fp32" else 1) * ulp
    err = np.abs(g - w)
    assert np.all(err <= tol), f"{what}: worst ratio {(err / tol).max()}"


SHAPES = [  # x, start, end, sections, positions' (B, S)
    ((2, 6, 3, 64), 0, 64, (12, 10, 10), (2, 6)),
    ((1, 7, 5, 64), 4, 60, (1, 0, 27), (1, 7)),      # an axis without pairs
    ((2, 5, 1, 40), 3, 33, (5, 5, 5), (1, 5)),       # odd start, positions shared by the batch
    ((3, 1, 4, 128), 0, 128, (16, 24, 24), (3, 1)),  # one token
    ((1, 3, 2, 1024), 0, 1024, (200, 200, 56, 56), (1, 3)),  # the longest slice, four axes
    ((2, 9, 13, 24), 2, 18, (8,), (2, 1)),           # one axis, one position a batch
    ((1, 2, 7, 16), 6, 8, (0, 1), (1, 1)),           # one pair
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("mode", ["interleave", "half"])
@pytest.mark.parametrize("order,spectrum", [("blocked", "own"), ("interleaved", "shared"),
                                            ("interleaved", "own"), ("blocked", "shared")])
@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_parity(k, order, spectrum, mode, dtype):
    shape, st, en, sections, pshape = SHAPES[k]
    pos = np.random.default_rng(k).integers(-300, 40000, size=(len(sections),) + pshape).astype(np.int32)
    for d in ("fwd", "bwd"):
        x = synth.normal(shape, dtype, 900 + k)
        kw = dict(mode=mode, order=order, spectrum=spectrum, base=10000.0 if k % 2 else 500000.0)
        got = run(d, x, pos, sections, st, en, dtype, **kw)
        check(got, x, pos, sections, st, en, dtype, d, f"{shape} {d} {kw}", **kw)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mode", ["interleave", "half"])
def test_one_axis_is_the_positions_call(mode, dtype):
    x = synth.normal((2, 33, 6, 128), dtype, 3)
    pos = np.random.default_rng(5).integers(0, 2 ** 24, size=(1, 2, 33)).astype(np.int32)
    got = run("fwd", x, pos, (48,), 8, 104, dtype, mode=mode)
    xd = to_dev(x, dtype)
    binding.rope_partial_inplace_fwd_pos(xd, torch.from_numpy(pos[0]).to(DEV), 8, 104, 10000.0, mode)
    torch.cuda.synchronize()
    assert np.array_equal(got, synth.from_torch(xd))


def test_strided_positions():
    """Positions as a view: axes innermost, every other token, padded batches."""
    x = synth.normal((2, 5, 3, 32), "fp32", 4)
    buf = np.random.default_rng(1).integers(0, 999, size=(3, 16, 3)).astype(np.int32)
    dev = torch.from_numpy(buf).to(DEV)
    view = dev[:2, 1:11:2].permute(2, 0, 1)  # (axes, B, S), strides (1, 48, 6)
    pos = np.ascontiguousarray(buf[:2, 1:11:2].transpose(2, 0, 1))
    got = run("fwd", x, view, (6, 5, 5), 0, 32, "fp32", order="interleaved")
    check(got, x, pos, (6, 5, 5), 0, 32, "fp32", "fwd", "strided", order="interleaved")


def test_many_tokens_and_a_second_stream():
    x = synth.normal((3, 1001, 7, 96), "fp16", 8)
    pos = np.random.default_rng(2).integers(0, 5000, size=(3, 3, 1001)).astype(np.int32)
    xd, pd = to_dev(x, "fp16"), torch.from_numpy(pos).to(DEV)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    binding.rope_partial_inplace_fwd_axes(xd, pd, (16, 16, 16), 0, 96, mode="half", spectrum="own",
                                          stream=stream)
    stream.synchronize()
    check(synth.from_torch(xd), x, pos, (16, 16, 16), 0, 96, "fp16", "fwd", "stream", mode="half",
          spectrum="own")


def test_empty_calls_change_nothing():
    pos = torch.zeros((2, 1, 1), dtype=torch.int32, device=DEV)
    x = torch.ones((2, 3, 4, 8), device=DEV)
    binding.rope_partial_inplace_fwd_axes(x, pos, (0, 0), 4, 4)
    binding.rope_partial_inplace_bwd_axes(x[:0], pos, (1, 1), 0, 4)
    torch.cuda.synchronize()
    assert torch.equal(x, torch.ones_like(x))


@pytest.mark.parametrize("mode", ["interleave", "half"])
@pytest.mark.parametrize("order", ["blocked", "interleaved"])
def test_gradient_through_autograd(mode, order):
    """x.grad against the formula (the transposed rotation of the upstream
    gradient), and against the difference quotient of the loss along a random
    direction.  The rotation is linear, so the quotient is exact but for
    rounding: each of the two losses sums N products of fp32 values with an
    error of about 1e-6 each (the bar above), all of either sign."""
    rng = np.random.default_rng(11)
    shape, sections = (2, 17, 3, 48), (5, 6, 5)
    x, w, d = (rng.standard_normal(shape).astype(np.float32) for _ in range(3))
    pos = rng.integers(0, 600, size=(3, 2, 17)).astype(np.int32)
    pd = torch.from_numpy(pos).to(DEV)
    kw = dict(partial_slice=[8, 40], rotary_mode=mode, order=order, spectrum="own")

    def loss(t):
        y = t * 1.0
        torch_op.inplace_axes_rotary_mul(y, pd, sections, **kw)
        return (y.double() * torch.from_numpy(w).to(DEV).double()).sum()

    xd = torch.from_numpy(x).to(DEV).requires_grad_(True)
    loss(xd).backward()
    got = xd.grad.cpu().numpy()
    want = ref.axes_rope(w, pos, sections, 8, 40, mode=mode, order=order, spectrum="own", backward=True)
    xm = np.abs(w).astype(np.float64)
    assert np.all(np.abs(got - want) <= 1e-6 * 2 * xm.max() + 1e-6 * np.abs(want))
    h = 0.25
    with torch.no_grad():
        dd = torch.from_numpy(d).to(DEV)
        diff = (loss(xd + h * dd) - loss(xd - h * dd)).item() / (2 * h)
    along = float((want * d).sum())
    n = x.size
    # two losses of n terms, each off by up to 2e-6 |x||w|, over 2 h
    assert abs(diff - along) <= 2 * n * 2e-6 * 4.0 / (2 * h)
    assert abs(diff - along) <= 1e-3 * np.sqrt(n)


def test_gradient_leaves_the_incoming_one_alone():
    x = torch.randn(1, 4, 2, 16, device=DEV, requires_grad=True)
    pos = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 1, 4)
    y = x * 1.0
    y.retain_grad()
    torch_op.inplace_axes_rotary_mul(y, pos, (4, 4), partial_slice=[0, 16])
    y.sum().backward()
    assert torch.equal(y.grad, torch.ones_like(y)) and not torch.equal(x.grad, y.grad)


def test_traced_by_torch_compile():
    pos = torch.arange(10, dtype=torch.int32, device=DEV).view(2, 1, 5)

    def f(t):
        y = t * 1.0
        torch.ops.place_partial_rope.inplace_axes_rotary_mul(y, pos, [4, 4], partial_slice=[0, 16])
        return y

    torch_op.register()
    x = torch.randn(1, 5, 2, 16, device=DEV)
    want = f(x)
    assert torch.equal(torch.compile(f, backend="aot_eager", fullgraph=True)(x), want)
