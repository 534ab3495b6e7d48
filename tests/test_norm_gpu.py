"""Norm and rotation in one pass, forward and backward, on the GPU, against the
64-bit formulas.

Bounds.  The kernels compute in fp32 and round once to the storage type (half a
step, eps / 2 of the result).  A sum over a row adds at most 32 terms in a thread
(8 chunks of 4, or 4 of 8), then 5 across lanes: its relative error is below 40 *
2^-24, half of that after the root.  With the products, the table's terms and the
last sums (fewer than 10 roundings) everything before the store is within 2^-18 of
the terms' magnitudes (64 * 2^-24).  A weight's gradient goes through at most
64 additions in a thread for the rows used here, 5 + 8 in a block and 32 + 38 across
at most 1216 blocks: fewer than 256, with its terms' errors below 2^-15.
"""
import numpy as np
import pytest
import torch

import step_ref as ref
from gpu_util import DEV
from place_partial_rope_gb300 import binding, torch_op

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

CASES = [  # B, S, Nq, Nk, D, n0, n1, start, end, mode
    (2, 5, 4, 2, 128, 0, 128, 0, 128, "half"),
    (1, 1, 1, 0, 64, 0, 64, 0, 64, "interleave"),
    (3, 7, 5, 3, 128, 0, 128, 34, 98, "interleave"),  # chunks that the slice cuts
    (1, 19, 1, 0, 576, 0, 512, 512, 576, "interleave"),  # a latent row
    (2, 3, 9, 1, 192, 0, 192, 128, 192, "half"),
    (2, 3, 3, 2, 96, 12, 90, 3, 41, "interleave"),  # odd start, a norm that cuts chunks
    (2, 4, 2, 7, 80, 0, 80, 5, 47, "half"),  # odd start, odd half
    (1, 6, 2, 1, 33, 1, 32, 2, 30, "half"),  # odd rows
    (1, 6, 2, 1, 33, 0, 33, 1, 31, "interleave"),
    (5, 1, 3, 3, 1024, 0, 1024, 0, 1024, "half"),
    (2, 2, 2, 2, 72, 0, 72, 0, 0, "interleave"),  # no rotation
    (4, 33, 8, 2, 256, 0, 256, 0, 64, "half"),
    (2, 3, 1, 1, 1, 0, 1, 0, 0, "half"),  # one lane
    (2, 3, 2, 1, 640, 64, 640, 0, 64, "half"),  # the turned lanes are not the normed ones
]
LAYOUTS = ["dense", "fused", "odd", "batch", "inplace"]


def placed(x, layout):
    """x (B, S, N, D) on the device: dense, one element into its buffer, or with
    space behind each batch."""
    B, S, N, D = x.shape
    if layout == "odd":
        buf = torch.full((B, S, N, D + 3), 7.0, dtype=x.dtype, device=DEV).flatten()
        v = buf[1:].as_strided((B, S, N, D), (S * N * (D + 3), N * (D + 3), D + 3, 1))
    elif layout == "batch":
        v = torch.full((B, S + 2, N, D), 7.0, dtype=x.dtype, device=DEV)[:, :S]
    else:
        v = torch.empty((B, S, N, D), dtype=x.dtype, device=DEV)
    return v.copy_(x)


def make(case, dtype, layout, seed, table="token"):
    B, S, Nq, Nk, D, n0, n1, st, en, mode = case
    g = torch.Generator().manual_seed(seed)
    kind = TYPES[dtype]
    heads = [Nq] + ([Nk] if Nk else [])
    host = [torch.randn((B, S, N, D), generator=g).to(kind) for N in heads]
    if layout == "fused":  # views of one projection's rows, queries and keys between each other
        whole = torch.cat(host + [torch.zeros((B, S, 1, D), dtype=kind)], 2).to(DEV)
        rows, at = [], 0
        for N in heads:
            rows.append(whole[:, :, at:at + N])
            at += N
    else:
        rows = [placed(x, layout) for x in host]
    shape = {"token": (B, S, 1, en - st), "seq": (1, S, 1, en - st), "one": (1, 1, 1, en - st)}[table]
    cos, sin = (torch.randn(shape, generator=g).to(kind) for _ in range(2))
    return host, rows, cos, sin, g


def weights(kind, heads, n, g):
    if kind is None:
        return [None] * len(heads), [None] * len(heads)
    host = [(1 + 0.5 * torch.randn(n, generator=g)).to(kind) for _ in heads]
    return host, [w.to(DEV) for w in host]


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def near(got, want, tol, what):
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), f"{what}: off by up to {np.nanmax(err / np.maximum(tol, 1e-300)):.2f} of the bound"


def half_step(t):
    return torch.finfo(t).eps / 2


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward(case, dtype, layout):
    c = CASES[case]
    B, S, Nq, Nk, D, n0, n1, st, en, mode = c
    kind = TYPES[dtype]
    host, rows, cos, sin, g = make(c, dtype, layout, case, ("token", "seq", "one")[case % 3])
    wtype = (kind, torch.float32, None)[(case + len(layout)) % 3]
    hw, dw = weights(wtype, host, n1 - n0, g)
    outs = [None if layout == "inplace" or (layout == "fused" and case % 2) else placed(torch.zeros_like(x), layout)
            for x in host]
    keep = [torch.full(x.shape[:3], -1.0, device=DEV) if case % 2 else None for x in host]
    before = [x.clone() for x in rows]
    pad = (None,) if Nk == 0 else ()
    binding.rope_partial_norm_fwd(*rows, *pad, *dw, *pad, cos.to(DEV), sin.to(DEV), st, en, eps=1e-5, norm=(n0, n1),
                                  mode=mode, q_out=outs[0], k_out=outs[1] if Nk else None, q_rstd=keep[0],
                                  k_rstd=keep[1] if Nk else None)
    torch.cuda.synchronize()
    for i, x in enumerate(host):
        want, mag, r = ref.norm_fwd(f64(x), f64(hw[i]), f64(cos), f64(sin), st, en, n0, n1, 1e-5, mode)
        got = rows[i] if outs[i] is None else outs[i]
        near(got, want, 2.0 ** -18 * mag + half_step(kind) * np.abs(want) * (1 + 2.0 ** -10) +
             (2.0 ** -25 if dtype == "fp16" else 0), "out")
        if keep[i] is not None:
            near(keep[i], r, 2.0 ** -18 * r, "rstd")
        if outs[i] is not None:
            assert torch.equal(rows[i], before[i])


def run_bwd(c, dtype, layout, seed, wtype, want_w=True, workspace=None):
    B, S, Nq, Nk, D, n0, n1, st, en, mode = c
    kind = TYPES[dtype]
    host, rows, cos, sin, g = make(c, dtype, layout, seed)
    hw, dw = weights(wtype, host, n1 - n0, g)
    hg = [torch.randn(x.shape, generator=g).to(kind) for x in host]
    grads = [placed(x, "dense" if layout == "fused" else layout) for x in hg]
    rstd = [(1.0 / (x[..., n0:n1].double() ** 2).mean(-1).add(1e-5).sqrt()).float() for x in host]
    outs = [None if layout == "inplace" else placed(torch.zeros_like(x), layout) for x in hg]
    gw = [torch.full((n1 - n0,), 9.0, device=DEV) if want_w else None for _ in host]
    pad = (None,) if Nk == 0 else ()
    before = [x.clone() for x in grads]
    binding.rope_partial_norm_bwd(*grads, *pad, *rows, *pad, *dw, *pad, *(x.to(DEV) for x in rstd), *pad, cos.to(DEV),
                                  sin.to(DEV), st, en, norm=(n0, n1), mode=mode, dq_out=outs[0],
                                  dk_out=outs[1] if Nk else None, dq_weight=gw[0],
                                  dk_weight=gw[1] if Nk else None, workspace=workspace)
    torch.cuda.synchronize()
    for i, x in enumerate(host):
        dx, mag, w, wmag = ref.norm_bwd(f64(hg[i]), f64(x), f64(hw[i]), f64(rstd[i]), f64(cos), f64(sin), st, en, n0,
                                        n1, mode)
        near(grads[i] if outs[i] is None else outs[i], dx,
             2.0 ** -18 * mag + half_step(kind) * np.abs(dx) * (1 + 2.0 ** -10) + (2.0 ** -25 if dtype == "fp16" else 0),
             "dx")
        if want_w:
            near(gw[i], w, 2.0 ** -15 * wmag, "dw")
        if outs[i] is not None:
            assert torch.equal(grads[i], before[i])
    return outs, gw


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_backward(case, dtype, layout):
    wtype = (TYPES[dtype], torch.float32, None)[(case + len(layout)) % 3]
    run_bwd(CASES[case], dtype, layout, 100 + case, wtype, want_w=case % 4 != 3)


def test_many_rows_and_the_same_bits_twice():
    c = (3, 1201, 6, 2, 128, 0, 128, 0, 128, "half")
    first = run_bwd(c, "bf16", "dense", 5, torch.float32)
    again = run_bwd(c, "bf16", "dense", 5, torch.float32)
    for a, b in zip(first[0] + first[1], again[0] + again[1]):
        assert torch.equal(a, b)


def test_gradient_against_differences():
    """Along random directions, fp32 rows: the differences are the 64-bit formula's, of
    step 1e-4, off by a term of step^2 (3e-8 of third derivatives of order 1)."""
    B, S, N, D, n0, n1, st, en, mode = 2, 3, 2, 24, 4, 24, 2, 20, "half"
    host, rows, cos, sin, g = make((B, S, N, 0, D, n0, n1, st, en, mode), "fp32", "dense", 3)
    x, w = f64(host[0]), 1 + 0.3 * np.random.default_rng(0).standard_normal(n1 - n0).astype(np.float32)
    gy = torch.randn(host[0].shape, generator=g)
    rstd = torch.empty((B, S, N), device=DEV)
    binding.rope_partial_norm_fwd(rows[0], None, torch.from_numpy(w).to(DEV), None, cos.to(DEV), sin.to(DEV), st, en,
                                  norm=(n0, n1), mode=mode, q_out=torch.empty_like(rows[0]), q_rstd=rstd)
    dx, dw = torch.empty_like(rows[0]), torch.empty(n1 - n0, device=DEV)
    binding.rope_partial_norm_bwd(gy.to(DEV), None, rows[0], None, torch.from_numpy(w).to(DEV), None, rstd, None,
                                  cos.to(DEV), sin.to(DEV), st, en, norm=(n0, n1), mode=mode, dq_out=dx,
                                  dq_weight=dw)

    def loss(x, w):
        return (ref.norm_fwd(x, w, f64(cos), f64(sin), st, en, n0, n1, 1e-6, mode)[0] * f64(gy)).sum()

    rng = np.random.default_rng(1)
    for _ in range(4):
        vx, vw = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        h = 1e-4
        want = (loss(x + h * vx, w + h * vw) - loss(x - h * vx, w - h * vw)) / (2 * h)
        got = (f64(dx) * vx).sum() + (f64(dw) * vw).sum()
        size = np.abs(f64(dx) * vx).sum() + np.abs(f64(dw) * vw).sum()
        assert abs(got - want) <= 1e-5 * size


def test_rows_that_are_not_finite_stay_alone():
    x = torch.randn((1, 64, 2, 128), dtype=torch.float32)
    x[0, 3, 1, 5], x[0, 9, 0, 127] = float("inf"), float("nan")
    out = torch.empty_like(x, device=DEV)
    binding.rope_partial_norm_fwd(x.to(DEV), None, None, None, None, None, 0, 0, q_out=out)
    bad = ~out.isfinite().all(-1).cpu()
    assert bad.nonzero().tolist() == [[0, 3, 1], [0, 9, 0]]


def test_no_rows():
    q = torch.empty((0, 4, 2, 16), device=DEV)
    binding.rope_partial_norm_fwd(q, None, None, None, None, None, 0, 0)
    w, dw = torch.ones(16, device=DEV), torch.full((16,), 3.0, device=DEV)
    binding.rope_partial_norm_bwd(q, None, q, None, w, None, torch.empty((0, 4, 2), device=DEV), None, None, None, 0,
                                  0, dq_weight=dw)
    assert not dw.any()


def test_streams_and_graphs():
    """A backward on a stream of its own, one captured and replayed on other rows, and an
    eager autograd graph of the same leaves alive meanwhile."""
    B, S, N, D = 2, 65, 3, 64
    g = torch.Generator(device=DEV).manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    q, w, cos, sin, dy = normal(B, S, N, D), normal(D), normal(1, S, 1, D), normal(1, S, 1, D), normal(B, S, N, D)
    leaf, wleaf = q.clone().requires_grad_(), w.clone().requires_grad_()
    alive = torch_op.norm_rotary(leaf, None, wleaf, None, cos, sin, partial_slice=[0, D])[0]  # its graph lives on
    rstd, out, dx, dw = torch.empty((B, S, N), device=DEV), torch.empty_like(q), torch.empty_like(q), torch.empty_like(w)
    ws = binding.norm_workspace(q)

    def step():
        binding.rope_partial_norm_fwd(leaf.detach(), None, wleaf.detach(), None, cos, sin, 0, D, q_out=out, q_rstd=rstd)
        binding.rope_partial_norm_bwd(dy, None, leaf.detach(), None, wleaf.detach(), None, rstd, None, cos, sin, 0, D,
                                      dq_out=dx, dq_weight=dw, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    with torch.no_grad():
        leaf.copy_(normal(B, S, N, D))
    graph.replay()
    torch.cuda.synchronize()
    kept = [t.clone() for t in (out, dx, dw)]
    step()
    torch.cuda.synchronize()
    for a, b in zip(kept, (out, dx, dw)):
        assert torch.equal(a, b)
    del alive


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_autograd(dtype):
    """The operator's gradients against torch's of the same formula in 64 bits."""
    B, S, Nq, Nk, D, n0, n1, st, en = 2, 5, 4, 2, 64, 0, 48, 16, 64
    kind = TYPES[dtype]
    g = torch.Generator().manual_seed(2)
    q, k = (torch.randn((B, S, N, D), generator=g).to(kind) for N in (Nq, Nk))
    qw, kw = (1 + 0.2 * torch.randn(n1 - n0, generator=g) for _ in range(2))
    cos, sin = (torch.randn((B, S, 1, en - st), generator=g).to(kind) for _ in range(2))
    leaves = [t.to(DEV).requires_grad_() for t in (q, k, qw, kw)]
    outs = torch_op.norm_rotary(leaves[0], leaves[1], leaves[2], leaves[3], cos.to(DEV), sin.to(DEV),
                                partial_slice=[st, en], norm_slice=[n0, n1], rotary_mode="half")
    up = [torch.randn(o.shape, generator=g).to(kind) for o in outs]
    torch.autograd.backward(outs, [u.to(DEV) for u in up])
    exact = [t.double().requires_grad_() for t in (q, k, qw, kw)]
    half = (en - st) // 2
    for x, w, u in ((exact[0], exact[2], up[0]), (exact[1], exact[3], up[1])):
        r = (x[..., n0:n1].square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        y = torch.cat([x[..., n0:n1] * r * w, x[..., n1:]], -1)
        s = y[..., st:en]
        turned = s * cos.double() + torch.cat([-s[..., half:], s[..., :half]], -1) * sin.double()
        torch.cat([y[..., :st], turned], -1).backward(u.double())
    for got, want in zip(leaves, exact):
        size = want.grad.abs().max().item()
        assert (got.grad.double().cpu() - want.grad).abs().max().item() <= (2 * half_step(got.dtype) + 1e-5) * size
    # sums: an expanded gradient whose last dim has no step
    leaf = q.to(DEV).requires_grad_()
    torch_op.norm_rotary(leaf, None, None, None, None, None)[0].sum().backward()
    assert leaf.grad.isfinite().all()
    with pytest.raises(RuntimeError):  # no second gradients
        leaf = q.to(DEV).requires_grad_()
        y = torch_op.norm_rotary(leaf, None, None, None, None, None)[0]
        (d,) = torch.autograd.grad(y.square().sum(), leaf, create_graph=True)
        d.sum().backward()
