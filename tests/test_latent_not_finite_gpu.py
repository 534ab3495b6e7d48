"""Attention over latent rows with infinities and NaN in drafted rows of chains, long ones too: they
reach the tokens that see them, and nobody else, and do not make the call take for ever."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from test_latent_gpu import Case

pytestmark = pytest.mark.gpu


def spoil(c, rows, lane, what):
    """The value of a lane in some rows (of the one request)."""
    flat = c.k.flatten(0, 2)
    at = torch.from_numpy(c.slots[0][rows]).to(flat.device)
    if c.store == "fp8":
        flat.view(torch.uint8)[at, lane] = 0x7f
    else:
        flat[at, lane] = what


def timed(c):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    c.run(scale=1 / 24)
    a.record()
    got = c.run(scale=1 / 24)
    b.record()
    torch.cuda.synchronize()
    return got, a.elapsed_time(b)


@pytest.mark.parametrize("store,page", [("bf16", 16), ("fp16", 5), ("fp8", 16)])
@pytest.mark.parametrize("n,first", [(40, 11), (300, 200)])
def test_nan_in_a_chain(n, first, store, page):
    dtype = "fp16" if store == "fp16" else "bf16"
    c = Case(dtype, store, [n], [n + 70], 2, 576, 512, page=page, tree=None, seed=n)
    want, want_lse = c.run(scale=1 / 24)
    spoil(c, np.array([70 + first]), 7, float("nan"))
    out, lse = c.run(scale=1 / 24)
    assert torch.equal(out[:first], want[:first]) and torch.equal(lse[:first], want_lse[:first])
    assert torch.isnan(out[first:]).any(-1).all() and torch.isnan(lse[first:]).all()


@pytest.mark.parametrize("store,page,H", [("bf16", 16, 2), ("fp16", 5, 2), ("fp16", 16, 64), ("bf16", 64, 128)])
@pytest.mark.parametrize("n,first", [(40, 11), (300, 200)])
def test_scores_of_minus_infinity_in_a_chain(n, first, store, page, H):
    """An infinite lane that makes the score -inf: a weight of 0, and a result that is not finite in
    that lane alone, for the tokens that see it."""
    c = Case(store, store, [n], [n + 70], H, 576, 512, page=page, tree=None, seed=n)
    c.q[..., 7] = -1.0
    want, want_lse = c.run(scale=1 / 24)
    rows = np.arange(70 + first, 70 + n)
    spoil(c, rows, 7, float("inf"))
    out, lse = c.run(scale=1 / 24)
    assert torch.equal(out[:first], want[:first]) and torch.equal(lse[:first], want_lse[:first])
    assert not torch.isfinite(out[first:, :, 7]).any()
    out = out.clone()
    out[..., 7] = 0
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    # the rows before, in 64 bits (bounds as in test_latent_gpu.py)
    k, q, u = c.numbers()[c.slots[0][:70 + first]], c.q.double().numpy(), 2.0 ** (-8 if store == "bf16" else -11)
    for i in (first, n - 1):
        for h in (0, H - 1):
            o, l, mag = ref.tree_attention(q[i:i + 1, h], k, k[:, :512], np.ones((1, len(k)), bool), 1 / 24)
            d = 584 * 2.0 ** -24 * (np.abs(q[i, h]) @ np.abs(k).T).max() / 24 + 2.0 ** -21
            o[:, 7] = 0
            err = np.abs(out[i, h].double().cpu().numpy() - o[0])
            assert np.all(err <= (u + 4 * d) * mag[0] + u * np.abs(o[0]) + 2.0 ** -32 * len(k) * np.abs(k).max())
            assert abs(lse[i, h].item() - l[0]) <= 2 * d + 2.0 ** -22 * abs(l[0])


@pytest.mark.parametrize("store,what", [("fp8", "nan"), ("bf16", "nan"), ("fp16", "inf")])
def test_a_long_chunk(store, what):
    """20000 tokens of one request, of which one row (or, infinite in a lane, every row from there
    on) is not finite: the others' results stay as they are, and the time does, about."""
    n, first = 20000, 9000
    dtype = "bf16" if store == "fp8" else store
    c = Case(dtype, store, [n], [n], 1, 576, 512, page=64, tree=None, seed=1)
    c.q[..., 7] = -1.0
    (want, want_lse), clean = timed(c)
    assert torch.isfinite(want).all()
    spoil(c, np.arange(first, n if what == "inf" else first + 1), 7, float(what))
    (out, lse), took = timed(c)
    assert torch.equal(out[:first], want[:first]) and torch.equal(lse[:first], want_lse[:first])
    assert not torch.isfinite(out[first:, :, 7]).any()
    assert torch.isnan(lse[first:]).all() if what == "nan" else torch.isfinite(lse).all()
    assert took < 20 * clean + 5, (took, clean)
