"""Attention over latent rows with 128 query heads and more: a request's row tiles come in
pairs, which two blocks walk in step.  Against the same sums in 64 bits."""
import numpy as np
import pytest
import torch

from test_latent_gpu import Case

pytestmark = pytest.mark.gpu
HEADS = [0, 63, 64, 127]


@pytest.mark.parametrize("store,page", [("bf16", 64), ("bf16", 16), ("bf16", 10), ("fp8", 32)])
@pytest.mark.parametrize("n", [1, 3])
def test_long_contexts(store, page, n):
    """Both tiles of a pair are split over many blocks and joined."""
    c = Case("bf16", store, [n, 2], [5000, 20011], 128, 576, 512, page=page, seed=n)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(*a, heads=HEADS)


@pytest.mark.parametrize("store,H", [("bf16", 128), ("int8", 128), ("fp16", 256), ("bf16", 192)])
def test_many_requests(store, H):
    """Whole runs, parts and requests without rows or tokens (192 heads: no pairs)."""
    rng = np.random.default_rng(H)
    ns = rng.integers(1, 4, 200).tolist()
    lens = [n + int(x) for n, x in zip(ns, np.exp(rng.uniform(0, 6, 200)))]
    for r in range(3, 200, 31):
        lens[r] = int(rng.integers(4000, 5000))
    ns[10] = ns[11] = 0
    lens[11] = 0
    c = Case("fp16" if store == "fp16" else "bf16", store, ns, lens, H, 128, 64, page=16, seed=H)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(*a, heads=[*HEADS, H - 1])


def test_one_short_request():
    c = Case("bf16", "bf16", [1], [70], 128, 576, 512, page=16, seed=1)
    c.check(*c.run())
