"""Attention over latent rows: a weight that stands alone, or outweighs the others, is not rounded."""
import numpy as np
import pytest
import torch

from gpu_util import DEV
from place_partial_rope_gb300 import binding
from test_latent_gpu import PAIRS, Case

pytestmark = pytest.mark.gpu


def is_row(c, out, row):
    """out (..., dv) is the row's values, rounded once (8-bit: after a product with a scale that the
    result has from sums in fp32, so that a value near the middle of a step may fall to either side)."""
    want = torch.from_numpy(c.numbers()[row, :c.dv]).to(DEV)
    if c.store not in ("fp8", "int8"):
        assert (out == want.to(out.dtype)).all()
    step = torch.finfo(out.dtype).eps / 2 * (1 + 2.0 ** -7)
    assert ((out.double() - want).abs() <= step * want.abs() + 2.0 ** -25).all()


@pytest.mark.parametrize("dtype,store", PAIRS)
@pytest.mark.parametrize("H", [1, 16, 40, 128])
def test_one_row(H, dtype, store):
    """A mean of one row is that row, whatever its score."""
    for seed in range(3):
        c = Case(dtype, store, [1], [1], H, 576, 512, page=16, seed=seed, scale_of_q=[1.0, 1.5, 0.3][seed])
        out, _ = c.run(scale=1 / 24)
        is_row(c, out, c.slots[0][0])


@pytest.mark.parametrize("dtype,store", PAIRS)
@pytest.mark.parametrize("length,at", [(20, 3), (64, 63), (300, 17), (300, 250), (20011, 15000)])
def test_a_row_that_outweighs_the_others(length, at, dtype, store):
    """Weights of 2^-60 and less beside it, in its tile and in others, in one part and in several."""
    c = Case(dtype, store, [1], [length], 16, 576, 512, page=64, tree=None, seed=length)
    row = c.slots[0][at]
    best = torch.from_numpy(c.numbers()[row]).to(DEV)
    c.q[:] = (best / best.norm() * 40).to(c.q.dtype).cpu()
    s = torch.from_numpy(c.numbers()[c.slots[0]]).to(DEV) @ c.q[0, 0].to(DEV).double()
    gap = (s[at] - s[torch.arange(length, device=DEV) != at].max()).item()
    out, lse = c.run(scale=60 / gap)
    is_row(c, out, row)
    assert abs(lse[0, 0].item() - 60 * s[at].item() / gap) <= 584 * 2.0 ** -23 * 60 * (c.q[0, 0].double().abs() @ best.cpu().abs()).item() / gap + 1e-5
