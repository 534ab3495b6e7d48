"""Attention over the cache at the edges of its numerics: against 64 bits with
the bounds of test_tree_gpu.py, or bit for bit against a call without the edge."""
import pytest
import torch

import serving_ref as ref
from gpu_util import DEV
from test_tree_gpu import Case

pytestmark = pytest.mark.gpu


def numbers(codes, scale, store):
    """Rows as 64-bit numbers from what the device holds."""
    c = codes.view(torch.uint8).flatten(0, 1).cpu().numpy()
    num = ref.fp8_values()[c] if store == "fp8" else c.view("int8").astype("float64")
    return num * scale.flatten(0, 1).double().cpu().numpy()[..., None]


@pytest.mark.parametrize("store", ["fp8", "int8"])
@pytest.mark.parametrize("G,d", [(40, 128), (100, 128), (200, 64)])
def test_a_value_scale_and_a_score_that_grow_in_one_tile(G, d, store):
    """Row 400 of each request has a score 2^10 above the rows before it, and
    values of a scale 2^20 above theirs: O and l of the tiles before shrink by
    both factors in one step, in tiles of 64, 128 and 256 query rows.  (Codes of
    1 in that row: it leads in every column, so that no column is made of weights
    below fp16's range, which the bounds do not cover.)  Requests enough that a
    block has a request's tiles to itself."""
    R, length = 210, 900
    c = Case("bf16", store, [1] * R, [length] * R, 1, G, d, d, page=64, tree=None, seed=G)
    c.q[..., 0] = 8.0
    slots = torch.tensor([int(s[400]) for s in c.slots], device=DEV)
    one = torch.tensor([1]).to(c.k.dtype).view(torch.uint8).item()
    k, v = (t.view(torch.uint8).flatten(0, 1) for t in (c.k, c.v))
    k[..., 0] = 0
    k[slots] = 0
    k[slots, :, 0] = one
    v[slots] = one
    c.ks *= 2.0 ** -6  # scores near 0
    c.ks.flatten(0, 1)[slots] = 7.0 / 8.0  # 7 nats, as q has 8 in that lane
    c.vs.flatten(0, 1)[slots] *= 2.0 ** 20
    c.rows = {"k": numbers(c.k, c.ks, store), "v": numbers(c.v, c.vs, store)}
    out, lse = c.run(scale=1.0)
    c.check(out, lse, scale=1.0)
