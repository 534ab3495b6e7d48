"""Attention over latent rows whose page table names pages that there are not, in long contexts: their rows
are zeros, as short ones' are."""
import numpy as np
import pytest
import torch

from place_partial_rope_gb300 import binding
from test_latent_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("store,page", [("bf16", 64), ("fp16", 128), ("bf16", 16), ("fp16", 20), ("fp8", 64)])
@pytest.mark.parametrize("H", [4, 128])
def test_pages_outside_the_cache(store, page, H):
    dtype = "fp16" if store == "fp16" else "bf16"
    c = Case(dtype, store, [2], [20011], H, 576, 512, page=page, tree=None, seed=H)
    per = -(-20011 // page)
    bad = np.random.default_rng(1).permutation(per - 1)[:per // 3]
    spare = sorted(set(range(c.k.shape[0])) - set(c.table[0].tolist()))[0]
    if c.ks is not None:
        c.ks[spare] = 0.0
    c.k.view(torch.uint8)[spare].zero_()
    got = []
    for outside in (True, False):
        table = c.table.copy()
        table[0, bad] = np.resize(np.array([2 ** 31 - 1, -1, c.k.shape[0], -2 ** 31], np.int32), len(bad)) if outside else spare
        q, qs, ln, _, _ = c.device()
        out, lse = torch.empty((2, H, 512), dtype=q.dtype, device=q.device), torch.empty((2, H), device=q.device)
        binding.rope_partial_latent_attention(q, c.cache, qs, ln, torch.from_numpy(table).to(q.device), out, lse=lse,
                                              scale=1 / 24, max_q=2)
        got.append((out, lse))
    torch.cuda.synchronize()
    assert torch.isfinite(got[0][0]).all()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
