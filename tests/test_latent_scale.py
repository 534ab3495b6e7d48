"""The scale of attention over latent rows: it is that of the heads' own query rows, which a call
without one does not know, and so says."""
import types
import warnings

import pytest
import torch

from place_partial_rope_gb300 import binding

DEV = "cuda"


def refused(**kw):
    """A call whose q has the wrong width: refused behind the look at the scale."""
    cache = types.SimpleNamespace(device=torch.device("cpu"), k_dim=576)
    with pytest.raises(binding.RopeError, match="576"):
        binding.rope_partial_latent_attention(torch.zeros(1, 2, 64, dtype=torch.bfloat16), cache, None, None, None,
                                              torch.zeros(1, 2, 512, dtype=torch.bfloat16), **kw)


def test_a_call_without_a_scale_warns():
    with pytest.warns(UserWarning, match=r"1 / sqrt\(576\)"):
        refused()


def test_a_call_with_a_scale_does_not():
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        refused(scale=192 ** -0.5)


@pytest.mark.gpu
def test_heads_multiplied_into_the_queries():
    """Heads of 128 + 64 lanes, keys and values made from latent rows of 512 lanes and 64 that
    all heads share: attention of the expanded heads, in 64 bits, and of the latent rows."""
    g = torch.Generator().manual_seed(3)
    H, n, page = 4, 300, 64
    up_k, up_v = (torch.randn((H, 128, 512), generator=g, dtype=torch.float64) / 512 ** 0.5 for _ in range(2))
    rows = torch.randn((5, page, 1, 576), generator=g).to(torch.bfloat16)
    row = rows.flatten(0, 2)[:n].double()
    own = torch.randn((2, H, 192), generator=g, dtype=torch.float64)
    q = torch.cat([torch.einsum("thd,hdc->thc", own[..., :128], up_k), own[..., 128:]], -1).to(torch.bfloat16)
    # what the heads' own rows would be for those (rounded) queries
    s = torch.einsum("thc,jc->thj", q[..., :512].double(), row[:, :512])
    s += torch.einsum("thc,jc->thj", q[..., 512:].double(), row[:, 512:])
    s *= 192 ** -0.5
    s[0, :, n - 1] = -torch.inf  # the first of two new tokens does not see the second
    p = s.softmax(-1)
    want = torch.einsum("thj,jc,hdc->thd", p, row[:, :512], up_v)
    i32 = dict(dtype=torch.int32, device=DEV)
    out = torch.empty((2, H, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((2, H), device=DEV)
    binding.rope_partial_latent_attention(q.to(DEV), binding.KVCache(rows.to(DEV)), torch.tensor([0, 2], **i32),
                                          torch.tensor([n], **i32), torch.arange(5, **i32)[None], out, lse=lse,
                                          scale=192 ** -0.5, max_q=2)
    got = torch.einsum("thc,hdc->thd", out.cpu().double(), up_v)
    # weights and results rounded once each to bf16: 2^-8 of the sums of sizes, and what those come
    # to through up_v; a score's fp32 sum of 576 products adds (576 + 8) 2^-24 of its size, twice
    mag = torch.einsum("thj,jc->thc", p, row[:, :512].abs())
    big = 192 ** -0.5 * torch.einsum("thc,jc->thj", q.double().abs(), row.abs()).amax(-1, keepdim=True)
    tol = (2 * 2.0 ** -8 + 4 * (584 * 2.0 ** -24 * big + 2.0 ** -21)) * mag
    assert ((got - want).abs() <= torch.einsum("thc,hdc->thd", tol, up_v.abs())).all()
    want = torch.logsumexp(s, -1)
    assert ((lse.cpu().double() - want).abs() <= 2 * (584 * 2.0 ** -24 * big[..., 0] + 2.0 ** -21) + 2.0 ** -22 * want.abs()).all()
