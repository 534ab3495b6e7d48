"""The paged cache's calls at the edges of what they take."""
import pytest
import torch

import serving_ref as ref
from gpu_util import DEV
from place_partial_rope_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("store", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("dk,dv", [(64, 64), (192, 128), (80, 48)])
def test_keys_and_values_read_into_one_tensor(dk, dv, store):
    """A head's key and value side by side, as one packed tensor holds them."""
    page, heads, T = 16, 3, 37
    k, v = (torch.zeros((4, page, heads, d), device=DEV).to(store) for d in (dk, dv))
    s = [torch.ones((4, page, heads), device=DEV) if store != torch.bfloat16 else None for _ in range(2)]
    cache = binding.KVCache(k, v, *s)
    slots = torch.randperm(4 * page, device=DEV)[:T]
    nk, nv = (torch.randn((T, heads, d), device=DEV).to(torch.bfloat16) for d in (dk, dv))
    binding.rope_partial_cache_write(cache, nk, nv, slots)
    want = [torch.empty_like(t) for t in (nk, nv)]
    binding.rope_partial_cache_read(cache, slots, *want)
    packed = torch.full((T, heads, dk + dv), 7.0, dtype=torch.bfloat16, device=DEV)
    binding.rope_partial_cache_read(cache, slots, packed[..., :dk], packed[..., dk:])
    torch.cuda.synchronize()
    assert torch.equal(packed, torch.cat(want, -1))


@pytest.mark.parametrize("mode", ["interleave", "half"])
@pytest.mark.parametrize("dk,start,end", [(65, 0, 64), (65, 1, 65), (127, 30, 100), (3, 1, 3)])
def test_a_rotation_in_rows_of_an_odd_length(dk, start, end, mode):
    T, heads, L = 19, 2, end - start
    k = torch.zeros((2, 16, heads, dk), dtype=torch.float16, device=DEV)
    new = torch.randn((T, heads, dk), device=DEV)
    cos, sin = torch.rand((T, L), device=DEV), torch.rand((T, L), device=DEV)
    slots = torch.randperm(32, device=DEV)[:T]
    binding.rope_partial_cache_write(binding.KVCache(k), new, None, slots, cos, sin, start, end, mode)
    torch.cuda.synchronize()
    x, c, s = new[..., start:end].cpu().numpy(), cos.cpu().numpy(), sin.cpu().numpy()
    want = new.cpu().numpy().copy()
    want[..., start:end] = ref.rotate_rows_fp32(x, c, s, 0, L, mode)
    assert torch.equal(k.flatten(0, 1)[slots].cpu(), torch.from_numpy(want).half())
