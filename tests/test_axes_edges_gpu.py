"""The positions call with several axes at the edges of its promises."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, to_dev
from place_partial_rope_gb300 import binding, synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["interleave", "half"])
@pytest.mark.parametrize("spectrum", ["shared", "own"])
@pytest.mark.parametrize("L", [64, 96, 128, 200, 1022])
def test_one_axis_is_the_positions_call_to_the_bit(L, spectrum, mode):
    """Far positions, where the last bits of a frequency count, in fp32."""
    x = synth.normal((1, 400, 2, 1024), "fp32", L)
    pos = np.random.default_rng(L).integers(2 ** 22, 2 ** 24, size=(1, 1, 400)).astype(np.int32)
    for base in (10000.0, 500000.0):
        one, many = to_dev(x, "fp32"), to_dev(x, "fp32")
        binding.rope_partial_inplace_fwd_axes(one, torch.from_numpy(pos).to(DEV), (L // 2,), 0, L, base=base,
                                              mode=mode, spectrum=spectrum)
        binding.rope_partial_inplace_fwd_pos(many, torch.from_numpy(pos[0]).to(DEV), 0, L, base, mode)
        torch.cuda.synchronize()
        assert torch.equal(one, many), (L, base)


def test_equal_positions_on_all_axes_are_the_positions_call_to_the_bit():
    """A text token among patches: the axes share one spectrum out."""
    x = synth.normal((1, 400, 2, 128), "fp32", 1)
    pos = np.random.default_rng(1).integers(2 ** 22, 2 ** 24, size=(1, 1, 400)).astype(np.int32)
    one, many = to_dev(x, "fp32"), to_dev(x, "fp32")
    binding.rope_partial_inplace_fwd_axes(one, torch.from_numpy(np.repeat(pos, 3, 0)).to(DEV), (24, 20, 20), 0, 128)
    binding.rope_partial_inplace_fwd_pos(many, torch.from_numpy(pos[0]).to(DEV), 0, 128)
    torch.cuda.synchronize()
    assert torch.equal(one, many)
