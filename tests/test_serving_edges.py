"""The C ABI of include/rope_serving.h at the edges of what it takes, without a
GPU (see test_serving_boundary.py)."""
import ctypes

import pytest

from place_partial_rope_gb300 import binding
from test_serving_boundary import INVALID, OK, attend, cache, i64, message

I64 = ctypes.c_int64


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def workspace(lib, c, dtype, Hq, max_q):
    n = I64()
    assert lib.rope_partial_tree_attention_workspace(ctypes.byref(c), dtype, Hq, max_q, 152, ctypes.byref(n)) == OK
    return n.value


@pytest.mark.parametrize("store", [0, 3, 4])
def test_a_cache_without_pages_has_one_kernel(lib, store):
    """The one for few query rows, whatever the hint: a tensor map, which the
    others fetch through, cannot be empty."""
    few = workspace(lib, cache(store=3), 0, 2, 1)  # 8-bit, up to 16 query rows a key head: that kernel
    empty = cache(store=store, pages=0, k=None, v=None, k_scale=None, v_scale=None)
    for max_q in (1, 60, 200):
        assert workspace(lib, empty, 0, 2, max_q) == few


@pytest.mark.parametrize("scale", [1e300, 1e39, 3.0e38, 1e-39, 1e-300])
def test_a_scale_that_fp32_does_not_hold_is_refused(lib, scale):
    """The kernels multiply by scale * log2(e) in fp32: infinity times a score of
    0, or 0 times the -inf of a row that is not seen, would be NaN."""
    assert attend(lib, cache(), scale=scale) == INVALID
    assert "scale" in message(lib)
    assert attend(lib, cache(), scale=scale, Tq=0) == INVALID


ONE = [  # a dim of one, with a stride that would break the 16-byte rule
    (dict(), dict(Tq=1, qst=(257, 64))),
    (dict(), dict(Tq=1, ost=(257, 64))),
    (dict(heads=1), dict(Hq=1, Tq=4, qst=(64, 3), ost=(64, 3))),
    (dict(heads=1, k_stride=i64(1024, 64, 1)), dict()),
    (dict(pages=1, v_stride=i64(7, 128, 64)), dict()),
    (dict(page=1, k_stride=i64(128, 9, 64)), dict()),
]


@pytest.mark.parametrize("c,kw", ONE)
def test_the_stride_of_a_dim_of_one_does_not_count(lib, c, kw):
    """(With a workspace of no bytes, so that nothing is launched anywhere.)"""
    assert attend(lib, cache(**c), nbytes=0, **kw) != OK
    assert "16-byte" not in message(lib)


@pytest.mark.parametrize("c,kw", [(dict(), dict(qst=(257, 64))), (dict(k_stride=i64(1031, 64, 64)), dict())])
def test_the_stride_of_other_dims_does(lib, c, kw):
    assert attend(lib, cache(heads=1, **c), nbytes=0, Hq=1, **kw) == INVALID
    assert "16-byte" in message(lib)
