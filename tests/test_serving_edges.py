"""The C ABI of include/rope_serving.h at the edges of what it takes, without a
GPU (see test_serving_boundary.py)."""
import ctypes
import random

import pytest
import torch

from place_partial_rope_gb300 import binding
from test_serving_boundary import A, C, INVALID, OK, attend, cache, i64, message

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


def read(lib, k, v, ks, vs, kd=64, vd=64, T=5):
    return lib.rope_partial_cache_read(ctypes.byref(cache(kd=kd, vd=vd)), C, T, k, v, 0, i64(*ks), i64(*vs), None)


# (Only where there is no device: these calls are right, and their addresses made up.)
@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("ks,vs,at,kd,vd", [
    ((256, 128), (256, 128), 128, 64, 64),   # a head's key and value side by side
    ((256, 128), (256, 128), -128, 64, 64),  # the value first
    ((768, 320), (768, 320), 384, 192, 128),
    ((700, 140), (700, 140), 140, 64, 64),   # with gaps
    ((300, 128), (300, 128), 128, 64, 64),   # heads' steps do not end with the token's
])
def test_keys_and_values_that_lie_between_each_other_may_be_read(lib, T, ks, vs, at, kd, vd):
    assert read(lib, A + 4096, A + 4096 + at, ks, vs, kd, vd, T) not in (OK, INVALID)
    assert "overlap" not in message(lib)


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("ks,vs,at,kd,vd", [
    ((256, 128), (256, 128), 126, 64, 64),
    ((256, 128), (256, 128), 130, 64, 64),
    ((256, 128), (128, 64), 128, 64, 64),    # of different steps
    ((300, 128), (300, 128), 400, 64, 64),   # a token's values reach into the next one's keys
    ((768, 320), (768, 320), 382, 192, 128),
])
def test_keys_and_values_that_overlap_may_not(lib, T, ks, vs, at, kd, vd):
    if T == 1 and at == 400:
        return  # one token: apart
    assert read(lib, A + 4096, A + 4096 + at, ks, vs, kd, vd, T) == INVALID
    assert "overlap" in message(lib)


def test_queries_and_results_that_lie_between_each_other(lib):
    assert attend(lib, cache(), qst=(512, 128), out=A + 128, ost=(512, 128), nbytes=0) != OK
    assert "overlap" not in message(lib)
    assert attend(lib, cache(), qst=(512, 128), out=A + 112, ost=(512, 128), nbytes=0) == INVALID
    assert "overlap" in message(lib)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
def test_no_overlap_of_what_is_read_is_missed(lib):
    """Layouts at random against the sets of their bytes."""
    rng = random.Random(3)
    taken = 0
    for _ in range(4000):
        T, heads, kd, vd = (rng.randint(1, n) for n in (4, 4, 6, 6))
        kh = kd + rng.randint(0, 8)
        vh = rng.choice([kh, kh, vd + rng.randint(0, 8)])
        kt = rng.choice([heads * kh, heads * 14, max(kd, rng.randint(0, 60))])
        vt = rng.choice([kt, kt, max(vd, rng.randint(0, 60))])
        if vh < vd or kt < kd or vt < vd:
            continue  # (refused for another reason)
        at = rng.randint(-80, 80)

        def places(p, t, h, d):
            return {p + i * t + j * h + x for i in range(T) for j in range(heads) for x in range(d)}

        shared = bool(places(0, kt, kh, kd) & places(at, vt, vh, vd))
        c = cache(heads=heads, kd=kd, vd=vd)
        st = lib.rope_partial_cache_read(ctypes.byref(c), C, T, A + 8192, A + 8192 + 2 * at, 0, i64(kt, kh), i64(vt, vh),
                                         None)
        assert not (shared and st != INVALID), (T, heads, (kt, kh, kd), (vt, vh, vd), at)
        taken += st != INVALID
    assert taken > 1500
