"""What the attention over latent rows refuses, without a GPU."""
import ctypes

import pytest

from place_partial_rope_gb300 import binding

OK, NULL, INVALID = 0, 1, 2
K, KS, Q, OUT, QS, LEN, TAB, TREE, LSE, WS = (0x10000000 + (i << 36) for i in range(10))
I64 = ctypes.c_int64


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def message(lib):
    return lib.rope_last_error_message().decode()


def cache(store=0, pages=8, page=16, heads=1, kd=576, v=None, vd=0, **kw):
    st = (I64 * 3)(page * heads * kd, heads * kd, kd)
    one = (I64 * 3)(page * heads, heads, 1)
    c = binding.RopeKVCache(K, v, None if store < 2 else KS, None, pages, page, heads, kd, vd, st, st, one, one, store, 0)
    for name, value in kw.items():
        setattr(c, name, value)
    return c


def call(lib, c=None, q=Q, dtype=0, Tq=4, Hq=8, vd=512, qst=(8 * 576, 576), qs=QS, ln=LEN, R=2, max_q=3, tab=TAB,
         pages=6, stride=6, tree=TREE, words=1, out=OUT, ost=(8 * 512, 512), lse=LSE, scale=0.1, ws=WS, wsn=1 << 34):
    c = cache() if c is None else c
    i2 = I64 * 2
    return lib.rope_partial_latent_attention(ctypes.addressof(c), q, dtype, Tq, Hq, vd, i2(*qst), qs, ln, R, max_q, tab,
                                             pages, stride, tree, words, out, i2(*ost), lse, scale, ws, wsn, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=2), INVALID, "bf16 (0) or fp16 (1)"),
    (dict(dtype=1), INVALID, "type of q"),
    (dict(vd=0), INVALID, "multiples of 16"),
    (dict(vd=24), INVALID, "multiples of 16"),
    (dict(vd=528), INVALID, "multiples of 16"),
    (dict(Hq=0), INVALID, "Hq"),
    (dict(max_q=0), INVALID, "max_q"),
    (dict(Tq=-1), INVALID, "Tq"),
    (dict(R=(1 << 24) + 1), INVALID, "R="),
    (dict(pages=1 << 28, stride=1 << 28), INVALID, "2^31"),
    (dict(stride=5), INVALID, "page_table_stride"),
    (dict(words=0), INVALID, "tree_words"),
    (dict(scale=0.0), INVALID, "scale"),
    (dict(scale=float("nan")), INVALID, "scale"),
    (dict(scale=1e39), INVALID, "scale"),
    (dict(q=0), NULL, "q, out"),
    (dict(tab=0), NULL, "page_table"),
    (dict(ws=0), NULL, "workspace"),
    (dict(q=Q + 8), INVALID, "16-byte"),
    (dict(qst=(8 * 576, 580)), INVALID, "16-byte"),
    (dict(ost=(8 * 512, 496)), INVALID, "apart"),
    (dict(out=Q), INVALID, "overlap"),
    (dict(out=K), INVALID, "overlap"),
    (dict(lse=OUT + 64), INVALID, "overlap"),
    (dict(ws=LEN & ~15), INVALID, "overlap"),
    (dict(lse=LSE + 2), INVALID, "aligned"),
])
def test_refusals(lib, kw, status, needle):
    assert call(lib, **kw) == status
    assert needle in message(lib)


@pytest.mark.parametrize("kw,needle", [
    (dict(heads=2), "one head"),
    (dict(v=K + (1 << 30), vd=64), "one head"),
    (dict(kd=592), "576"),
    (dict(kd=520), "multiples of 16"),
])
def test_caches_that_it_does_not_take(lib, kw, needle):
    assert call(lib, c=cache(**kw)) == INVALID
    assert needle in message(lib)


def test_empty_calls(lib):
    assert call(lib, Tq=0, q=0, out=0) == OK
    assert call(lib, R=0, tab=0) == OK


def test_workspace(lib):
    n = I64()
    ref = ctypes.byref(n)
    for store, H, most, rows in ((0, 16, 1, 16), (3, 16, 2, 32), (4, 128, 1, 64)):
        c = cache(store=store)
        assert lib.rope_partial_latent_attention_workspace(ctypes.addressof(c), 0, H, 512, most, 152, ref) == OK
        assert n.value >= 2 * 152 * rows * (512 * 4 + 8)
    c = cache()
    assert lib.rope_partial_latent_attention_workspace(ctypes.addressof(c), 0, 16, 512, 1, -1, ref) == INVALID
    assert lib.rope_partial_latent_attention_workspace(ctypes.addressof(c), 0, 16, 512, 1, 152, None) == NULL
