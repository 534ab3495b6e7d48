"""The example that runs the serving operators together, end to end against 64
bits from what went in: rotated rows through the quantised cache to the
attention and back.

Bounds: a rotated value is off by its output type's rounding (2^-8 bf16) of the
pair's size; a code by half a step, which is at most 2^-4 of the value or 2^-10
of the row's largest number over 448.  The attention is compared with the
cache as it is, by the bounds of tests/test_tree_gpu.py.
"""
import importlib.util
import math
import os

import numpy as np
import pytest

import serving_ref as ref

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tree_decode.py")
    spec = importlib.util.spec_from_file_location("tree_decode", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("seed", [0, 1])
def test_example(seed):
    ex = example()
    r = ex.run(seed)
    num = lambda t: t.double().cpu().numpy()  # noqa: E731
    raw, keys = num(r["raw_keys"]), num(r["keys"])
    want = ref.axes_rope(raw[None], r["positions"].numpy()[:, None], ex.SECTIONS, *ex.SLICE)[0]
    size = np.abs(raw) + np.abs(raw.reshape(*raw.shape[:-1], -1, 2)[..., ::-1].reshape(raw.shape))
    assert np.all(np.abs(keys - want) <= 2.0 ** -8 * size)

    # what the cache holds of both requests' rows: the written rows, to half a code
    def stored(new, drafts):
        x = np.concatenate([num(new), num(drafts)])
        codes, scale = ref.quantise_fp32(x.astype(np.float32), "fp8")
        y = ref.fp8_values()[codes] * scale.astype(np.float64)[..., None]
        top = np.abs(x).max(-1, keepdims=True)
        assert np.all(np.abs(y - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 / 448 * top + 1e-6 * top)
        return y[:len(new)], y[len(new):]

    k, new_k = stored(r["keys"], r["new_k"])
    v, new_v = stored(r["values"], r["new_v"])
    q, out, lse = num(r["q"]), num(r["out"]), num(r["lse"])
    scale, group, c0, d0 = 1 / math.sqrt(ex.DIM), ex.HEADS_Q // ex.HEADS_K, 0, 0
    for tree, c, d in zip(r["parents"], r["context"], r["drafted"]):
        rows_k, rows_v = (np.concatenate([a[c0:c0 + c], b[d0:d0 + d]]) for a, b in ((k, new_k), (v, new_v)))
        sees = np.zeros((d, c + d), bool)
        sees[:, :c] = True
        for i, p in enumerate(tree):
            sees[i, c:] = False if p < 0 else sees[p, c:]
            sees[i, c + i] = True
        for h in range(ex.HEADS_Q):
            kk, vv = rows_k[:, h // group], rows_v[:, h // group]
            o, l, mag = ref.tree_attention(q[d0:d0 + d, h], kk, vv, sees, scale)
            big = scale * (np.abs(q[d0:d0 + d, h]) @ np.abs(kk).T).max(-1)
            e = ((ex.DIM + 8) * 2.0 ** -24 * big + 2.0 ** -21)[:, None]
            assert np.all(np.abs(out[d0:d0 + d, h] - o) <= (2.0 ** -11 + 4 * e) * mag + 2.0 ** -8 * np.abs(o) + 1e-30)
            assert np.all(np.abs(lse[d0:d0 + d, h] - l) <= 2 * e[:, 0] + 2.0 ** -22 * np.abs(l))
        c0, d0 = c0 + c, d0 + d

    # the accepted branch comes back as the numbers that the cache holds
    for got, held in ((r["kept_k"], new_k), (r["kept_v"], new_v)):
        want = held[[0, 1, 3]]
        assert np.all(np.abs(num(got) - want) <= 2.0 ** -8 * np.abs(want))
