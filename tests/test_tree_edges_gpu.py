"""Attention over the cache at the edges of its numerics: against 64 bits with
the bounds of test_tree_gpu.py, or bit for bit against a call without the edge."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from gpu_util import DEV
from place_partial_rope_gb300 import binding
from test_tree_gpu import Case

pytestmark = pytest.mark.gpu


def numbers(codes, scale, store):
    """Rows as 64-bit numbers from what the device holds."""
    c = codes.view(torch.uint8).flatten(0, 1).cpu().numpy()
    num = ref.fp8_values()[c] if store == "fp8" else c.view("int8").astype("float64")
    with np.errstate(invalid="ignore"):
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
    c.ns = c.ns[:24]  # of these, which are like the others
    c.check(out, lse, scale=1.0)


# tokens, query heads, lanes: the narrow kernel, and tiles of 64, 128 and 256 rows
ROWS = [(6, 2, 128), (6, 1, 256), (15, 1, 64), (30, 1, 64), (30, 2, 128), (25, 4, 128), (40, 4, 64)]


def one_row_apart(store, n, G, d, spoil):
    """A call in which only token 3 sees row prefix + 3, whose bytes `spoil`
    changes (page and place given); its results and those without the change."""
    got = []
    for spoilt in (True, False):
        c = Case("bf16", store, [n], [n + 270], 1, G, d, d, page=16, seed=n + G)
        # token i hangs on i - 1, but for token 3, which hangs on the context and has no children
        c.words = binding.rope_partial_tree_mask([-1, 0, 1, -1] + [2 if i == 4 else i - 1 for i in range(4, n)]).numpy()
        if spoilt:
            spoil(c, *divmod(int(c.slots[0][270 + 3]), c.page))
        got.append((c, *c.run()))
    keep = [i for i in range(n) if i != 3]
    (c, out, lse), (_, want, want_lse) = got
    assert torch.isfinite(want).all() and torch.isfinite(want_lse).all()
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])
    assert (lse[3] - want_lse[3]).abs().max() <= 1e-5  # the keys are as they were
    return c, out


@pytest.mark.parametrize("store", ["fp8", "int8"])
@pytest.mark.parametrize("n,G,d", ROWS)
@pytest.mark.parametrize("scale", [float("inf"), 1e30, 2.0 ** 60, 3e38])
def test_a_value_scale_that_others_do_not_see(n, G, d, scale, store):
    """An infinite or huge scale of a drafted row changes no token that does not
    see the row; the one that does gets what the row says.  Its bound: a weight
    is off by u of the largest product of weight and scale, so a result by u of
    the largest sum over columns."""
    def spoil(c, page, off):
        c.vs[page, off] = scale
        c.rows["v"] = numbers(c.v, c.vs, store)

    c, out = one_row_apart(store, n, G, d, spoil)
    if scale > 1e38:  # infinity, or numbers past bf16's range
        assert not torch.isfinite(out[3]).all()
        return
    sees = ref.tree_sees(n, c.lens[0], 270, c.words)[3:4]
    for h in range(G):
        q = c.q[3:4, h].double().numpy()
        k, v = (c.rows[x][c.slots[0], 0] for x in ("k", "v"))
        o, _, mag = ref.tree_attention(q, k, v, sees, d ** -0.5)
        big = d ** -0.5 * (abs(q) @ abs(k).T).max()
        e = (d + 8) * 2.0 ** -24 * big + 2.0 ** -21
        err = abs(out[3, h].double().cpu().numpy() - o[0])
        assert (err <= (2.0 ** -11 + 4 * e) * mag.max() + 2.0 ** -8 * abs(o[0])).all()


@pytest.mark.parametrize("n,G,d", ROWS)
@pytest.mark.parametrize("code", [0x7f, 0xff])
def test_a_code_of_nan_that_others_do_not_see(n, G, d, code):
    """e4m3 codes of NaN in a drafted row's values: the token that sees them gets
    NaN in their columns, and nobody else does."""
    def spoil_values(c, page, off):
        c.v.view(torch.uint8)[page, off, :, 1::2] = code

    _, out = one_row_apart("fp8", n, G, d, spoil_values)
    assert torch.isnan(out[3, :, 1::2]).all() and torch.isfinite(out[3, :, 0::2]).all()


@pytest.mark.parametrize("store", ["bf16", "fp8"])
@pytest.mark.parametrize("n,G", [(2, 2), (30, 1), (40, 4)])
def test_a_cache_without_pages(n, G, store):
    """No rows at all, and (every page number lying outside) rows of zeros."""
    dtype = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}[store]
    k, v = (torch.empty((0, 16, 1, 64), dtype=dtype, device=DEV) for _ in range(2))
    s = [torch.empty((0, 16, 1), device=DEV) if store == "fp8" else None for _ in range(2)]
    cache = binding.KVCache(k, v, *s)
    q = torch.randn((n, G, 64), device=DEV).to(torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    for length, width in ((0, 0), (0, 4), (n, 4)):
        out, lse = torch.full_like(q, 7.0), torch.full((n, G), 7.0, device=DEV)
        binding.rope_partial_tree_attention(q, cache, i32(0, n), i32(length),
                                            torch.zeros((1, width), dtype=torch.int32, device=DEV), out, lse=lse)
        torch.cuda.synchronize()
        assert not out.any()
        if length == 0:
            assert torch.isneginf(lse).all()
        else:  # a chain: token i sees i + 1 rows with a score of 0
            want = torch.log(torch.arange(1, n + 1, device=DEV).double())[:, None].expand(n, G)
            assert (lse.double() - want).abs().max() <= 2.0 ** -20


@pytest.mark.parametrize("store", ["bf16", "fp16", "fp8", "int8"])
@pytest.mark.parametrize("n,G", [(2, 2), (30, 1), (40, 4)])
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -120])
def test_scores_of_nearly_zero(n, G, scale, store):
    """A scale so small that every score is 0 to fp32, with queries of zeros among
    the others: the mean of the rows that a token sees."""
    dtype = "fp16" if store == "fp16" else "bf16"
    c = Case(dtype, store, [n], [n + 90], 1, G, 64, 64, page=16, seed=n)
    c.q[0] = 0
    c.check(*c.run(scale=scale), scale=scale)


@pytest.mark.parametrize("n,G", [(2, 2), (30, 1), (40, 4)])
def test_large_scales_and_queries_of_zeros(n, G):
    """8-bit: a query row's power of two times the scale stays a number."""
    c = Case("bf16", "fp8", [n], [n + 90], 1, G, 64, 64, page=16, seed=n)
    c.q[:] = 0
    c.check(*c.run(scale=2.0 ** 100), scale=2.0 ** 100)
    c.q[:, :, 0] = 2.0 ** 100  # scores past fp32, but the keys' lane is 0
    c.k.view(torch.uint8)[..., 0] = 0
    c.rows["k"][..., 0] = 0
    c.check(*c.run(scale=2.0 ** 100), scale=2.0 ** 100)


@pytest.mark.parametrize("store", ["bf16", "fp8"])
@pytest.mark.parametrize("G", [2, 40])
def test_strides_of_dims_of_one(G, store):
    """One token, one key head and one page, whose strides are no multiples of
    anything: results, and rows written and read, as with the usual ones."""
    c = Case("bf16", store, [1], [60], 1, G, 64, 64, page=64, tree=None, seed=G, spare=0)
    want, _ = c.run()

    def odd(t, dims):
        st = [101 + 2 * i if i in dims else s for i, s in enumerate(t.stride())]
        return t.as_strided(t.shape, st)

    q, qs, ln, table, _ = c.device()
    k, v = odd(c.k, (0, 2)), odd(c.v, (0, 2))
    ks, vs = (None, None) if c.ks is None else (odd(c.ks, (0, 2)), odd(c.vs, (0, 2)))
    cache = binding.KVCache(k, v, ks, vs)
    out = torch.empty((1, G, 64), dtype=torch.bfloat16, device=DEV)
    binding.rope_partial_tree_attention(odd(q, (0,)), cache, qs, ln, table, odd(out, (0,)), max_q=1)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    slot = torch.tensor([61], device=DEV)
    rows = [torch.randn((1, 1, 64), device=DEV).to(torch.bfloat16) for _ in range(2)]
    binding.rope_partial_cache_write(cache, odd(rows[0], (0, 1)), odd(rows[1], (0, 1)), slot)
    a, b = ([torch.empty_like(r) for r in rows] for _ in range(2))
    binding.rope_partial_cache_read(cache, slot, odd(a[0], (0, 1)), odd(a[1], (0, 1)))
    binding.rope_partial_cache_read(c.cache, slot, *b)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for x, y in zip(a, rows):
        assert (x.double() - y.double()).abs().max() <= 2.0 ** -4 * y.abs().max()


def test_a_call_of_seconds():
    """A run of a block that takes longer than any wait inside the kernel may
    stand still: 152 tokens of 256 heads over 2^29 rows (one page, over and over).
    The bound is loose: 2^22 fp32 sums of one thread follow each other, each rounded
    by up to 2^-24 of the sum, so l and O are within a quarter."""
    n, G, page = 152, 256, 4096
    length = 2 ** 29
    dtype = torch.bfloat16
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn((1, page, 1, 64), generator=g).to(torch.float16).to(DEV) for _ in range(2))
    cache = binding.KVCache(k.to(dtype), v.to(dtype))
    q = (torch.randn((n, G, 64), generator=g) / 8).to(DEV, torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty((n, G), device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    table = torch.zeros((1, length // page), dtype=torch.int32, device=DEV)
    binding.rope_partial_tree_attention(q, cache, i32(0, n), i32(length), table, out, lse=lse, scale=1.0)
    torch.cuda.synchronize()
    kk, vv = (t.to(dtype).to(torch.float16).double()[0, :, 0] for t in (k, v))
    s = q.double() @ kk.T
    assert (lse.double() - torch.logsumexp(s, -1) - np.log(length / page)).abs().max() <= -np.log(0.75)
    assert (out.double() - s.softmax(-1) @ vv).abs().max() <= 0.5 / 0.75 * vv.abs().max()
