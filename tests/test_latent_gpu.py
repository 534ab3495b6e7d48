"""Attention over a paged cache of latent rows, against the same sums in 64 bits over the
rows that a token sees.

Bounds, per element, with u = 2^-8 (bf16 products) or 2^-11 (fp16 products), u_out the
output type's, and A = sum_j p_j |v_j| / sum_j p_j:
  |out - exact| <= (u + 4 d) A + u_out |exact| + tiny,
  |lse - exact| <= 2 d + 2^-22 |exact|,
d bounding the error of a score as in test_tree_gpu.py: the fp32 sum of dk products, each
exact in fp32, is off by at most dk 2^-24 of the sum of their sizes, the scales and base-2
steps by 8 2^-24 of it, 2^x by 2^-22.  u counts the one rounding of p (with the row's
scale); a weight below fp16's normal range is off by 2^-25 of the largest weight's unit,
2^-25 / 2^7 of the largest weight: `tiny` counts that for each row.
"""
import math

import numpy as np
import pytest
import torch

import serving_ref as ref
from gpu_util import DEV
from place_partial_rope_gb300 import binding

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
STORES = {**TYPES, "fp8": torch.float8_e4m3fn, "int8": torch.int8}


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Case:
    """Requests with given drafts and cache lengths, in pages in random order; what no
    request owns (other pages, the ends of last pages) is NaN."""

    def __init__(self, dtype, store, ns, lens, H, dk, dv, page, tree="random", seed=0, pad=0, scale_of_q=1.0, spare=3):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.dtype, self.store, self.ns, self.lens = dtype, store, ns, lens
        self.H, self.dk, self.dv, self.page = H, dk, dv, page
        per = [-(-n // page) for n in lens]
        pages = sum(per) + spare
        order = rng.permutation(pages)
        self.table = np.full((len(ns), max(per + [1])), -1, np.int32)
        at = 0
        for r, p in enumerate(per):
            self.table[r, :p] = order[at:at + p]
            at += p
        self.place()
        used = np.concatenate(self.slots + [np.zeros(0, np.int64)])
        x = torch.randn((pages * page, dk), generator=g)
        s = None
        if store in ref.TOP:
            codes, sc = ref.quantise_fp32(x.numpy(), store)
            t = torch.from_numpy(codes.view(np.uint8).copy()).view(STORES[store])
            s = torch.full((pages * page,), float("nan"))
            s[used] = torch.from_numpy(sc)[used]
            s = s.view(pages, page, 1)
        else:
            x = x.to(STORES[store])
            t = torch.full_like(x, float("nan"))
            t[used] = x[used]
        wide = torch.zeros((pages, page, 1, dk + pad), dtype=t.dtype)
        wide.view(torch.uint8).fill_(0x7f)  # NaN, or large
        wide.view(torch.uint8).view(pages, page, -1)[..., :dk * t.element_size()] = \
            t.view(torch.uint8).view(pages, page, -1)
        self.k = wide.to(DEV)[..., :dk]
        self.ks = None if s is None else s.to(DEV)
        self.cache = binding.KVCache(self.k, k_scale=self.ks)
        self.Tq = sum(ns)
        self.q = (torch.randn((self.Tq, H, dk), generator=g) * scale_of_q).to(TYPES[dtype])
        self.q_start = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        self.words = None
        if tree == "random":
            w = max(1, -(-max(ns + [1]) // 64))
            self.words = np.zeros((self.Tq, w), np.int64)
            for r, n in enumerate(ns):
                parents = [-1 if i == 0 else int(rng.integers(-1, i)) for i in range(n)]
                got = binding.rope_partial_tree_mask(parents).numpy()
                self.words[self.q_start[r]:self.q_start[r + 1], :got.shape[1]] = got

    def place(self):
        self.slots = [self.table[r, np.arange(n) // self.page].astype(np.int64) * self.page + np.arange(n) % self.page
                      for r, n in enumerate(self.lens)]

    def numbers(self):
        """The rows in 64 bits, from what the device holds."""
        if self.store in ref.TOP:
            c = self.k.contiguous().view(torch.uint8).flatten(0, 2).cpu().numpy()
            num = ref.fp8_values()[c] if self.store == "fp8" else c.view(np.int8).astype(np.float64)
            with np.errstate(invalid="ignore"):
                return num * self.ks.flatten().double().cpu().numpy()[:, None]
        return self.k.flatten(0, 2).double().cpu().numpy()

    def device(self):
        dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
        return (self.q.to(DEV), dev(self.q_start), dev(np.array(self.lens, np.int32)), dev(self.table),
                dev(self.words))

    def run(self, scale=None, max_q=None, **kw):
        q, qs, ln, table, tree = self.device()
        out = torch.full((self.Tq, self.H, self.dv), 77.0, dtype=TYPES[self.dtype], device=DEV)
        lse = torch.full((self.Tq, self.H), 77.0, device=DEV)
        binding.rope_partial_latent_attention(q, self.cache, qs, ln, table, out, lse=lse, tree=tree, scale=scale,
                                              max_q=max_q or max(self.ns + [1]), **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, scale=None, heads=None):
        scale = scale or 1 / math.sqrt(self.dk)
        u = 2.0 ** -8 if self.store == "bf16" else 2.0 ** -11
        u_out = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -11
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        q, rows = self.q.double().numpy(), self.numbers()
        heads = heads or (range(self.H) if self.H <= 8 else sorted({0, 1, self.H // 2, self.H - 1}))
        for r, n in enumerate(self.ns):
            if n == 0:
                continue
            at = slice(self.q_start[r], self.q_start[r + 1])
            sees = ref.tree_sees(n, self.lens[r], self.lens[r] - n, None if self.words is None else self.words[at])
            k = rows[self.slots[r]]
            for h in heads:
                o, l, mag = ref.tree_attention(q[at, h], k, k[:, :self.dv], sees, scale)
                big = scale * (np.abs(q[at, h]) @ np.abs(k).T).max(-1, initial=0)
                d = ((self.dk + 8) * 2.0 ** -24 * big + 2.0 ** -21)[:, None]
                none = np.isneginf(l)
                # sum_j 2^-32 (largest p scale_j) codes / sum_j p_j, with codes below 448
                small = 2.0 ** -32 * len(k) * np.abs(k).max(initial=0) if self.store != "bf16" else 0.0
                tol = (u + 4 * d) * mag + u_out * np.abs(o) + small + 1e-30
                err = np.abs(out[at, h] - o)
                assert np.all(err <= tol), (r, h, np.nanmax(err / tol), np.argwhere(~(err <= tol))[:4])
                assert np.array_equal(np.isneginf(lse[at, h]), none)
                assert np.all(out[at, h][none] == 0)
                e = np.abs(lse[at, h][~none] - l[~none])
                assert np.all(e <= 2 * d[~none, 0] + 2.0 ** -22 * np.abs(l[~none])), (r, h, e.max())


PAIRS = [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp8"), ("fp16", "int8"), ("bf16", "int8"), ("fp16", "fp8")]
LENGTHS = [  # drafts, cache lengths (with the drafts)
    ([1], [1]),
    ([1], [65]),
    ([1, 1, 1], [700, 1, 129]),
    ([4], [4]),                       # nothing but the drafts
    ([5, 1, 0, 3], [64, 0, 9, 128]),  # an empty request, and one with no cache rows at all
    ([13, 2], [300, 66]),
    ([33], [97]),
]
DIMS = [(576, 512), (288, 256), (80, 48), (320, 320), (16, 16), (192, 128)]


@pytest.mark.parametrize("dtype,store", PAIRS)
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("k", range(len(LENGTHS)))
def test_parity(k, dims, dtype, store):
    ns, lens = LENGTHS[k]
    H = [1, 16, 5, 3, 40, 8][(k + DIMS.index(dims)) % 6]
    c = Case(dtype, store, ns, lens, H, *dims, page=[16, 1, 48, 64, 3][(k + dims[0] // 16) % 5], seed=k,
             pad=16 if k % 2 else 0)
    c.check(*c.run())


@pytest.mark.parametrize("dtype,store", PAIRS[:4])
@pytest.mark.parametrize("ns,H", [([1], 128), ([3, 1], 64), ([17], 1), ([2], 16), ([4, 9], 20), ([130, 70], 4),
                                  ([2, 1], 200)])
def test_query_rows(ns, H, dtype, store):
    """Row counts around the tiles of 16, 32 and 64 query rows, and many of them; trees of
    more than 64 tokens (several words)."""
    c = Case(dtype, store, ns, [n + 77 + 60 * i for i, n in enumerate(ns)], H, 576, 512, page=16, seed=len(ns) + H)
    c.check(*c.run())


@pytest.mark.parametrize("store", ["bf16", "int8"])
@pytest.mark.parametrize("n", [1, 6, 40, 300])
def test_chains(n, store):
    """Without a tree: causal decoding, and a chunk of a prompt."""
    c = Case("bf16", store, [n, 1], [n + 41, 250], 4, 128, 64, page=32, tree=None, seed=n)
    c.check(*c.run())


@pytest.mark.parametrize("store,page", [("bf16", 64), ("bf16", 20), ("fp8", 64)])
@pytest.mark.parametrize("n,H", [(1, 8), (12, 2), (5, 32)])
def test_long_contexts_are_split_and_joined(n, H, store, page):
    """Lengths that many blocks share: the split depends on the device only, and the parts
    are joined in one order, so two runs agree bit for bit."""
    c = Case("bf16", store, [n, 2], [5000, 20011], H, 576, 512, page=page, seed=n)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(*a, heads=[0, H - 1])


@pytest.mark.parametrize("store,page", [("bf16", 32), ("fp16", 12), ("int8", 32)])
@pytest.mark.parametrize("H", [4, 30, 64])
def test_short_and_long_requests_together(H, store, page):
    """Several runs of one tile a block, between long ones and empty ones."""
    rng = np.random.default_rng(H)
    ns = rng.integers(1, 4, 300).tolist()
    lens = [n + int(x) for n, x in zip(ns, np.exp(rng.uniform(0, 6, 300)))]
    for r in range(3, 300, 31):
        lens[r] = int(rng.integers(4000, 5000))
    ns[10] = ns[11] = 0
    lens[11] = 0
    c = Case("fp16" if store == "fp16" else "bf16", store, ns, lens, H, 96, 64, page=page, seed=H)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(*a, heads=[0, H - 1])


def test_a_wrong_hint_costs_time_only():
    c = Case("bf16", "bf16", [33, 5], [200, 90], 4, 576, 512, page=16, seed=3)
    for hint in (1, 5, 8, 1000):
        c.check(*c.run(max_q=hint))


@pytest.mark.parametrize("store,page", [("bf16", 16), ("bf16", 5), ("fp16", 16), ("fp8", 16), ("int8", 16)])
@pytest.mark.parametrize("n,H", [(6, 2), (30, 1), (40, 4)])
def test_not_finite_where_nobody_looks(n, H, store, page):
    """Infinities and NaN in drafted rows reach the tokens that see them, and nobody else."""
    dtype = "fp16" if store == "fp16" else "bf16"
    # token i hangs on i - 1, but for token 3, which hangs on the context and has no
    # children: only token 3 sees row prefix + 3
    parents = [-1, 0, 1, -1] + [2 if i == 4 else i - 1 for i in range(4, n)]
    got = []
    for spoilt in (True, False):
        c = Case(dtype, store, [n], [n + 70], H, 576, 512, page=page, seed=n)
        c.words = binding.rope_partial_tree_mask(parents).numpy()
        if spoilt:
            at = divmod(int(c.slots[0][70 + 3]), c.page)
            if store == "int8":
                c.ks[at] = float("inf")
            elif store == "fp8":
                c.k.view(torch.uint8)[at[0], at[1], :, 1::2] = 0xff
            else:
                c.k[at[0], at[1], :, 1::2] = float("inf")
                c.k[at[0], at[1], :, 3::4] = float("nan")
        got.append(c.run())
    (out, lse), (want, want_lse) = got
    # (an infinite scale may make the score -inf, of a weight of 0, and the sum a number)
    assert not torch.isfinite(out[3]).all(-1).any() and (store == "int8" or torch.isnan(lse[3]).all())
    keep = [i for i in range(n) if i != 3]
    assert torch.isfinite(want).all() and torch.isfinite(want_lse).all()
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])


def test_rows_that_see_nothing():
    c = Case("bf16", "bf16", [3, 20], [3, 20], 2, 576, 512, page=16, seed=2)
    c.words[:] = 0
    c.words[4] = 1 << 1
    out, lse = c.run()
    c.check(out, lse)
    assert torch.isneginf(lse[[0, 1, 2, 3, 5]]).all() and torch.isfinite(lse[4]).all()


@pytest.mark.parametrize("dtype,store", [("bf16", "fp8"), ("fp16", "int8")])
@pytest.mark.parametrize("n", [2, 30])
def test_scales_and_queries_of_any_size(n, dtype, store):
    """8-bit caches: scales that grow along the row by twenty powers of two, queries as much
    larger; zero and negative scales among them."""
    c = Case(dtype, store, [n], [600], 2, 576, 512, page=16, seed=n, scale_of_q=2.0 ** 7)
    up = torch.exp2(torch.arange(600) * 20.0 / 600 - 27).to(DEV)
    flat = c.ks.view(-1)
    flat[torch.from_numpy(c.slots[0]).to(DEV)] *= up
    flat[int(c.slots[0][17])] = 0.0
    flat[int(c.slots[0][400])] *= -1.0
    c.check(*c.run())


@pytest.mark.parametrize("store", ["fp8", "int8"])
def test_nothing_but_scales_of_zero(store):
    """Rows of zeros by their scale: the mean of nothing, and the rows counted."""
    c = Case("bf16", store, [3], [90], 4, 576, 512, page=16, seed=1)
    c.ks.nan_to_num_(0.0)
    c.ks.zero_()
    out, lse = c.run()
    assert not out.any()
    c.check(out, lse)


def test_scores_that_grow_along_the_cache():
    """The maximum moves on in many tiles, by more and by less than it may lag."""
    for step in (0.05, 0.4):
        c = Case("fp16", "fp16", [2], [2000], 3, 576, 512, page=16, seed=4)
        c.q[..., 0] = 1.0
        rows = torch.from_numpy(c.slots[0]).to(DEV)
        c.k.flatten(0, 2)[rows, 0] = (torch.arange(2000, device=DEV) * step * 24 % 1000).to(torch.float16)
        c.check(*c.run())


def test_a_flat_tail_of_small_weights_is_kept():
    """One row with a large score before 40000 rows whose weights are 2^-22 of its own:
    together they are 1 % of the sum, and the values there are not small."""
    n_rows, gap = 40001, 22 * math.log(2) / 8.0
    c = Case("fp16", "fp16", [1], [n_rows], 1, 64, 48, page=64, seed=4)
    c.q.zero_()
    c.q[0, 0, 63] = 8.0
    flat, rows = c.k.flatten(0, 2), torch.from_numpy(c.slots[0]).to(DEV)
    flat[rows] = 64.0
    flat[rows, 63] = 0.0
    flat[int(c.slots[0][0])] = 0.0
    flat[int(c.slots[0][0]), 63] = gap
    c.check(*c.run(scale=1.0), scale=1.0)


@pytest.mark.parametrize("store", ["bf16", "fp16", "fp8", "int8"])
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -120])
def test_scores_of_nearly_zero(scale, store):
    dtype = "fp16" if store == "fp16" else "bf16"
    c = Case(dtype, store, [5], [95], 4, 64, 64, page=16, seed=5)
    c.q[0] = 0
    c.check(*c.run(scale=scale), scale=scale)


def test_strides_streams_and_a_kept_workspace():
    """q and out as slices of packed tensors, a page table wider than needed, a stream of its
    own, one workspace for two calls."""
    c = Case("bf16", "fp8", [7, 3], [150, 333], 3, 576, 512, page=16, seed=6)
    q, qs, ln, table, tree = c.device()
    packed = torch.zeros((c.Tq, 2 * c.H, 576), dtype=torch.bfloat16, device=DEV)
    packed[:, c.H:] = q
    wide = torch.full((2, table.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    lse = torch.empty((c.Tq, c.H), device=DEV)
    ws = binding.latent_attention_workspace(q, c.cache, 512, 7)
    ws.fill_(0xff)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out = packed[:, :c.H, 64:]
    for _ in range(2):
        binding.rope_partial_latent_attention(packed[:, c.H:], c.cache, qs, ln, wide, out, lse=lse, tree=tree, max_q=7,
                                              workspace=ws, stream=stream)
    stream.synchronize()
    c.check(out, lse)
    assert torch.equal(packed[:, c.H:], q) and not packed[:, :c.H, :64].any()


def test_two_calls_at_once():
    """Two streams, each with a workspace of its own."""
    cases = [Case("bf16", "bf16", [2, 1], [3000, 700], 16, 576, 512, page=16, seed=s) for s in (1, 2)]
    got, streams = [], [torch.cuda.Stream() for _ in cases]
    args = []
    for c in cases:
        q, qs, ln, table, tree = c.device()
        out, lse = torch.empty((c.Tq, c.H, c.dv), dtype=torch.bfloat16, device=DEV), torch.empty((c.Tq, c.H), device=DEV)
        args.append((q, c.cache, qs, ln, table, out, lse, tree, binding.latent_attention_workspace(q, c.cache, 512, 2)))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (q, cache, qs, ln, table, out, lse, tree, ws) in zip(streams, args):
            binding.rope_partial_latent_attention(q, cache, qs, ln, table, out, lse=lse, tree=tree, max_q=2,
                                                  workspace=ws, stream=s)
    torch.cuda.synchronize()
    for c, a in zip(cases, args):
        c.check(a[5], a[6])
    del got


@pytest.mark.parametrize("page", [16, 10])
def test_values_only_the_device_sees(page):
    """Offsets, lengths and page numbers out of range read nothing outside the tensors, and
    tokens of no request stay as they were."""
    c = Case("bf16", "bf16", [2, 2], [40, 33], 2, 576, 512, page=page, seed=1)
    c.k.nan_to_num_(0.5)
    q, qs, ln, table, tree = c.device()
    out = torch.full((4, 2, 512), 5.0, dtype=torch.bfloat16, device=DEV)
    table[0, 1] = 10 ** 9
    table[1, 0] = -7
    ln[0] = 2 ** 30
    ln[1] = -5
    qs[2] = 2 ** 30
    binding.rope_partial_latent_attention(q, c.cache, qs, ln, table, out, tree=tree, max_q=2)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and (out[2:] == 0).all()
    q, qs, ln, table, tree = c.device()
    out2 = torch.full((4, 2, 512), 5.0, dtype=torch.bfloat16, device=DEV)
    qs[1], qs[2] = 0, 1  # request 0 has no tokens, request 1 has one; the rest are nobody's
    binding.rope_partial_latent_attention(q, c.cache, qs, ln, table, out2, tree=tree, max_q=2)
    torch.cuda.synchronize()
    assert (out2[1:] == 5.0).all() and torch.isfinite(out2[0]).all()


@pytest.mark.parametrize("store", ["bf16", "fp8"])
@pytest.mark.parametrize("n,H", [(2, 2), (30, 1), (40, 4)])
def test_a_cache_without_pages(n, H, store):
    """No rows at all, and (every page number lying outside) rows of zeros."""
    k = torch.empty((0, 16, 1, 64), dtype=STORES[store], device=DEV)
    cache = binding.KVCache(k, k_scale=torch.empty((0, 16, 1), device=DEV) if store == "fp8" else None)
    q = torch.randn((n, H, 64), device=DEV).to(torch.bfloat16)
    for length, width in ((0, 0), (0, 4), (n, 4)):
        out, lse = torch.full((n, H, 48), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((n, H), 7.0, device=DEV)
        binding.rope_partial_latent_attention(q, cache, i32(0, n), i32(length),
                                              torch.zeros((1, width), dtype=torch.int32, device=DEV), out, lse=lse)
        torch.cuda.synchronize()
        assert not out.any()
        if length == 0:
            assert torch.isneginf(lse).all()
        else:  # a chain: token i sees i + 1 rows with a score of 0
            want = torch.log(torch.arange(1, n + 1, device=DEV).double())[:, None].expand(n, H)
            assert (lse.double() - want).abs().max() <= 2.0 ** -20


def test_many_requests():
    """More requests than a block has threads."""
    rng = np.random.default_rng(0)
    ns = [int(x) for x in rng.integers(0, 4, size=700)]
    lens = [n + int(x) for n, x in zip(ns, rng.integers(0, 90, size=700))]
    c = Case("bf16", "int8", ns, lens, 2, 64, 64, page=16, seed=5)
    c.check(*c.run())


def test_offsets_past_32_bits():
    """Pages whose rows lie more than 4 GB into the cache, 16-bit (copied as boxes, and row
    by row) and 8-bit."""
    for store, page, pages in (("bf16", 64, 61000), ("bf16", 20, 195000), ("fp8", 64, 122000)):
        k = torch.empty((pages, page, 1, 576), dtype=STORES[store], device=DEV)
        s = torch.ones((pages, page, 1), device=DEV) if store == "fp8" else None
        own = [pages - 1, 3, pages - 2, 7, pages - 3, 8, pages - 4, 9][:-(-150 // page)]
        for p in own:
            k[p].copy_(torch.randn((page, 1, 576), device=DEV).to(torch.float16))
        q = torch.randn((3, 4, 576), device=DEV).to(torch.bfloat16)
        out = torch.empty((3, 4, 512), dtype=torch.bfloat16, device=DEV)
        binding.rope_partial_latent_attention(q, binding.KVCache(k, k_scale=s), i32(0, 3), i32(150), i32(*own)[None], out)
        kk = torch.cat([k[p] for p in own]).to(torch.float16).double()[:150, 0]
        z = torch.einsum("qhd,kd->hqk", q.double(), kk) / 24
        j = torch.arange(150, device=DEV)
        z = z.masked_fill(j[None, None] > 147 + torch.arange(3, device=DEV)[None, :, None], -math.inf)
        want = torch.einsum("hqk,kd->qhd", z.softmax(-1), kk[:, :512])
        assert (out.double() - want).abs().max() <= 2.0 ** -7 * kk.abs().max()
        del k, s


def test_in_a_cuda_graph():
    """Captured once; lengths and pages may change between replays."""
    c = Case("bf16", "bf16", [4, 4], [100, 300], 16, 576, 512, page=16, seed=9, spare=40)
    c.k.nan_to_num_(0.25)
    q, qs, ln, table, tree = c.device()
    out = torch.empty((c.Tq, c.H, c.dv), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((c.Tq, c.H), device=DEV)
    ws = binding.latent_attention_workspace(q, c.cache, 512, 4)

    def step():
        binding.rope_partial_latent_attention(q, c.cache, qs, ln, table, out, lse=lse, tree=tree, max_q=4, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([100, 300], [50, 4], [99, 211]):
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.lens = lens
        c.place()
        c.check(out, lse)


@pytest.mark.parametrize("store", ["bf16", "fp8"])
def test_strides_of_dims_of_one(store):
    """One token and one page, whose strides are no multiples of anything."""
    c = Case("bf16", store, [1], [60], 8, 576, 512, page=64, tree=None, seed=2, spare=0)
    want, _ = c.run()

    def odd(t, dims):
        return t.as_strided(t.shape, [101 + 2 * i if i in dims else s for i, s in enumerate(t.stride())])

    q, qs, ln, table, _ = c.device()
    cache = binding.KVCache(odd(c.k, (0, 2)), k_scale=None if c.ks is None else odd(c.ks, (0, 2)))
    out = torch.empty((1, 8, 512), dtype=torch.bfloat16, device=DEV)
    binding.rope_partial_latent_attention(odd(q, (0,)), cache, qs, ln, table, odd(out, (0,)), max_q=1)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
