"""Attention of drafted tokens over a paged cache, against the same sums in 64
bits over the rows that a token sees.

Bounds, per element, with u = 2^-8 (bf16 products) or 2^-11 (fp16 products),
u_out the output type's, and A = sum_j p_j |v_j| / sum_j p_j:
  |out - exact| <= (u + 4 d) A + u_out |exact| + tiny,
  |lse - exact| <= 2 d + 2^-22 |exact|,
where d bounds the error of a score: the fp32 sum of Dk products, each exact
in fp32, is off by at most Dk 2^-24 of the sum of their sizes, S = scale
max_j sum_d |q_d k_jd|, the scale and base-2 steps by 4 2^-24 S, and 2^x by
2^-22; an error d of the scores changes p relative to its sum by up to 2 d, and
again as much covers the sums over rows (whose fp32 rounding is below 2^-24
per row of a tile's partial sums).  u counts the one rounding of p.
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


class Case:
    """Requests with given drafts and cache lengths, in pages in random order;
    what no request owns (other pages, the ends of last pages) is NaN."""

    def __init__(self, dtype, store, ns, lens, Hk, G, dk, dv, page, tree="random", seed=0, head_major=False,
                 scale_of_q=1.0, spare=3):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.dtype, self.store, self.ns, self.lens = dtype, store, ns, lens
        self.Hk, self.G, self.dk, self.dv, self.page = Hk, G, dk, dv, page
        per = [-(-n // page) for n in lens]
        pages = sum(per) + spare
        order = rng.permutation(pages)
        width = max(per + [1])
        self.table = np.full((len(ns), width), -1, np.int32)
        at = 0
        for r, p in enumerate(per):
            self.table[r, :p] = order[at:at + p]
            at += p
        self.slots = [self.table[r, np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
                      for r, n in enumerate(lens)]
        used = np.concatenate(self.slots + [np.zeros(0, np.int64)])
        self.rows, tensors = {}, []
        for name, d in (("k", dk), ("v", dv)):
            x = torch.randn((pages * page, Hk, d), generator=g)
            s = None
            if store in ref.TOP:
                codes, sc = ref.quantise_fp32(x.numpy(), store)
                codes = torch.from_numpy(codes.view(np.uint8).copy())
                num = (ref.fp8_values()[codes.numpy()] if store == "fp8"
                       else codes.numpy().view(np.int8).astype(np.float64))
                self.rows[name] = num * sc.astype(np.float64)[..., None]
                t = codes.view(STORES[store]).view(pages, page, Hk, d)
                s = torch.full((pages * page, Hk), float("nan"))
                s[used] = torch.from_numpy(sc)[used]
                s = s.view(pages, page, Hk)
            else:
                x = x.to(STORES[store])
                self.rows[name] = x.double().numpy()
                t = torch.full_like(x, float("nan"))
                t[used] = x[used]
                t = t.view(pages, page, Hk, d)
            if head_major:
                t = t.permute(0, 2, 1, 3).contiguous().to(DEV).permute(0, 2, 1, 3)
            else:
                t = t.to(DEV)
            tensors.append((t, None if s is None else s.to(DEV)))
        (self.k, self.ks), (self.v, self.vs) = tensors
        self.cache = binding.KVCache(self.k, self.v, self.ks, self.vs)
        self.Tq, self.Hq = sum(ns), Hk * G
        self.q = (torch.randn((self.Tq, self.Hq, dk), generator=g) * scale_of_q).to(TYPES[dtype])
        self.q_start = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        self.words = None
        if tree == "random":
            w = max(1, -(-max(ns + [1]) // 64))
            self.words = np.zeros((self.Tq, w), np.int64)
            for r, n in enumerate(ns):
                parents = [-1 if i == 0 else int(rng.integers(-1, i)) for i in range(n)]
                got = binding.rope_partial_tree_mask(parents).numpy()
                self.words[self.q_start[r]:self.q_start[r + 1], :got.shape[1]] = got

    def device(self):
        dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
        return (self.q.to(DEV), dev(self.q_start), dev(np.array(self.lens, np.int32)), dev(self.table),
                dev(self.words))

    def run(self, scale=None, max_q=None, out=None, **kw):
        q, qs, ln, table, tree = self.device()
        if out is None:
            out = torch.full((self.Tq, self.Hq, self.dv), 77.0, dtype=TYPES[self.dtype], device=DEV)
        lse = torch.full((self.Tq, self.Hq), 77.0, device=DEV)
        binding.rope_partial_tree_attention(q, self.cache, qs, ln, table, out, lse=lse, tree=tree, scale=scale,
                                            max_q=max_q or max(self.ns + [1]), **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, scale=None, edit=None):
        scale = scale or 1 / math.sqrt(self.dk)
        u = 2.0 ** -8 if self.store == "bf16" else 2.0 ** -11
        u_out = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -11
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        q = self.q.double().numpy()
        for r, n in enumerate(self.ns):
            if n == 0:
                continue
            at = slice(self.q_start[r], self.q_start[r + 1])
            words = None if self.words is None else self.words[at]
            sees = ref.tree_sees(n, self.lens[r], self.lens[r] - n, words)
            for h in range(self.Hq):
                k, v = (self.rows[x][self.slots[r], h // self.G] for x in ("k", "v"))
                o, l, mag = ref.tree_attention(q[at, h], k, v, sees, scale)
                big = scale * (np.abs(q[at, h]) @ np.abs(k).T).max(-1, initial=0)
                d = ((self.dk + 8) * 2.0 ** -24 * big + 2.0 ** -21)[:, None]
                tol = (u + 4 * d) * mag + u_out * np.abs(o) + 1e-30
                err = np.abs(out[at, h] - o)
                assert np.all(err <= tol), (r, h, (err / tol).max())
                none = np.isneginf(l)
                assert np.array_equal(np.isneginf(lse[at, h]), none)
                assert np.all(out[at, h][none] == 0)
                e = np.abs(lse[at, h][~none] - l[~none])
                assert np.all(e <= 2 * d[~none, 0] + 2.0 ** -22 * np.abs(l[~none])), (r, h)


LENGTHS = [  # drafts, cache lengths (with the drafts)
    ([1], [1]),
    ([1], [65]),
    ([1, 1, 1], [700, 1, 129]),
    ([4], [4]),                       # nothing but the drafts
    ([5, 1, 0, 3], [64, 0, 9, 128]),  # an empty request, and one with no cache rows at all
    ([13, 2], [300, 66]),
    ([33], [97]),
]
HEADS = [(1, 1), (2, 4), (1, 12), (3, 1)]
DIMS = [(64, 64), (128, 128), (192, 128), (80, 48), (256, 256), (16, 16)]


@pytest.mark.parametrize("dtype,store", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp8"), ("fp16", "int8"),
                                         ("bf16", "int8"), ("fp16", "fp8")])
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("k", range(len(LENGTHS)))
def test_parity(k, dims, dtype, store):
    ns, lens = LENGTHS[k]
    Hk, G = HEADS[(k + DIMS.index(dims)) % len(HEADS)]
    c = Case(dtype, store, ns, lens, Hk, G, *dims, page=[16, 1, 48, 64, 3][(k + dims[0]) % 5], seed=k,
             head_major=k % 2 == 1)
    c.check(*c.run())


@pytest.mark.parametrize("store", ["bf16", "fp16", "fp8", "int8"])
@pytest.mark.parametrize("ns,G", [([9], 1), ([17], 1), ([8, 20], 4), ([64], 2), ([64], 5), ([40, 64], 8),
                                  ([130, 70], 4)])
def test_many_query_rows(ns, G, store):
    """Row counts around the kernels' row tiles: 9 to 520 a key head, and trees
    of more than 64 tokens (several words)."""
    dtype = "fp16" if store == "fp16" else "bf16"
    c = Case(dtype, store, ns, [n + 77 + 60 * i for i, n in enumerate(ns)], 2, G, 128, 128, page=16, seed=len(ns) + G)
    c.check(*c.run())


@pytest.mark.parametrize("store", ["bf16", "int8"])
@pytest.mark.parametrize("n", [1, 6, 40, 300])
def test_chains(n, store):
    """Without a tree: causal decoding, and a chunk of a prompt."""
    c = Case("bf16", store, [n, 1], [n + 41, 250], 2, 2, 64, 64, page=32, tree=None, seed=n)
    c.check(*c.run())


@pytest.mark.parametrize("store", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [1, 12, 70])
def test_long_contexts_are_split_and_joined(n, store):
    """Lengths that many blocks share: the split depends on the device only,
    and the parts are joined in one order, so two runs agree bit for bit."""
    c = Case("bf16", store, [n, 2], [5000, 20011], 1, 2, 64, 64, page=64, seed=n)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(*a)


@pytest.mark.parametrize("store", ["bf16", "fp16", "fp8"])
def test_few_query_rows_over_many_tiles(store):
    """One to three tokens a request at a batch whose cache is large: another
    kernel than that of a few requests (16-bit), and the workspace serves both."""
    rng = np.random.default_rng(11)
    ns = rng.integers(1, 4, 56).tolist()
    lens = (rng.integers(0, 700, 56) + ns).tolist()
    lens[7], lens[8] = ns[7], 2048
    dtype = "fp16" if store == "fp16" else "bf16"
    c = Case(dtype, store, ns, lens, 2, 4, 64, 64, page=16, seed=5)
    q = c.q.to(DEV)
    one, few = (binding.tree_attention_workspace(q, c.cache, n) for n in (1, 3))
    assert one.numel() == few.numel()
    c.check(*c.run(workspace=few))


@pytest.mark.parametrize("store,most", [("bf16", 3), ("fp8", 3), ("bf16", 20), ("int8", 20)])
def test_short_and_long_requests_together(store, most):
    """Many tiles a block, where a request's start counts as several of them
    when the work is cut: short requests between long ones, and empty ones."""
    rng = np.random.default_rng(most)
    ns = rng.integers(1, most + 1, 64).tolist()
    lens = [n + int(x) for n, x in zip(ns, np.exp(rng.uniform(0, 6, 64)))]
    for r in range(3, 64, 7):
        lens[r] = int(rng.integers(8000, 10000))
    ns[10] = ns[11] = 0
    lens[11] = 0
    c = Case("bf16", store, ns, lens, 4, 2, 16, 16, page=32, seed=most)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(*a)


def test_a_wrong_hint_costs_time_only():
    c = Case("bf16", "bf16", [33, 5], [200, 90], 2, 4, 128, 128, page=16, seed=3)
    for hint in (1, 8, 20, 1000):
        c.check(*c.run(max_q=hint))


@pytest.mark.parametrize("store", ["bf16", "fp16", "fp8", "int8"])
@pytest.mark.parametrize("n,G", [(6, 2), (30, 1), (40, 4)])
def test_not_finite_where_nobody_looks(n, G, store):
    """Infinities and NaN in drafted rows reach the tokens that see them, and
    nobody else."""
    dtype = "fp16" if store == "fp16" else "bf16"
    c = Case(dtype, store, [n], [n + 70], 1, G, 64, 64, page=16, seed=n)
    # token i hangs on i - 1, but for token 3, which hangs on the context and
    # has no children: only token 3 sees row prefix + 3
    parents = [-1, 0, 1, -1] + [2 if i == 4 else i - 1 for i in range(4, n)]
    c.words = binding.rope_partial_tree_mask(parents).numpy()
    slot = c.slots[0][70 + 3]
    page, off = divmod(int(slot), c.page)
    if store in ref.TOP:
        c.ks[page, off] = float("nan")
        c.vs[page, off] = float("nan")
    else:
        c.k[page, off] = float("nan")
        c.v[page, off, :, 1::2] = float("inf")
    out, lse = c.run()
    seen = out[3], lse[3]
    assert torch.isnan(lse[3]).all() and torch.isnan(out[3, :, 1::2]).all()
    # the others are as if the row were not there
    keep = [i for i in range(n) if i != 3]
    assert torch.isfinite(out[keep]).all() and torch.isfinite(lse[keep]).all()
    d = Case(dtype, store, [n], [n + 70], 1, G, 64, 64, page=16, seed=n)
    d.words = c.words
    want, want_lse = d.run()
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])
    del seen


@pytest.mark.parametrize("store", ["bf16", "fp16"])
def test_an_infinite_value_that_is_seen(store):
    """A drafted value of infinity gives infinity to the tokens that see it, in
    its columns only; -inf and +inf together give NaN."""
    c = Case(store, store, [20], [50], 1, 2, 64, 64, page=16, seed=8)
    parents = [-1] + [0] * 19
    c.words = binding.rope_partial_tree_mask(parents).numpy()
    for i, x in ((5, float("inf")), (0, -float("inf"))):
        page, off = divmod(int(c.slots[0][30 + i]), c.page)
        c.v[page, off, 0, 7 if i else 9] = x
    c.v[divmod(int(c.slots[0][30 + 6]), c.page)[0], int(c.slots[0][30 + 6]) % c.page, 0, 9] = float("inf")
    out, _ = c.run()
    o = out.float().cpu()
    assert torch.isposinf(o[5, :, 7]).all() and torch.isneginf(o[[i for i in range(20) if i != 6]][:, :, 9]).all()
    assert torch.isnan(o[6, :, 9]).all()
    rest = torch.ones(64, dtype=torch.bool)
    rest[7] = rest[9] = False
    assert torch.isfinite(o[:, :, rest]).all() and torch.isfinite(o[[0, 1, 6], :, 7]).all()


def test_rows_that_see_nothing():
    c = Case("bf16", "bf16", [3, 20], [3, 20], 1, 2, 64, 64, page=16, seed=2)
    c.words[:] = 0
    c.words[4] = 1 << 1
    out, lse = c.run()
    c.check(out, lse)
    assert torch.isneginf(lse[[0, 1, 2, 3, 5]]).all() and torch.isfinite(lse[4]).all()


@pytest.mark.parametrize("store", ["fp8", "int8"])
@pytest.mark.parametrize("n", [2, 30])
def test_scales_and_queries_of_any_size(n, store):
    """8-bit caches: values' scales that grow along the row by twenty powers of
    two, and queries past fp16's range (the keys' scales shrink alike)."""
    c = Case("bf16", store, [n], [600], 1, 2, 64, 64, page=16, seed=n, scale_of_q=2.0 ** 20)
    up = torch.exp2(torch.arange(600) * 20.0 / 600 - 30)
    for j, s in enumerate(c.slots[0]):
        page, off = divmod(int(s), c.page)
        c.vs[page, off] *= up[j].item()
        c.ks[page, off] *= 2.0 ** -20
        c.rows["v"][s] *= np.float64(np.float32(1)) * (c.vs[page, off].double().cpu().numpy() /
                                                       (c.vs[page, off] / up[j].item()).double().cpu().numpy())[:, None]
        c.rows["k"][s] *= 2.0 ** -20
    # the codes times the scales as the device holds them
    codes = c.v.view(torch.uint8).flatten(0, 1).cpu().numpy()
    num = ref.fp8_values()[codes] if store == "fp8" else codes.view(np.int8).astype(np.float64)
    c.rows["v"] = num * c.vs.flatten(0, 1).double().cpu().numpy()[..., None]
    c.check(*c.run())


def test_a_flat_tail_of_small_weights_is_kept():
    """One row with a large score before 40000 rows whose weights are 2^-22 of
    its own: together they are 1 % of the sum, and the values there are not
    small."""
    n_rows = 40001
    c = Case("fp16", "fp16", [1], [n_rows], 1, 1, 64, 64, page=64, seed=4)
    c.q.zero_()
    c.q[0, 0, 0] = 8.0
    flat = c.k.flatten(0, 1)
    flat.zero_()
    gap = 22 * math.log(2) / 8.0
    first = int(c.slots[0][0])
    flat[first, 0, 0] = gap
    c.rows["k"][:] = 0
    c.rows["k"][first, 0, 0] = float(torch.tensor(gap).half())
    v = c.v.flatten(0, 1)
    rows = torch.from_numpy(c.slots[0]).to(DEV)
    v[rows] = 64.0
    v[first] = 0.0
    c.rows["v"][:] = 64.0
    c.rows["v"][first] = 0.0
    c.check(*c.run(scale=1.0), scale=1.0)


def test_strides_streams_and_a_kept_workspace():
    """q and out as slices of packed tensors, a page table wider than needed, a
    stream of its own, one workspace for two calls."""
    c = Case("bf16", "fp8", [7, 3], [150, 333], 2, 3, 64, 64, page=16, seed=6)
    q, qs, ln, table, tree = c.device()
    packed = torch.zeros((c.Tq, 3 * c.Hq, 64), dtype=torch.bfloat16, device=DEV)
    packed[:, c.Hq:2 * c.Hq] = q
    wide = torch.full((2, table.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    lse = torch.empty((c.Tq, c.Hq), device=DEV)
    ws = binding.tree_attention_workspace(q, c.cache, 7)
    ws.fill_(0xff)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        binding.rope_partial_tree_attention(packed[:, c.Hq:2 * c.Hq], c.cache, qs, ln, wide, packed[:, 2 * c.Hq:],
                                            lse=lse, tree=tree, max_q=7, workspace=ws, stream=stream)
    stream.synchronize()
    c.check(packed[:, 2 * c.Hq:], lse)
    assert torch.equal(packed[:, c.Hq:2 * c.Hq], q) and not packed[:, :c.Hq].any()


def test_values_only_the_device_sees():
    """Offsets, lengths and page numbers out of range read nothing outside the
    tensors: lengths stop at the page table, offsets at Tq, and a page that is
    not there counts as rows of zeros."""
    c = Case("bf16", "bf16", [2, 2], [40, 33], 1, 2, 64, 64, page=16, seed=1)
    c.k.nan_to_num_(0.5)
    c.v.nan_to_num_(0.5)
    q, qs, ln, table, tree = c.device()
    out = torch.full((4, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    table[0, 1] = 10 ** 9
    table[1, 0] = -7
    ln[0] = 2 ** 30
    ln[1] = -5
    qs[2] = 2 ** 30
    binding.rope_partial_tree_attention(q, c.cache, qs, ln, table, out, tree=tree, max_q=2)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    assert (out[2:] == 0).all()  # no rows
    c2 = Case("bf16", "bf16", [2, 2], [40, 33], 1, 2, 64, 64, page=16, seed=1)
    q, qs, ln, table, tree = c2.device()
    out2 = torch.full((4, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    qs[1], qs[2] = 0, 1  # request 0 has no tokens, request 1 has one; the rest are nobody's
    binding.rope_partial_tree_attention(q, c2.cache, qs, ln, table, out2, tree=tree, max_q=2)
    torch.cuda.synchronize()
    assert (out2[1:] == 5.0).all() and torch.isfinite(out2[0]).all()


def test_many_requests():
    """More requests than a block has threads."""
    rng = np.random.default_rng(0)
    ns = [int(x) for x in rng.integers(0, 4, size=700)]
    lens = [n + int(x) for n, x in zip(ns, rng.integers(0, 90, size=700))]
    c = Case("bf16", "int8", ns, lens, 1, 2, 64, 64, page=16, seed=5)
    c.check(*c.run())


def test_offsets_past_32_bits():
    """Pages whose rows lie more than 4 GB into the cache, 16-bit and 8-bit."""
    for store, pages in (("bf16", 17000), ("fp8", 33000)):
        Hk, d, page = 16, 128, 64
        k = torch.empty((pages, page, Hk, d), dtype=STORES[store], device=DEV)
        v = torch.empty_like(k)
        s = [torch.ones((pages, page, Hk), device=DEV) if store == "fp8" else None for _ in range(2)]
        cache = binding.KVCache(k, v, *s)
        own = [pages - 1, 3, pages - 2]
        small = torch.randn((3, page, Hk, d), device=DEV)
        for t in (k, v):
            for i, p in enumerate(own):
                t[p].copy_(small[i].to(torch.float16) * (1 if t is k else -1))
        q = torch.randn((3, Hk, d), device=DEV).to(torch.bfloat16)
        out = torch.empty((3, Hk, d), dtype=torch.bfloat16, device=DEV)
        qs, ln = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 3], [150]))
        table = torch.tensor([own], dtype=torch.int32, device=DEV)
        binding.rope_partial_tree_attention(q, cache, qs, ln, table, out)
        kk = torch.cat([k[p] for p in own]).to(torch.float16).double()[:150].permute(1, 0, 2)
        vv = torch.cat([v[p] for p in own]).to(torch.float16).double()[:150].permute(1, 0, 2)
        z = q.double().permute(1, 0, 2) @ kk.transpose(1, 2) / math.sqrt(d)
        j = torch.arange(150, device=DEV)
        z = z.masked_fill(j[None, None] > 147 + torch.arange(3, device=DEV)[None, :, None], -math.inf)
        want = (z.softmax(-1) @ vv).permute(1, 0, 2)
        assert (out.double() - want).abs().max() <= 2.0 ** -7 * vv.abs().max()
        del k, v, cache


def test_in_a_cuda_graph():
    """Captured once; lengths and pages may change between replays."""
    c = Case("bf16", "bf16", [4, 4], [100, 300], 2, 2, 128, 128, page=16, seed=9, spare=40)
    q, qs, ln, table, tree = c.device()
    out = torch.empty((c.Tq, c.Hq, c.dv), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((c.Tq, c.Hq), device=DEV)
    ws = binding.tree_attention_workspace(q, c.cache, 4)

    def step():
        binding.rope_partial_tree_attention(q, c.cache, qs, ln, table, out, lse=lse, tree=tree, max_q=4,
                                            workspace=ws)

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
        c.slots = [c.table[r, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16
                   for r, n in enumerate(lens)]
        c.check(out, lse)
