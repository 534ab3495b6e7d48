"""Rounds of speculative decoding over a latent cache, all operators of a step together:
pages for the drafted tokens, their latent rows normed and turned, written, attended by
normed and turned queries, and the pages of what was not accepted given back.  Checked
against 64-bit sums over the rows that each request has accepted so far."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import step_ref
from gpu_util import DEV
from place_partial_rope_gb300 import binding

pytestmark = pytest.mark.gpu

H, LAT, ROT, PAGE, PAGES, ROOM = 6, 64, 32, 16, 40, 12
D = LAT + ROT


class Step:
    """What a serving program keeps, and one step over it."""

    def __init__(self, dtype, store, R, T, seed):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.R, self.T = dtype, R, T
        i32 = dict(dtype=torch.int32, device=DEV)
        kind = store or dtype
        self.rows = torch.zeros((PAGES, PAGE, 1, D), dtype=kind, device=DEV)
        self.scale = torch.zeros((PAGES, PAGE, 1), device=DEV) if store else None
        self.cache = binding.KVCache(self.rows, k_scale=self.scale)
        self.table = torch.full((R, ROOM), -1, **i32)
        self.free = torch.randperm(PAGES, generator=g).to(torch.int32).to(DEV)
        self.count = torch.tensor([PAGES], **i32)
        self.len, self.n, self.keep = (torch.zeros(R, **i32) for _ in range(3))
        self.q_start, self.granted = torch.zeros(R + 1, **i32), torch.zeros(R, **i32)
        self.slots, self.positions = torch.zeros(T, dtype=torch.int64, device=DEV), torch.zeros(T, **i32)
        angle = torch.arange(4096, dtype=torch.float64)[:, None] * 10000.0 ** -(torch.arange(ROT // 2).double() / (ROT // 2))
        self.cos, self.sin = (f(angle).repeat_interleave(2, -1).to(dtype).to(DEV) for f in (torch.cos, torch.sin))
        self.w = (1 + 0.2 * torch.randn(LAT, generator=g)).to(DEV)
        self.wq = (1 + 0.2 * torch.randn(LAT, generator=g)).to(DEV)
        self.x = torch.zeros((1, T, 1, D), dtype=dtype, device=DEV)
        self.q = torch.zeros((1, T, H, D), dtype=dtype, device=DEV)
        self.k, self.qn = torch.zeros_like(self.x), torch.zeros_like(self.q)
        self.out = torch.zeros((T, H, LAT), dtype=dtype, device=DEV)
        self.lse = torch.zeros((T, H), device=DEV)
        self.ws = binding.latent_attention_workspace(self.qn[0], self.cache, LAT, T)

    def __call__(self):
        binding.rope_partial_cache_grow(self.len, self.n, self.table, self.free, self.count, PAGE, self.q_start,
                                        self.slots, positions=self.positions, granted=self.granted)
        at = self.positions.long()
        cos, sin = self.cos[at][None, :, None], self.sin[at][None, :, None]
        binding.rope_partial_norm_fwd(self.x, None, self.w, None, cos, sin, LAT, D, norm=(0, LAT), q_out=self.k)
        binding.rope_partial_norm_fwd(self.q, None, self.wq, None, cos, sin, LAT, D, norm=(0, LAT), q_out=self.qn)
        binding.rope_partial_cache_write(self.cache, self.k[0], None, self.slots)
        binding.rope_partial_latent_attention(self.qn[0], self.cache, self.q_start, self.len, self.table, self.out,
                                              lse=self.lse, max_q=self.T, workspace=self.ws)
        binding.rope_partial_cache_trim(self.len, self.keep, self.table, self.free, self.count, PAGE)


@pytest.mark.parametrize("dtype,store,captured", [(torch.bfloat16, None, False), (torch.float16, torch.int8, False),
                                                  (torch.bfloat16, torch.float8_e4m3fn, True)])
def test_rounds(dtype, store, captured):
    rng = np.random.default_rng(1)
    R, T, rounds = 5, 64, 6
    s = Step(dtype, store, R, T, 3)
    graph = None
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s()  # no tokens yet
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s()
    have = [np.zeros((0, D)) for _ in range(R)]
    u, u_out = (2.0 ** -8 if dtype is torch.bfloat16 and not store else 2.0 ** -11), torch.finfo(dtype).eps / 2
    for _ in range(rounds):
        n = rng.integers(0, 13, R)
        kept = [int(rng.integers(0, a + 1)) for a in n]
        s.n.copy_(torch.from_numpy(n.astype(np.int32)))
        s.keep.copy_(torch.tensor([len(h) + a for h, a in zip(have, kept)], dtype=torch.int32))
        s.x.copy_(torch.from_numpy(rng.standard_normal((1, T, 1, D))))
        s.q.copy_(torch.from_numpy(rng.standard_normal((1, T, H, D))))
        s.out.fill_(9.0)
        graph.replay() if captured else s()
        torch.cuda.synchronize()
        assert s.granted.bool().all()
        start = np.concatenate([[0], np.cumsum(n)])
        assert s.q_start.tolist() == start.tolist() and (s.slots[start[-1]:] == -1).all()
        # the rows as the norm says, then as the cache holds them
        pos = np.concatenate([np.arange(len(h), len(h) + a) for h, a in zip(have, n)]).astype(int)
        assert s.positions[:start[-1]].tolist() == pos.tolist()
        cos, sin = (t.double().cpu().numpy()[pos][:, None] for t in (s.cos, s.sin))
        x = s.x.double().cpu().numpy()[0, :start[-1]]
        want, mag, _ = step_ref.norm_fwd(x, s.w.double().cpu().numpy(), cos, sin, LAT, D, 0, LAT, 1e-6, "interleave")
        k = s.k.double().cpu().numpy()[0, :start[-1]]
        assert np.all(abs(k - want) <= 2.0 ** -18 * mag + u_out * abs(want) * 1.01)
        if store:
            full = s.rows.view(torch.uint8).flatten(0, 1)[s.slots[:start[-1]]][:, 0].cpu().numpy()
            num = ref.fp8_values()[full] if store is torch.float8_e4m3fn else full.view(np.int8).astype(np.float64)
            rows = num * s.scale.flatten().double()[s.slots[:start[-1]]].cpu().numpy()[:, None]
            step = 2.0 ** -4 if store is torch.float8_e4m3fn else 2.0 ** -7  # of a value; of the row's largest
            assert np.all(abs(rows - k[:, 0]) <= step * abs(k[:, 0]).max(-1, keepdims=True))
        else:
            rows = s.rows.flatten(0, 2)[s.slots[:start[-1]]].double().cpu().numpy()
            assert np.array_equal(rows, k[:, 0])
        q, out, lse = (t.double().cpu().numpy() for t in (s.qn[0], s.out, s.lse))
        for r in range(R):
            at = slice(start[r], start[r + 1])
            all_rows = np.concatenate([have[r], rows[at]])
            sees = ref.tree_sees(int(n[r]), len(all_rows), len(have[r]), None)
            for h in range(H):
                o, l, m = ref.tree_attention(q[at, h], all_rows, all_rows[:, :LAT], sees, D ** -0.5)
                big = D ** -0.5 * (abs(q[at, h]) @ abs(all_rows).T).max(-1, initial=0)
                d = ((D + 8) * 2.0 ** -24 * big + 2.0 ** -21)[:, None]
                assert np.all(abs(out[at, h] - o) <= (u + 4 * d) * m + u_out * abs(o) + 1e-6), (r, h)
                assert np.all(abs(lse[at, h] - l) <= 2 * d[:, 0] + 2.0 ** -22 * abs(l))
            have[r] = all_rows[:len(have[r]) + kept[r]]
        assert (s.out[start[-1]:] == 9.0).all()  # tokens of no request
        assert s.len.tolist() == [len(h) for h in have]
    held = sum(-(-len(h) // PAGE) for h in have)
    assert s.count.tolist() == [PAGES - held]
    assert sorted(s.free[:PAGES - held].tolist() + [p for p in s.table.flatten().tolist() if p >= 0]) == list(range(PAGES))
