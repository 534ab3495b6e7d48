"""Pages dealt out to a batch of requests and taken back, on the GPU: whole numbers,
equal to those of the requests taken one by one on the host."""
import numpy as np
import pytest
import torch

import step_ref as ref
from gpu_util import DEV
from place_partial_rope_gb300 import binding

pytestmark = pytest.mark.gpu


def batch(R, page, len_hi, n_hi, spare, seed, room=0):
    rng = np.random.default_rng(seed)
    ln = rng.integers(0, len_hi + 1, R).astype(np.int32)
    n = rng.integers(0, n_hi + 1, R).astype(np.int32)
    held = -(-ln // page)
    wide = max(1, int((-(-(ln + n) // page)).max(initial=0)) + room)
    pages = rng.permutation(int(held.sum()) + spare).astype(np.int32)
    table = np.full((R, wide), -1, np.int32)
    at = 0
    for r in range(R):
        table[r, :held[r]] = pages[at:at + held[r]]
        at += held[r]
    free = np.full(len(pages) + 1, -9, np.int32)
    free[:spare] = pages[at:]
    return ln, n, table, free, spare


class State:
    def __init__(self, ln, n, table, free, count, page, T, stride=0):
        self.page, self.T = page, T
        self.ln, self.n, self.free = (torch.from_numpy(x.copy()).to(DEV) for x in (ln, n, free))
        self.wide = torch.full((table.shape[0], table.shape[1] + stride), 77, dtype=torch.int32, device=DEV)
        self.table = self.wide[:, :table.shape[1]]
        self.table.copy_(torch.from_numpy(table))
        self.count = torch.tensor([count], dtype=torch.int32, device=DEV)
        R = len(ln)
        self.q_start = torch.full((R + 1,), 5, dtype=torch.int32, device=DEV)
        self.slots = torch.full((T,), 5, dtype=torch.int64, device=DEV)
        self.positions = torch.full((T,), 5, dtype=torch.int32, device=DEV)
        self.granted = torch.full((R,), 5, dtype=torch.int32, device=DEV)

    def grow(self, optional=True, stream=None):
        binding.rope_partial_cache_grow(self.ln, self.n, self.table, self.free, self.count, self.page, self.q_start,
                                        self.slots, positions=self.positions if optional else None,
                                        granted=self.granted if optional else None, stream=stream)

    def trim(self, keep, stream=None):
        binding.rope_partial_cache_trim(self.ln, keep, self.table, self.free, self.count, self.page, stream=stream)


def same(got, want, what):
    assert np.array_equal(got.cpu().numpy(), want), what


def check_grow(s, ln, n, table, free, count, page, T):
    want = ref.grow(ln, n, table, free, count, page, T)
    s.grow()
    torch.cuda.synchronize()
    for got, w, what in zip((s.ln, s.table, s.count, s.q_start, s.slots, s.positions, s.granted),
                            (want[0], want[1], np.array([want[2]]), *want[3:]),
                            ("kv_len", "table", "count", "q_start", "slots", "positions", "granted")):
        same(got, w, what)
    same(s.free, free, "the stack is only read")
    assert (s.wide[:, table.shape[1]:] == 77).all()
    return want


CASES = [  # R, page, len_hi, n_hi, spare, T - tokens, stride
    (1, 64, 200, 1, 4, 0, 0),
    (1, 1, 5, 9, 20, 3, 1),
    (7, 16, 100, 40, 30, 5, 3),
    (7, 16, 100, 40, 6, 5, 3),        # runs out of pages on the way
    (7, 16, 100, 40, 0, 0, 0),        # none to begin with
    (300, 64, 5000, 4, 300, 20, 0),
    (513, 24, 900, 70, 600, -100, 2),  # more tokens than places, and than pages
    (2048, 16, 300, 3, 5000, 1, 0),
    (2049, 16, 300, 3, 500, 1, 0),
    (5000, 8, 60, 33, 30000, 7, 0),
    (64, 128, 4000, 9000, 6000, 0, 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_grow_and_trim(case):
    R, page, len_hi, n_hi, spare, more, stride = CASES[case]
    ln, n, table, free, count = batch(R, page, len_hi, n_hi, spare, case)
    T = max(0, int(n.sum()) + more)
    s = State(ln, n, table, free, count, page, T, stride)
    got = check_grow(s, ln, n, table, free, count, page, T)
    rng = np.random.default_rng(100 + case)
    keep = rng.integers(-3, len_hi + n_hi, R).astype(np.int32)
    keep[rng.random(R) < 0.3] = 0
    want = ref.trim(got[0], keep, got[1], free, got[2], page)
    s.trim(torch.from_numpy(keep).to(DEV))
    torch.cuda.synchronize()
    for g, w, what in zip((s.ln, s.table, s.free, s.count), (*want[:3], np.array([want[3]])),
                          ("kv_len", "table", "free", "count")):
        same(g, w, what)


def test_taken_back_leaves_all_as_it_was():
    ln, n, table, free, count = batch(777, 16, 500, 50, 900, 3)
    s = State(ln, n, table, free, count, 16, int(n.sum()))
    s.grow()
    assert int(s.granted.sum()) < 777
    s.trim(torch.from_numpy(ln).to(DEV))
    torch.cuda.synchronize()
    for got, w in ((s.ln, ln), (s.table, table), (s.free, free), (s.count, np.array([count]))):
        same(got, w, "as before")


def test_numbers_out_of_range():
    """Lengths below 0 and beyond the table, negative counts, tokens that no table has room
    for, a stack that counts more than it holds."""
    ln = np.array([-5, 3, 1 << 30, 16, 8], np.int32)
    n = np.array([4, -7, 0, 2 ** 31 - 1, 9], np.int32)
    table = np.arange(20, dtype=np.int32).reshape(5, 4)
    free = np.arange(100, 108, dtype=np.int32)
    s = State(ln, n, table, free, 50, 4, 6)
    s.grow()
    torch.cuda.synchronize()
    assert s.q_start.tolist() == [0, 4, 4, 4, 2 ** 31 - 1, 2 ** 31 - 1]
    assert s.granted.tolist() == [1, 1, 1, 0, 0]
    assert s.ln.tolist() == [4, 3, 16, 16, 8]
    assert s.count.tolist() == [7]
    assert s.slots.tolist() == [107 * 4, 107 * 4 + 1, 107 * 4 + 2, 107 * 4 + 3, -1, -1]
    assert s.positions.tolist() == [0, 1, 2, 3, 16, 17]
    assert s.table.tolist() == [[107, 1, 2, 3]] + table[1:].tolist()
    s.trim(torch.tensor([-1, 99, 0, 5, 8], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    # 7 on the stack and 1 + 4 + 2 that come back: it holds 8, and the uppermost are dropped
    assert s.ln.tolist() == [0, 3, 0, 5, 8] and s.count.tolist() == [8]
    assert s.free.tolist() == [100, 101, 102, 103, 104, 105, 106, 15]
    assert s.table.tolist() == [[-1, 1, 2, 3], [4, 5, 6, 7], [-1] * 4, [12, 13, -1, -1], [16, 17, 18, 19]]


def test_nothing():
    s = State(np.zeros(0, np.int32), np.zeros(0, np.int32), np.zeros((0, 1), np.int32), np.arange(3, dtype=np.int32),
              3, 16, 4)
    s.grow()
    s.trim(s.n)
    torch.cuda.synchronize()
    assert s.q_start.tolist() == [0] and s.slots.tolist() == [-1] * 4 and s.positions.tolist() == [0] * 4
    assert s.count.tolist() == [3]


def test_without_the_optional_outputs():
    ln, n, table, free, count = batch(33, 16, 50, 5, 40, 4)
    a, b = (State(ln, n, table, free, count, 16, int(n.sum())) for _ in range(2))
    a.grow()
    b.grow(optional=False)
    torch.cuda.synchronize()
    assert torch.equal(a.slots, b.slots) and torch.equal(a.table, b.table)
    assert (b.positions == 5).all() and (b.granted == 5).all()


def test_captured_rounds():
    """Three replays of a round (grow, some drafts accepted) walk on as three calls do, on a
    stream of their own."""
    ln, n, table, free, count = batch(200, 16, 300, 6, 400, 5, room=4)
    s = State(ln, n, table, free, count, 16, int(n.sum()))
    took = torch.from_numpy(np.random.default_rng(6).integers(0, 4, 200).astype(np.int32)).to(DEV)
    keep = torch.zeros_like(took)

    def round_():
        torch.add(s.ln, took, out=keep)
        s.grow()
        s.trim(keep)

    graph = torch.cuda.CUDAGraph()
    first = [t.clone() for t in (s.ln, s.table, s.free, s.count)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        round_()
    torch.cuda.synchronize()
    for t, x in zip((s.ln, s.table, s.free, s.count), first):
        t.copy_(x)
    with torch.cuda.graph(graph):
        round_()
    want = (ln, table, free, count)
    for _ in range(3):
        graph.replay()
        g = ref.grow(want[0], n, want[1], want[2], want[3], 16, s.T)
        want = ref.trim(g[0], want[0] + took.cpu().numpy(), g[1], want[2], g[2], 16)
    torch.cuda.synchronize()
    for got, w in zip((s.ln, s.table, s.free, s.count), (*want[:3], np.array([want[3]]))):
        same(got, w, "after three rounds")
    same(s.slots, g[4], "slots of the last")
