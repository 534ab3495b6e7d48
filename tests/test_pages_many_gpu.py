"""Pages taken back from a few long requests, and dealt out by every shape of grid: whole numbers, equal
to those of the requests taken one by one on the host."""
import numpy as np
import pytest
import torch

import step_ref as ref
from gpu_util import DEV
from test_pages_gpu import State, batch, check_grow, same

pytestmark = pytest.mark.gpu


def ended(R, rows, page, room=0):
    """R requests of `rows` rows each, whose pages lie in any order, and an empty stack."""
    held = -(-rows // page)
    order = np.random.default_rng(R).permutation(R * held).astype(np.int32)
    table = np.full((R, held + room), -1, np.int32)
    table[:, :held] = order.reshape(R, held)
    return np.full(R, rows, np.int32), np.zeros(R, np.int32), table, np.full(R * held, -9, np.int32), 0


@pytest.mark.parametrize("R", [1, 2, 32, 33, 512, 513])
@pytest.mark.parametrize("rows,page,room", [(70000, 16, 0), (3000, 1, 5), (900, 64, 100), (5, 2, 0)])
def test_pages_of_long_requests_come_back(R, rows, page, room):
    """All of them, of requests that have ended; then, of others, all but a few."""
    ln, n, table, free, count = ended(R, rows, page, room)
    rng = np.random.default_rng(R + page)
    for keep in (np.zeros(R, np.int32), rng.integers(0, rows + 1, R).astype(np.int32)):
        s = State(ln, n, table, free, count, page, 1)
        want = ref.trim(ln, keep, table, free, count, page)
        s.trim(torch.from_numpy(keep).to(DEV))
        torch.cuda.synchronize()
        for g, w, what in zip((s.ln, s.table, s.free, s.count), (*want[:3], np.array([want[3]])),
                              ("kv_len", "table", "free", "count")):
            same(g, w, what)


def test_few_requests_are_no_slower_than_more():
    """The pages of 32 requests of 131072 rows come back as fast as those of 33."""
    took = {}
    for R in (32, 33):
        ln, n, table, free, count = ended(R, 131072, 16)
        s = State(ln, n, table, free, count, 16, 1)
        keep = torch.zeros(R, dtype=torch.int32, device=DEV)
        held = s.table.clone()
        times = []
        for _ in range(8):
            s.table.copy_(held)
            s.ln.fill_(131072)
            s.count.zero_()
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            s.trim(keep)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        took[R] = min(times)
    assert took[32] < 1.5 * took[33], took


@pytest.mark.parametrize("T", [1024, 1025, 4096, 4097, 8192, 8193, 12000, 16383, 16384, 16385])
@pytest.mark.parametrize("R", [3, 512, 2048, 2049, 5000])
def test_grow_by_every_grid(T, R):
    """One block, clusters of 2 and 4 blocks, and the grid with a launch after it; requests that fill a
    chunk of 2048 and those that go on; twice, as the first call's lengths are the second's."""
    ln, n, table, free, count = batch(R, 16, 300, 2 * T // R, max(4, T // 20), T + R, room=2 * T // R // 16 + 2)
    s = State(ln, n, table, free, count, 16, T)
    got = check_grow(s, ln, n, table, free, count, 16, T)
    want = ref.grow(got[0], n, got[1], free, got[2], 16, T)
    s.grow()
    torch.cuda.synchronize()
    for g, w, what in zip((s.ln, s.table, s.count, s.q_start, s.slots, s.positions, s.granted),
                          (want[0], want[1], np.array([want[2]]), *want[3:]),
                          ("kv_len", "table", "count", "q_start", "slots", "positions", "granted")):
        same(g, w, what)
